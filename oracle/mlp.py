"""Oracle: the dense MLP's gated product, low-rank adapters of many requests, and
dropout from a counter-based generator, with their gradients, in float64.

Test infrastructure only; see the package docstring.

Launch post ("Introducing Beam"), sections "Mixture of Experts" (dense SwiGLU in the
first layers) and "Post-training" (rank-16 adapters). The generator is Philox4x32-10
(Salmon et al., SC 2011).
"""

import math

import numpy as np

_ERFC = np.vectorize(math.erfc, otypes=[np.float64])


def activation(g, act):
    """act(g) and its derivative."""
    g = np.asarray(g, dtype=np.float64)
    if act == "silu":
        s = 1.0 / (1.0 + np.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    p = 0.5 * _ERFC(-g / math.sqrt(2.0))
    return g * p, p + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)


def gated_linear(x, wg, wu, act="silu", add_gate=0.0, add_up=0.0):
    """(h, gate, up)."""
    gate, up = x @ wg.T + add_gate, x @ wu.T + add_up
    return activation(gate, act)[0] * up, gate, up


def gated_linear_backward(dh, x, wg, wu, gate, up, act="silu"):
    """dict(d_gate, d_up, dx, d_w_gate, d_w_up)."""
    f, df = activation(gate, act)
    dg, du = dh * up * df, dh * f
    return dict(d_gate=dg, d_up=du, dx=dg @ wg + du @ wu, d_w_gate=dg.T @ x, d_w_up=du.T @ x)


def lora(x, a, b, index, scale=None, base=None):
    """(out, v): tokens one after the other."""
    T, R, N = x.shape[0], a.shape[1], b.shape[1]
    v = np.zeros((T, R))
    out = np.zeros((T, N)) if base is None else np.array(base, dtype=np.float64)
    for t in range(T):
        i = index[t]
        if 0 <= i < a.shape[0]:
            v[t] = a[i] @ x[t]
            out[t] += (1.0 if scale is None else scale[i]) * (b[i] @ v[t])
    return out, v


def lora_backward(dy, x, v, a, b, index, scale=None, base=None):
    """(dx, d_a, d_b)."""
    dx = np.zeros(x.shape) if base is None else np.array(base, dtype=np.float64)
    da, db = np.zeros(a.shape), np.zeros(b.shape)
    for t in range(x.shape[0]):
        i = index[t]
        if 0 <= i < a.shape[0]:
            f = 1.0 if scale is None else scale[i]
            dv = f * (b[i].T @ dy[t])
            dx[t] += a[i].T @ dv
            da[i] += np.outer(dv, x[t])
            db[i] += f * np.outer(dy[t], v[t])
    return dx, da, db


def philox(counter, key):
    """The four output words of Philox4x32-10 for a counter of four words and a key of two."""
    c, k, m = list(counter), list(key), 0xFFFFFFFF
    for _ in range(10):
        p, q = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(q >> 32) ^ c[1] ^ k[0], q & m, (p >> 32) ^ c[3] ^ k[1], p & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    return c


def random16(i, seed, offset):
    """The 16 bits of element i."""
    m = 0xFFFFFFFF
    w = philox([(i // 8) & m, (i // 8) >> 32, offset & m, offset >> 32], [seed & m, seed >> 32])
    return (w[i % 8 // 2] >> (16 * (i % 2))) & 0xFFFF


def dropout_factor(n, p, seed, offset=0, first=0):
    """What elements first .. first + n - 1 are multiplied with: 0 or 1 / (1 - q), q =
    p in steps of 1 / 65536."""
    border = math.floor(p * 65536 + 0.5)
    u = np.array([random16(i, seed, offset) for i in range(first, first + n)])
    return np.where(u >= border, 65536.0 / max(65536 - border, 1), 0.0)
