"""Pins of the oracles of the norm and the routing of given logits: their
gradients against central differences of their own forwards, and special
cases with known answers."""

import numpy as np
import pytest

from oracle import e4m3, gate, norm, routing


def test_norm_special_cases():
    # a row of equal values has unit norm; the gain scales it
    s, y = norm.add_rms_norm(np.full((1, 8), 3.0), np.arange(8.0), 0.0)
    assert np.array_equal(s, np.full((1, 8), 3.0)) and np.allclose(y[0], np.arange(8.0), rtol=1e-15)
    # eps stands inside the root: mean square 1, eps 3 -> half
    _, y = norm.add_rms_norm(np.ones((1, 4)), np.ones(4), 3.0)
    assert np.array_equal(y, np.full((1, 4), 0.5))
    # the stream and the new part with their weights
    s, _ = norm.add_rms_norm(np.ones((1, 4)), np.ones(4), 1e-6, np.full((1, 4), 2.0), 0.5, 4.0)
    assert np.array_equal(s, np.full((1, 4), 5.0))


def test_norm_quantized_forms():
    rng = np.random.default_rng(0)
    y = rng.standard_normal((5, 96))
    y[2] = 0.0
    c, sc = norm.quantize_row(y)
    assert sc[2] == 1.0 and not c[2].any()
    assert np.abs(e4m3.decode(c)).max(axis=1)[[0, 1, 3, 4]].tolist() == [448.0] * 4
    c, b = norm.quantize_block(y)
    v = e4m3.decode(c).reshape(5, 3, 32) * np.exp2(b.astype(float) - 127)[:, :, None]
    # half a step of 3 mantissa bits, or the saturation of [448, 512)
    assert np.abs(v.reshape(5, 96) - y).max() <= np.abs(y).max() / 8
    assert (b[2] == 0).all()


@pytest.mark.parametrize("with_stream", [False, True])
def test_norm_gradient_against_differences(with_stream):
    rng = np.random.default_rng(1)
    T, H, eps, keep, add = 3, 7, 0.1, 0.8, 0.6
    x, st, gain = rng.standard_normal((T, H)), rng.standard_normal((T, H)), rng.standard_normal(H)
    dy, dso = rng.standard_normal((T, H)), rng.standard_normal((T, H))

    def loss(x, st, gain):
        s, y = norm.add_rms_norm(x, gain, eps, st if with_stream else None, keep, add)
        return (y * dy).sum() + (s * dso).sum()

    s, _ = norm.add_rms_norm(x, gain, eps, st if with_stream else None, keep, add)
    grads = norm.add_rms_norm_backward(dy, s, gain, eps, dso, keep, add)
    for i, (v, g) in enumerate(zip((x, st, gain), grads)):
        if i == 1 and not with_stream:
            continue
        for at in np.ndindex(v.shape):
            a = [x, st, gain]
            hi, lo = v.copy(), v.copy()
            hi[at] += 1e-5
            lo[at] -= 1e-5
            a[i] = hi
            up = loss(*a)
            a[i] = lo
            assert abs((up - loss(*a)) / 2e-5 - g[at]) < 1e-7, (i, at)


def test_gate_equals_the_blocks_routing():
    """Sigmoid, bias, 8 groups, top 2 of a group: the block's own routing oracle."""
    rng = np.random.default_rng(2)
    x, w, b = rng.standard_normal((40, 16)), rng.standard_normal((256, 16)), 0.1 * rng.standard_normal(256)
    ref = routing.route(x, w, b)
    idx, p, counts = gate.gate(x @ w.T, 8, b, n_group=8, topk_group=4)
    assert np.array_equal(idx, ref["idx"]) and np.allclose(p, ref["w"], rtol=1e-12)
    assert np.array_equal(counts, np.bincount(ref["idx"].ravel(), minlength=256))


def test_gate_masks_and_ties():
    z = np.zeros((3, 6))
    z[1, [0, 1]] = -np.inf
    z[2] = np.nan
    idx, w, counts = gate.gate(z, 2, kind="softmax")
    assert idx.tolist() == [[0, 1], [2, 3], [0, 1]]
    assert w.tolist() == [[0.5, 0.5], [0.5, 0.5], [0.0, 0.0]] and counts.sum() == 6
    idx, w, _ = gate.gate(z, 2, kind="softmax", valid=[1, 0, 1], renormalise=False)
    assert idx[1].tolist() == [-1, -1] and np.allclose(w[0], 1 / 6)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_gate_gradient_against_differences(kind, renormalise):
    rng = np.random.default_rng(3)
    T, E, k, rsf = 4, 9, 3, 2.5
    z, dw = rng.standard_normal((T, E)), rng.standard_normal((T, k))
    idx, _, _ = gate.gate(z, k, kind=kind)
    g = gate.gate_backward(dw, z, idx, kind, renormalise, rsf)

    def loss(z):
        total = 0.0
        for t in range(T):  # the chosen experts stay
            p = gate.scores(z[t], kind)[0][idx[t]]
            total += rsf * (dw[t] * (p / p.sum() if renormalise else p)).sum()
        return total

    for at in np.ndindex(z.shape):
        hi, lo = z.copy(), z.copy()
        hi[at] += 1e-5
        lo[at] -= 1e-5
        assert abs((loss(hi) - loss(lo)) / 2e-5 - g[at]) < 1e-7, at
