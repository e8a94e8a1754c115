"""Oracle: the RMS norm of the residual stream with the stream's own update,
its E4M3 outputs, and its gradient, in float64.

Test infrastructure only; see the package docstring.

Launch post ("Introducing Beam"), section "Residual Stream": sandwich norm,
depth-scaled residual. Per row: s = keep * stream + add * x, y = s / sqrt(mean
of s^2 + eps) * gain. The E4M3 outputs are those of oracle.e4m3 on exact
quotients: per row with the scale amax / 448, or per 32 columns with the OCP
MXFP8 scale 2^(floor(log2 amax) - 8), at least 2^-127.
"""

import numpy as np

from . import e4m3

BLOCK = 32


def add_rms_norm(x, gain, eps, stream=None, keep=1.0, add=1.0):
    """(s, y) of [T, H] rows, float64."""
    s = add * np.asarray(x, dtype=np.float64)
    if stream is not None:
        s = s + keep * np.asarray(stream, dtype=np.float64)
    y = s / np.sqrt(np.mean(s * s, axis=1, keepdims=True) + eps) * np.asarray(gain, np.float64)
    return s, y


def quantize_row(y):
    """(codes [T, H] uint8, scale [T]): scale amax / 448 (1 for a row of zeros)."""
    amax = np.abs(y).max(axis=1)
    scale = np.where(amax > 0, amax / e4m3.FP8_MAX, 1.0)
    return e4m3.encode(y / scale[:, None]), scale


def quantize_block(y):
    """(codes [T, H] uint8, E8M0 bytes [T, H / 32])."""
    T, H = y.shape
    b = y.reshape(T, H // BLOCK, BLOCK)
    amax = np.abs(b).max(axis=2)
    _, ex = np.frexp(amax)
    e = np.where(amax > 0, np.clip(ex - 1 - 8, -127, 127), -127).astype(np.int64)
    return e4m3.encode(np.ldexp(b, -e[:, :, None]).reshape(T, H)), (e + 127).astype(np.uint8)


def add_rms_norm_backward(dy, s, gain, eps, d_stream=None, keep=1.0, add=1.0):
    """(dx, d_stream_in, d_gain)."""
    dy, s, gain = (np.asarray(a, dtype=np.float64) for a in (dy, s, gain))
    v = np.mean(s * s, axis=1, keepdims=True) + eps
    n = s / np.sqrt(v)
    g = dy * gain
    ds = (g - n * np.mean(g * n, axis=1, keepdims=True)) / np.sqrt(v)
    if d_stream is not None:
        ds = ds + np.asarray(d_stream, dtype=np.float64)
    return add * ds, keep * ds, np.sum(dy * n, axis=0)
