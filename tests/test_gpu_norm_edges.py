"""The RMS norm and its gradient at the ends of fp32's range and with values
that are not finite, against oracle.norm in float64. The tolerances are those
of test_gpu_norm.py, whose checks are used."""

import numpy as np
import pytest
import torch

import group_limited_routing_amd as gl
import oracle
from test_gpu_norm import ADD, DT, KEEP, _close, _dev, _gain, _rows, f64

pytestmark = pytest.mark.gpu

# rows whose squares are beyond fp32 at either end, and ordinary ones between
SCALES = [1e20, 1e-25, 1.0, 1e30, 1e-35, 3e37, 1e18, 1e-19]
SHAPES = [7, 64, 512, 1001, 5120, 20000]


def _wide_rows(H, dtype, seed):
    x = torch.cat([_rows(1, H, torch.float32, seed + i).clamp(-3, 3) * s for i, s in enumerate(SCALES)])
    return x.to(DT[dtype])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-30])
@pytest.mark.parametrize("H", SHAPES)
def test_norm_of_any_magnitude(H, eps, dtype):
    """The same y with and without codes, and the formula's, for rows of any size."""
    x, w = _wide_rows(H, dtype, 31), _gain(H, 32)
    _, y = oracle.norm.add_rms_norm(f64(x), f64(w), float(np.float32(eps)))
    mag = np.abs(y)
    plain, coded = gl.add_rms_norm(x, w, norm_eps=eps), gl.add_rms_norm(x, w, norm_eps=eps, quant="row")
    _close(plain["y"], y, mag, "y")
    _close(coded["y"], y, mag, "y with codes")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_of_large_rows_and_gains(dtype):
    """A product of row and gain beyond the largest number, whose norm is not."""
    x = _wide_rows(520, dtype, 33)
    w = _gain(520, 34) * 1e4
    _, y = oracle.norm.add_rms_norm(f64(x), f64(w), 0.0)
    _close(gl.add_rms_norm(x, w, norm_eps=0.0)["y"], y, np.abs(y), "y")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("eps", [0.0, 1e-30])
@pytest.mark.parametrize("H", SHAPES)
def test_norm_gradient_of_any_magnitude(H, eps, dtype):
    """As in test_norm_gradient. With rows of 1e37, 1 / rms is next to the
    smallest normal number, 2^-126, and gradients of the stream are subnormal:
    their last two fp32 roundings are off by 2^-150 each, and a bf16 one by 2^-134."""
    s, w = _wide_rows(H, dtype, 35), _gain(H, 36)
    T = s.shape[0]
    dy = _rows(T, H, DT[dtype], 37)
    eps = float(np.float32(eps))
    r = gl.add_rms_norm_backward(dy, s, w, keep=KEEP, add=ADD, norm_eps=eps)
    dx, dsi, dw = oracle.norm.add_rms_norm_backward(f64(dy), f64(s), f64(w), eps, None, KEEP, ADD)
    inv = 1 / np.sqrt(np.mean(f64(s) ** 2, 1, keepdims=True) + eps)
    n, g = np.abs(f64(s)) * inv, np.abs(f64(dy) * f64(w))
    mag = inv * (g + n * np.mean(g * n, 1, keepdims=True))
    big = float(torch.finfo(DT[dtype]).max)
    for name, ref, factor in (("dx", dx, ADD), ("d_stream_in", dsi, KEEP)):
        held = np.abs(ref) < big
        tol = 2.0 ** (-8 if dtype == "bf16" else -24) * np.abs(ref) + 512 * 2.0 ** -24 * factor * mag
        tol += 2.0 ** -149 + (2.0 ** -134 if dtype == "bf16" else 0.0)
        err = np.abs(np.where(held, f64(r[name]) - ref, 0.0))
        assert (err <= tol).all(), (name, float((err / tol).max()))
    _close(r["d_norm_weight"], dw, np.sum(np.abs(f64(dy)) * n, 0), "dw", 64 + T // 64 + 80)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", SHAPES)
def test_norm_gradient_in_place_of_any_magnitude(H, dtype):
    """dx over dy or s, whose rows out of range are read a second time."""
    s, w, dy = _wide_rows(H, dtype, 43), _gain(H, 44), _rows(8, H, DT[dtype], 45)
    ref = gl.add_rms_norm_backward(dy, s, w, norm_eps=0.0)["dx"]
    cfg = gl.BeamMoeNorm(H, gl.BEAM_BF16 if dtype == "bf16" else gl.BEAM_F32, 1.0, 1.0, 0.0, 0)
    for over in ("dy", "s"):
        a, b = dy.clone(), s.clone()
        dx = a if over == "dy" else b
        st = gl.lib().beam_moe_add_rms_norm_backward(
            cfg, 8, a.data_ptr(), b.data_ptr(), w.data_ptr(), None, dx.data_ptr(), None, None, None, 0,
            torch.cuda.current_stream().cuda_stream)
        assert st == gl.BEAM_OK and torch.equal(dx.nan_to_num(), ref.nan_to_num()), over


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [5, 64, 520, 5120])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_norm_codes_of_a_gain_that_is_not_finite(value, H, dtype):
    """Codes with row scales: no code stands for a NaN or an infinity of y by
    itself, so the row's scale does."""
    x, w = _rows(4, H, DT[dtype], 38), _gain(H, 39)
    w[H // 2] = value
    r = gl.add_rms_norm(x, w, quant="row")
    y = r["y"].float()
    assert not torch.isfinite(y[:, H // 2]).any() and torch.isfinite(y[:, :H // 2]).all()
    assert torch.isnan(r["q_scale"]).all()
    assert torch.isnan(r["q"].float() * r["q_scale"][:, None]).all()


def _steps(T, H):
    """Additions in a row on a weight gradient: the rows of a workgroup's thread,
    the four waves beside each other of narrow rows, a share's partials (32
    shares) and the shares."""
    per = 4 if H <= 512 else 1
    groups = min(-(-T // per), 768)
    return -(-T // (groups * per)) + (3 if per == 4 else 0) + -(-groups // 32) + 31


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 1), (70, 64), (1100, 96), (3500, 72), (33, 1001), (2049, 520), (5000, 512)])
def test_norm_weight_gradient_sums(T, H, dtype):
    """dw within the roundings of its own sum: each addition is at most u of the
    magnitudes' sum off, a term dy n has 48 roundings at most in n (see
    test_gpu_norm.py) and one for the product."""
    dy, s, w = _rows(T, H, DT[dtype], 40), _rows(T, H, DT[dtype], 41, 2.0), _gain(H, 42)
    got = gl.add_rms_norm_backward(dy, s, w, norm_eps=1e-6)["d_norm_weight"]
    eps = float(np.float32(1e-6))
    n = f64(s) / np.sqrt(np.mean(f64(s) ** 2, 1, keepdims=True) + eps)
    ref, mag = np.sum(f64(dy) * n, 0), np.sum(np.abs(f64(dy) * n), 0)
    err = np.abs(f64(got) - ref)
    tol = 2.0 ** -24 * (49 + _steps(T, H)) * 1.001 * mag
    assert (err <= tol).all(), float((err / tol).max())
