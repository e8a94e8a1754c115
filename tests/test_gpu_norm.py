"""GPU parity of the RMS norm with the residual's addition, its E4M3 outputs
and its gradient, against oracle.norm in float64.

Tolerances, with u = 2^-24 (half a step of fp32) and h the half step of the
output type: an fp32 value passes through at most 2 roundings for s, 3 for the
two products and the root, and the mean square's own error, halved by the
root: a sum of H <= 65536 squares is at most 64 terms in a thread, 6 lane steps
and 15 waves, each adding one rounding relative to the sum (all terms are
positive). That is at most 2 + 3 + (64 + 1 + 6 + 15) / 2 = 48 roundings; 64 are
allowed. The E4M3 codes and E8M0 bytes are decided in fp64 and have to be equal.
"""

import numpy as np
import pytest
import torch

import group_limited_routing_amd as gl
import oracle
from parity import Guarded, guarded_out

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
KEEP, ADD, EPS = (float(np.float32(v)) for v in (0.9534625892455924, 0.30151134457776363, 1e-5))


def _dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


def _rows(T, H, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, H), generator=g) * scale).to(dtype).to(_dev())


def _gain(H, seed):
    g = torch.Generator().manual_seed(seed)
    return (1.0 + 0.2 * torch.randn(H, generator=g)).to(_dev())


def f64(t):
    return t.detach().cpu().double().numpy()


def _close(got, ref, mag, what, roundings=64):
    """|got - ref| within the output's half step plus `roundings` of fp32 on `mag`."""
    tol = HALF[got.dtype] * (np.abs(ref) + roundings * U * mag) + roundings * U * mag + 1e-37
    err = np.abs(f64(got) - ref)
    assert (err <= tol).all(), (what, float((err / tol).max()))


SHAPES = [(1, 1), (3, 7), (5, 32), (2, 64), (130, 96), (9, 511), (4, 512), (33, 520), (17, 1001),
          (7, 2560), (64, 5120), (3, 8191), (2, 16384), (2, 16416), (1, 40961), (2, 65536)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", SHAPES)
def test_norm_values(T, H, dtype):
    dt = DT[dtype]
    x, st, w = _rows(T, H, dt, 1), _rows(T, H, dt, 2, 3.0), _gain(H, 3)
    for stream in (None, st):
        r = gl.add_rms_norm(x, w, stream_in=stream, keep=KEEP, add=ADD, norm_eps=EPS)
        s, y = oracle.norm.add_rms_norm(f64(x), f64(w), float(np.float32(EPS)),
                                        None if stream is None else f64(st), KEEP, ADD)
        mag = np.abs(f64(x)) * ADD + (0 if stream is None else np.abs(f64(st)) * KEEP)
        rms = np.sqrt(np.mean(s * s, 1, keepdims=True) + EPS)
        _close(r["y"], y, mag / rms * np.abs(f64(w)), "y")
        if stream is None:
            assert r["stream_out"] is None
        else:
            _close(r["stream_out"], s, mag, "stream_out")
        assert r["q"] is None and r["q_scale"] is None


@pytest.mark.parametrize("quant", ["row", "block"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [s for s in SHAPES if s[1] < 40000])
def test_norm_codes(T, H, dtype, quant):
    if quant == "block" and H % 32:
        with pytest.raises(gl.BeamMoeError):
            gl.add_rms_norm(_rows(T, H, DT[dtype], 4), _gain(H, 5), quant="block")
        return
    x, st, w = _rows(T, H, DT[dtype], 4), _rows(T, H, DT[dtype], 5, 2.0), _gain(H, 6)
    if T > 2:
        x[1], st[1] = 0.0, 0.0  # a row of zeros
        x[2, H // 2:], st[2, H // 2:] = 0.0, 0.0
        x[0] *= 1e-20  # a row that only eps keeps from underflow
        st[0] *= 1e-20
    r = gl.add_rms_norm(x, w, stream_in=st, keep=KEEP, add=ADD, norm_eps=EPS, quant=quant,
                        return_y=H % 64 == 0)
    assert (r["y"] is not None) == (H % 64 == 0)
    _, y = oracle.norm.add_rms_norm(f64(x), f64(w), float(np.float32(EPS)), f64(st), KEEP, ADD)
    codes = r["q"].view(torch.uint8).cpu().numpy()
    if quant == "row":
        ref, sc = oracle.norm.quantize_row(y)
        got = f64(r["q_scale"])
        assert (np.abs(got - sc) <= 1.001 * U * sc).all()  # one rounding
    else:
        ref, sc = oracle.norm.quantize_block(y)
        assert np.array_equal(r["q_scale"].cpu().numpy(), sc)
    # -0 and +0 are the same value
    assert np.array_equal(np.where(codes == 128, 0, codes), np.where(ref == 128, 0, ref))


def test_norm_non_finite_rows_stay_apart():
    """An infinity or NaN spoils its own row only (block scales: the NaN byte)."""
    x, w = _rows(6, 256, torch.float32, 7), _gain(256, 8)
    clean = gl.add_rms_norm(x, w, quant="block")
    x[1, 5], x[4, 200] = float("inf"), float("nan")
    for quant in (None, "row", "block"):
        r = gl.add_rms_norm(x, w, quant=quant)
        good = [0, 2, 3, 5]
        assert torch.isfinite(r["y"][good]).all() and torch.isnan(r["y"][4]).all()
        assert torch.isnan(r["y"][1, 5]) and (r["y"][1, :5] == 0).all()
        if quant == "row":
            assert torch.isfinite(r["q_scale"][good]).all() and torch.isnan(r["q_scale"][[1, 4]]).all()
        if quant == "block":
            assert torch.equal(r["q_scale"][good], clean["q_scale"][good])
            assert (r["q_scale"][4] == 255).all() and r["q_scale"][1, 0] == 255
            assert (r["q"].view(torch.uint8)[4] == 0x7F).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_in_place(dtype):
    """stream_out may be stream_in or x; the norm reads them first."""
    T, H = 50, 1000
    x, st, w = _rows(T, H, DT[dtype], 9), _rows(T, H, DT[dtype], 10), _gain(H, 11)
    ref = gl.add_rms_norm(x, w, stream_in=st, keep=KEEP, add=ADD, quant="row")
    for target in ("stream_in", "x"):
        a, b = x.clone(), st.clone()
        out = b if target == "stream_in" else a
        r = gl.add_rms_norm(a, w, stream_in=b, keep=KEEP, add=ADD, quant="row", stream_out=out)
        assert r["stream_out"].data_ptr() == out.data_ptr()
        for k in ("stream_out", "y", "q_scale"):
            assert torch.equal(r[k], ref[k]), (target, k)
        assert torch.equal(r["q"].view(torch.uint8), ref["q"].view(torch.uint8))


def test_norm_writes_its_rows_only():
    """Not a byte around the stream's rows or the backward's workspace changes."""
    for T, H in ((5, 1001), (3, 64), (2, 5120)):
        x, w = _rows(T, H, torch.bfloat16, 12), _gain(H, 13)
        g, out = guarded_out(x)
        gl.add_rms_norm(x, w, stream_in=x, stream_out=out)
        cfg = gl.BeamMoeNorm(H, gl.BEAM_BF16, 1.0, 1.0, 1e-6, 0)
        need = gl.lib().beam_moe_add_rms_norm_backward_workspace_bytes(cfg, T)
        ws = Guarded(need, _dev(), "workspace")
        gl.add_rms_norm_backward(x, x, w, workspace=ws.view)
        g.check()
        ws.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (70, 64), (5, 512), (1100, 96), (3500, 72), (33, 1001),
                                 (2049, 520), (300, 5120), (3, 16384), (2, 20000), (1, 65536)])
def test_norm_gradient(T, H, dtype):
    """ds adds two sums of H terms (at most 86 roundings each, one of them of
    terms with both signs: relative to the sum of magnitudes) and a few more
    roundings: 256 cover them. dw sums over rows: a group's rows one after the
    other, its groups 16 apart and 16 waves."""
    dt = DT[dtype]
    dy, s, d = _rows(T, H, dt, 14), _rows(T, H, dt, 15, 2.0), _rows(T, H, dt, 16)
    w = _gain(H, 17)
    for dso, keep in ((d, KEEP), (None, ADD)):
        r = gl.add_rms_norm_backward(dy, s, w, d_stream_out=dso, keep=keep, add=ADD, norm_eps=EPS)
        eps = float(np.float32(EPS))
        dx, dsi, dw = oracle.norm.add_rms_norm_backward(
            f64(dy), f64(s), f64(w), eps, None if dso is None else f64(d), keep, ADD)
        inv = 1 / np.sqrt(np.mean(f64(s) ** 2, 1, keepdims=True) + eps)
        n, g = np.abs(f64(s)) * inv, np.abs(f64(dy) * f64(w))
        mag = inv * (g + n * np.mean(g * n, 1, keepdims=True)) + (0 if dso is None else np.abs(f64(d)))
        _close(r["dx"], dx, ADD * mag, "dx", 256)
        _close(r["d_stream_in"], dsi, keep * mag, "d_stream_in", 256)
        assert (r["d_stream_in"] is r["dx"]) == (keep == ADD)
        _close(r["d_norm_weight"], dw, np.sum(np.abs(f64(dy)) * n, 0), "dw", 64 + T // 64 + 80)


def test_norm_gradient_parts_left_out():
    """Without the weight's or the stream's gradient the rest is the same, bit for bit."""
    T, H = 600, 1024
    dy, s, w = _rows(T, H, torch.bfloat16, 18), _rows(T, H, torch.bfloat16, 19), _gain(H, 20)
    full = gl.add_rms_norm_backward(dy, s, w, keep=KEEP, add=ADD)
    for kw in (dict(weight_grad=False), dict(stream_grad=False)):
        r = gl.add_rms_norm_backward(dy, s, w, keep=KEEP, add=ADD, **kw)
        assert torch.equal(r["dx"], full["dx"])
        if "weight_grad" in kw:
            assert r["d_norm_weight"] is None and torch.equal(r["d_stream_in"], full["d_stream_in"])
        else:
            assert r["d_stream_in"] is None and torch.equal(r["d_norm_weight"], full["d_norm_weight"])
    again = gl.add_rms_norm_backward(dy, s, w, keep=KEEP, add=ADD,
                                     workspace=torch.full((1 << 24,), 255, dtype=torch.uint8,
                                                          device=_dev()))
    assert torch.equal(again["d_norm_weight"], full["d_norm_weight"])


def test_norm_gradient_against_differences():
    """Central differences of the kernel's own forward (fp32), on a loss that
    weighs y and the stream."""
    T, H = 2, 40
    x, st, w = _rows(T, H, torch.float32, 21), _rows(T, H, torch.float32, 22), _gain(H, 23)
    dy, dso = _rows(T, H, torch.float32, 24), _rows(T, H, torch.float32, 25)

    def loss(x, st, w):
        r = gl.add_rms_norm(x, w, stream_in=st, keep=KEEP, add=ADD, norm_eps=EPS)
        return float((r["y"].double() * dy.double()).sum() + (r["stream_out"].double() * dso.double()).sum())

    s = gl.add_rms_norm(x, w, stream_in=st, keep=KEEP, add=ADD, norm_eps=EPS)["stream_out"]
    r = gl.add_rms_norm_backward(dy, s, w, d_stream_out=dso, keep=KEEP, add=ADD, norm_eps=EPS)
    h = 2.0 ** -6
    for i, name in enumerate(("dx", "d_stream_in", "d_norm_weight")):
        for at in (0, 7, 39):
            args = [[x, st, w], [x, st, w]]
            for side, sign in zip(args, (1, -1)):
                v = side[i].clone()
                v.view(-1)[at] += sign * h
                side[i] = v
            diff = (loss(*args[0]) - loss(*args[1])) / (2 * h)
            # third derivatives of order 1 times h^2 / 6, and 80 terms' fp32 roundings over 2 h
            assert abs(diff - float(r[name].view(-1)[at])) <= 10 * h * h / 6 + 80 * 4 * U / h, (name, at)


def test_norm_no_rows():
    x, w = _rows(0, 64, torch.bfloat16, 1), _gain(64, 2)
    r = gl.add_rms_norm(x, w, stream_in=x, quant="block")
    assert r["y"].shape == (0, 64) and r["q_scale"].shape == (0, 2)
    b = gl.add_rms_norm_backward(x, x, w)
    assert b["dx"].shape == (0, 64) and (b["d_norm_weight"] == 0).all()
