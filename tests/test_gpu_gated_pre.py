"""The gated product's gate and up kept in fp32, and the gradient from them: against
oracle.mlp in float64 with the bounds of test_gpu_gated.py, less the roundings to bf16
that are not made, through every kernel that writes them."""

import ctypes

import numpy as np
import pytest
import torch

import group_limited_routing_amd as gl
import oracle
from parity import Guarded
from test_gpu_gated import HALF, U, _act_err, _dev, _f, _rand

pytestmark = pytest.mark.gpu

SMALL = [(1, 8, 8), (1, 256, 1000), (16, 72, 264), (17, 512, 136), (33, 264, 520), (65, 64, 128), (131, 1000, 264),
         (257, 328, 520)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,H,F", SMALL)
def test_pair_and_gradient(T, H, F, act):
    """gate and up have the accuracy of their sums, and with it d_gate near the zeros of
    the activation's derivative, which a pair rounded to bf16 does not leave it: the
    error of gate counts with |act''|, at most 0.8."""
    x, wg, wu = _rand((T, H), 1), _rand((F, H), 2, 2 * H ** -0.5), _rand((F, H), 3, H ** -0.5)
    ag, au, dh = _rand((T, F), 4), _rand((T, F), 5), _rand((T, F), 6)
    fw = gl.gated_linear(x, wg, wu, activation=act, add_gate=ag, add_up=au, return_pre=True,
                         pre_dtype=torch.float32)
    bf = gl.gated_linear(x, wg, wu, activation=act, add_gate=ag, add_up=au, return_pre=True)
    assert fw["gate"].dtype == fw["up"].dtype == torch.float32
    for k in ("h", "gate", "up"):  # the same sums
        assert torch.equal(fw[k].to(torch.bfloat16), bf[k])
    xs, wgs, wus = _f(x), _f(wg), _f(wu)
    _, gate, up = oracle.mlp.gated_linear(xs, wgs, wus, act, _f(ag), _f(au))
    eg = (2 * H + 2) * U * (np.abs(xs) @ np.abs(wgs).T + np.abs(_f(ag)))
    eu = (2 * H + 2) * U * (np.abs(xs) @ np.abs(wus).T + np.abs(_f(au)))
    assert (np.abs(_f(fw["gate"]) - gate) <= eg).all() and (np.abs(_f(fw["up"]) - up) <= eu).all()
    r = gl.gated_linear_backward(dh, x, wg, wu, fw["gate"], fw["up"], activation=act)
    f, df = oracle.mlp.activation(gate, act)
    d, ed = np.abs(_f(dh)), 0.8 * eg + _act_err(gate, act, True)
    ef = 1.2 * eg + _act_err(gate, act) * np.abs(f) + 4 * U * np.abs(f)
    for name, ref, e in (("d_gate", _f(dh) * up * df, d * ((np.abs(up) + eu) * ed + np.abs(df) * eu)),
                         ("d_up", _f(dh) * f, d * ef)):
        e = e + 2.0 ** -30
        err = np.abs(_f(r[name]) - ref)
        assert (err <= HALF * (np.abs(ref) + e) + e).all(), (name, err.max())
    # the products are of these d_gate and d_up: as from any other pair
    dg, du = _f(r["d_gate"]), _f(r["d_up"])
    for name, pairs, K in (("dx", ((dg, wgs), (du, wus)), 2 * F), ("d_w_gate", ((dg.T, xs),), T),
                           ("d_w_up", ((du.T, xs),), T)):
        want = sum(a @ b for a, b in pairs)
        e = (2 * K + 64) * U * sum(np.abs(a) @ np.abs(b) for a, b in pairs)
        assert (np.abs(_f(r[name]) - want) <= HALF * (np.abs(want) + e) + e).all(), name


def test_zero_of_the_derivative():
    """gates of silu'(g) = 0 to fp32: d_gate is small, where a bf16 pair has 2^-8 |g| / 2 of
    dh up, and has it right to a bf16 rounding and the fp32 derivative's error."""
    z = -1.2784645427610738
    F, H = 64, 8
    x = torch.zeros((1, H), dtype=torch.bfloat16, device=_dev())
    w = torch.zeros((F, H), dtype=torch.bfloat16, device=_dev())
    one = torch.ones((1, F), device=_dev())
    g = torch.tensor([z * (1 + (i - 32) * 2.0 ** -14) for i in range(F)], dtype=torch.float64).float()[None].to(_dev())
    r = gl.gated_linear_backward(one.bfloat16(), x, w, w, g, one)
    want = oracle.mlp.activation(_f(g), "silu")[1]
    err = np.abs(_f(r["d_gate"]) - want)
    # s (1 + g (1 - s)) with |g| < 2: s one step off, the difference from 1 as many of 1
    assert (err <= HALF * np.abs(want) + 8 * U).all()
    assert np.abs(want).max() < 2.0 ** -8 and (_f(r["d_gate"]) * want >= 0).all()


@pytest.mark.parametrize("T,H,F", [(2552, 488, 3272), (6369, 392, 336), (67, 3984, 5592), (196, 128, 8440),
                                   (700, 5120, 320), (9, 264, 10240)])
def test_every_tile(T, H, F):
    """Whole and cut tiles of each size, against fp64 on the GPU: the sum's error as
    test_gpu_gated._near has it, half a step of fp32."""
    x, wg, wu = _rand((T, H), 1), _rand((F, H), 2, H ** -0.5), _rand((F, H), 3, H ** -0.5)
    r = gl.gated_linear(x, wg, wu, return_pre=True, pre_dtype=torch.float32)
    bf = gl.gated_linear(x, wg, wu, return_pre=True)
    for k, w in (("gate", wg), ("up", wu)):
        want = x.double() @ w.double().t().contiguous()
        err = (r[k].double() - want).abs()
        assert (err <= U * want.abs() + 16 * H ** 0.5 * U * want.abs().max()).all(), k
        assert torch.equal(r[k].to(torch.bfloat16), bf[k])
    assert torch.equal(r["h"], bf["h"])


@pytest.mark.parametrize("T,H,F", [(1, 72, 40), (30, 520, 136), (77, 328, 264), (300, 200, 264), (40, 4104, 72)])
def test_writes_stay_inside(T, H, F):
    dev, L = _dev(), gl.lib()
    x, wg, wu = _rand((T, H), 1), _rand((F, H), 2), _rand((F, H), 3)
    cfg = gl.BeamMoeGated(H, F, 0, gl.BEAM_BF16, 1)
    need = L.beam_moe_gated_linear_workspace_bytes(ctypes.byref(cfg), T)
    h, ws = Guarded(2 * T * F, dev, "h"), Guarded(max(need, 256), dev, "workspace")
    gate, up = Guarded(4 * T * F, dev, "gate"), Guarded(4 * T * F, dev, "up")
    assert L.beam_moe_gated_linear(ctypes.byref(cfg), T, x.data_ptr(), wg.data_ptr(), wu.data_ptr(), None, None,
                                   h.view.data_ptr(), gate.view.data_ptr(), up.view.data_ptr(), ws.view.data_ptr(),
                                   need, None) == gl.BEAM_OK
    for g in (h, ws, gate, up):
        g.check()
    r = gl.gated_linear(x, wg, wu, return_pre=True, pre_dtype=torch.float32)
    assert torch.equal(gate.tensor((T, F), torch.float32), r["gate"])
    assert torch.equal(up.tensor((T, F), torch.float32), r["up"])
    # d_gate and d_up in dh's memory and beside it
    dh = h.tensor((T, F), torch.bfloat16).clone()
    want = gl.gated_linear_backward(dh, x, wg, wu, r["gate"], r["up"], input_grad=False, weight_grad=False)
    du = Guarded(2 * T * F, dev, "d_up")
    assert L.beam_moe_gated_linear_backward(ctypes.byref(cfg), T, dh.data_ptr(), None, None, None,
                                            gate.view.data_ptr(), up.view.data_ptr(), dh.data_ptr(),
                                            du.view.data_ptr(), None, None, None, None, 0, None) == gl.BEAM_OK
    du.check()
    assert torch.equal(dh, want["d_gate"]) and torch.equal(du.tensor((T, F), torch.bfloat16), want["d_up"])
