"""GPU parity of the gated product and its gradient, against oracle.mlp in float64.

Tolerances. Products of bf16 values are exact in fp32; a sum of K of them in fp32 is
at most 2 K 2^-24 of the sum of magnitudes off (one step for each addition, one for
the alignment inside a matrix instruction). The activation in fp32: its exponential
takes an argument that is 2^-24 |g| off and, as the reciprocal, gives about one step,
so act(g) is (|g| + 8) 2^-23 |act(g)| off (gelu: erfc's argument counts g^2 / 2 times,
(g^2 + 16) 2^-23), a derivative of at most 1.2 carries the error of g on, and the
derivative itself is (|g| + 16) 2^-22 off, gelu's (g^2 + 16) 2^-22. Then one rounding to bf16, half a
step, 2^-8. The products of the gradient are tested on the bf16 d_gate and d_up that
the call returns, which are their operands.
"""

import ctypes

import numpy as np
import pytest
import torch

import group_limited_routing_amd as gl
import oracle
from parity import Guarded

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = 2.0 ** -8


def _dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


def _rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).to(_dev())


def _f(t):
    return t.cpu().double().numpy()


def _act_err(g, act, deriv=False):
    base = np.abs(g) if act == "silu" else g * g
    return (base + 16) * 2.0 ** (-22 if deriv else -23)


def _near(got, want, K, name):
    """A sum of K products in fp32, rounded to bf16, for inputs with random signs. The
    rounding to bf16 has a root mean square of at most 2^-8 / sqrt(3) of the value. Those of
    the sum are as good as random: K^0.5 2^-24 of what it grows to on its way, which is below
    the largest result; 8 standard deviations for the elementwise bound, and twice that
    where a product of two such sums is taken."""
    err = got.double() - want
    assert err.norm() <= 1.01 * HALF / 3 ** 0.5 * want.norm(), name
    bound = HALF * want.abs() + 16 * K ** 0.5 * U * want.abs().max()
    assert (err.abs() <= bound).all(), (name, (err.abs() - bound).max())


def _check_forward(r, x, wg, wu, act, ag=None, au=None):
    xs, wgs, wus = _f(x), _f(wg), _f(wu)
    add = [0.0 if t is None else _f(t) for t in (ag, au)]
    h, gate, up = oracle.mlp.gated_linear(xs, wgs, wus, act, *add)
    K = xs.shape[1]
    eg = (2 * K + 2) * U * (np.abs(xs) @ np.abs(wgs).T + np.abs(add[0]))
    eu = (2 * K + 2) * U * (np.abs(xs) @ np.abs(wus).T + np.abs(add[1]))
    f = oracle.mlp.activation(gate, act)[0]
    eh = (1.2 * eg + _act_err(gate, act) * np.abs(f) + 2.0 ** -30) * (np.abs(up) + eu) + np.abs(f) * eu
    for name, ref, e in (("h", h, eh), ("gate", gate, eg), ("up", up, eu)):
        if r[name] is not None:
            err = np.abs(_f(r[name]) - ref)
            assert (err <= HALF * (np.abs(ref) + e) + e).all(), (name, err.max())


SHAPES = [(1, 8, 8), (1, 256, 1000), (2, 40, 24), (3, 1000, 136), (5, 2048, 64), (16, 72, 264), (17, 512, 136),
          (33, 264, 520), (64, 1032, 40), (65, 64, 128), (100, 136, 1000), (128, 512, 256), (131, 1000, 264),
          (257, 328, 520), (300, 2056, 136), (520, 96, 1288)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,H,F", SHAPES)
def test_gated_linear(T, H, F, act):
    x, wg, wu = _rand((T, H), 1), _rand((F, H), 2, 2 * H ** -0.5), _rand((F, H), 3, H ** -0.5)
    ag, au = _rand((T, F), 4), _rand((T, F), 5)
    full = gl.gated_linear(x, wg, wu, activation=act, add_gate=ag, add_up=au, return_pre=True)
    _check_forward(full, x, wg, wu, act, ag, au)
    plain = gl.gated_linear(x, wg, wu, activation=act)
    assert plain["gate"] is None and plain["up"] is None
    _check_forward(plain, x, wg, wu, act)
    # one of the two, and none: the same sums
    _check_forward(gl.gated_linear(x, wg, wu, activation=act, add_up=au), x, wg, wu, act, None, au)
    assert torch.equal(gl.gated_linear(x, wg, wu, activation=act, return_pre=True)["h"], plain["h"])


@pytest.mark.parametrize("T,H,F", [(700, 5120, 320), (64, 5120, 2560), (1030, 512, 2600), (2100, 264, 1032),
                                   (48, 2560, 10240), (2048, 1024, 2048)])
def test_gated_linear_larger(T, H, F):
    """Sizes of a layer, against fp64 on the GPU; see _near()."""
    x, wg, wu = _rand((T, H), 1), _rand((F, H), 2, H ** -0.5), _rand((F, H), 3, H ** -0.5)
    r = gl.gated_linear(x, wg, wu, return_pre=True)
    g = x.double() @ wg.double().t().contiguous()
    u = x.double() @ wu.double().t().contiguous()
    for name, ref in (("gate", g), ("up", u), ("h", g * torch.sigmoid(g) * u)):
        _near(r[name], ref, H, name)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,H,F", SHAPES)
def test_gated_linear_backward(T, H, F, act):
    x, wg, wu = _rand((T, H), 1), _rand((F, H), 2, H ** -0.5), _rand((F, H), 3, H ** -0.5)
    dh, gate, up = _rand((T, F), 6), _rand((T, F), 7, 2.0), _rand((T, F), 8)
    r = gl.gated_linear_backward(dh, x, wg, wu, gate, up, activation=act)
    ref = oracle.mlp.gated_linear_backward(*(_f(t) for t in (dh, x, wg, wu, gate, up)), act)
    f, _ = oracle.mlp.activation(_f(gate), act)
    mag = np.abs(_f(dh))
    for name, e in (("d_up", mag * np.abs(f) * (_act_err(_f(gate), act) + 4 * U)),
                    ("d_gate", mag * np.abs(_f(up)) * _act_err(_f(gate), act, True))):
        e = e + 2.0 ** -30
        err = np.abs(_f(r[name]) - ref[name])
        assert (err <= HALF * (np.abs(ref[name]) + e) + e).all(), name
    dg, du, xs, wgs, wus = (_f(t) for t in (r["d_gate"], r["d_up"], x, wg, wu))
    for name, pairs, K in (("dx", ((dg, wgs), (du, wus)), 2 * F), ("d_w_gate", ((dg.T, xs),), T),
                           ("d_w_up", ((du.T, xs),), T)):
        want = sum(a @ b for a, b in pairs)
        e = (2 * K + 64) * U * sum(np.abs(a) @ np.abs(b) for a, b in pairs)
        err = np.abs(_f(r[name]) - want)
        assert (err <= HALF * (np.abs(want) + e) + e).all(), (name, err.max())
    part = gl.gated_linear_backward(dh, x, wg, wu, gate, up, activation=act, input_grad=False)
    assert part["dx"] is None and torch.equal(part["d_w_up"], r["d_w_up"])
    part = gl.gated_linear_backward(dh, x, wg, wu, gate, up, activation=act, weight_grad=False)
    assert part["d_w_gate"] is None and torch.equal(part["dx"], r["dx"])
    assert torch.equal(part["d_gate"], r["d_gate"])


@pytest.mark.parametrize("T,H,F", [(1500, 1024, 512), (40, 5120, 2560), (3, 1024, 5000), (257, 520, 2056),
                                   (2048, 512, 1024), (4100, 264, 296), (1024, 2048, 1024)])
def test_gated_linear_backward_larger(T, H, F):
    x, wg, wu = _rand((T, H), 1), _rand((F, H), 2, H ** -0.5), _rand((F, H), 3, H ** -0.5)
    dh, gate, up = _rand((T, F), 6), _rand((T, F), 7), _rand((T, F), 8)
    r = gl.gated_linear_backward(dh, x, wg, wu, gate, up)
    dg, du, xd = r["d_gate"].double(), r["d_up"].double(), x.double()
    for name, want, K in (("dx", dg @ wg.double() + du @ wu.double(), 2 * F),
                          ("d_w_gate", dg.t().contiguous() @ xd, T), ("d_w_up", du.t().contiguous() @ xd, T)):
        _near(r[name], want, K, name)


def test_gradient_against_differences():
    """The returned gradients against central differences of the fp64 definition along
    random directions (bf16 gradients: half a step of each entry, added up)."""
    T, H, F = 9, 40, 24
    x, wg, wu, dh = _rand((T, H), 1), _rand((F, H), 2, 0.2), _rand((F, H), 3, 0.2), _rand((T, F), 6)
    fw = gl.gated_linear(x, wg, wu, return_pre=True)
    r = gl.gated_linear_backward(dh, x, wg, wu, fw["gate"], fw["up"])
    v = [_f(t) for t in (x, wg, wu)]
    rng = np.random.default_rng(0)
    for i, name in enumerate(("dx", "d_w_gate", "d_w_up")):
        d = rng.standard_normal(v[i].shape)
        step = 1e-5

        def loss(s):
            w = list(v)
            w[i] = w[i] + s * d
            return (oracle.mlp.gated_linear(*w)[0] * _f(dh)).sum()

        want = (loss(step) - loss(-step)) / (2 * step)
        g = _f(r[name])
        # the gradient's rounding, and those of gate, up, d_gate and d_up before it: each
        # 2^-8 of a factor, of magnitudes whose sum over the reduction is below 8 here
        tol = HALF * (np.abs(g * d).sum() + 4 * 8 * np.abs(d).sum())
        assert abs((g * d).sum() - want) <= tol


@pytest.mark.parametrize("T", [1, 20, 70, 200])
def test_rows_do_not_touch_each_other(T):
    """An infinity or a NaN in one token's row changes that row alone, and rows that a
    tile adds past the last token reach nothing."""
    H, F = 264, 136
    x, wg, wu = _rand((T, H), 1), _rand((F, H), 2, 0.1), _rand((F, H), 3, 0.1)
    clean = gl.gated_linear(x, wg, wu)["h"]
    bad = x.clone()
    bad[T - 1, 5], bad[T // 2, 7] = float("nan"), float("inf")
    h = gl.gated_linear(bad, wg, wu)["h"]
    keep = [t for t in range(T) if t not in (T - 1, T // 2)]
    assert torch.equal(h[keep], clean[keep])
    assert torch.isnan(h[T - 1]).all() and not torch.isfinite(h[T // 2]).any()
    # the last weight row
    w2 = wg.clone()
    w2[F - 1] = float("nan")
    h = gl.gated_linear(x, w2, wu)["h"]
    assert torch.equal(h[:, :F - 1], clean[:, :F - 1]) and torch.isnan(h[:, F - 1]).all()
    # gradients: a bad column of x spoils that column of the weights' gradients alone
    dh, gate, up = _rand((T, F), 6), _rand((T, F), 7), _rand((T, F), 8)
    good = gl.gated_linear_backward(dh, x, wg, wu, gate, up)
    bad = x.clone()
    bad[T - 1, H - 1] = float("inf")
    r = gl.gated_linear_backward(dh, bad, wg, wu, gate, up)
    assert torch.equal(r["d_w_gate"][:, :H - 1], good["d_w_gate"][:, :H - 1])
    assert not torch.isfinite(r["d_w_up"][:, H - 1]).any() and torch.equal(r["dx"], good["dx"])
    dh2 = dh.clone()
    dh2[0] = float("nan")
    r = gl.gated_linear_backward(dh2, x, wg, wu, gate, up)
    assert torch.equal(r["dx"][1:], good["dx"][1:]) and torch.isnan(r["dx"][0]).all()


def test_activation_tails():
    """gate from -inf to inf by add_gate alone: the values and the derivatives' limits."""
    vals = torch.tensor([-3e38, -200.0, -90.0, -20.0, -6.0, -1e-3, -0.0, 0.0, 1e-38, 1e-3, 6.0, 20.0, 90.0, 3e38,
                         -5.0, 5.0]).to(torch.bfloat16).to(_dev())
    F = vals.numel()
    x = torch.zeros((1, 8), dtype=torch.bfloat16, device=_dev())
    w = torch.zeros((F, 8), dtype=torch.bfloat16, device=_dev())
    one = torch.ones((1, F), dtype=torch.bfloat16, device=_dev())
    g = _f(vals)
    for act in ("silu", "gelu"):
        h = gl.gated_linear(x, w, w, activation=act, add_gate=vals[None].contiguous(), add_up=one)["h"]
        b = gl.gated_linear_backward(one, x, w, w, vals[None].contiguous(), one, activation=act)
        with np.errstate(over="ignore", invalid="ignore"):
            f, d = oracle.mlp.activation(np.clip(g, -700, 700), act)
            f = np.where(g > 700, g, f)
        for got, ref in ((h, f), (b["d_up"], f), (b["d_gate"], d)):
            err = np.abs(_f(got)[0] - ref)
            rel = HALF + _act_err(np.clip(g, -100, 100), act, True)
            assert (err <= rel * np.abs(ref) + 2.0 ** -100).all(), (act, g, _f(got), ref)


@pytest.mark.parametrize("T,H,F", [(1, 72, 40), (30, 520, 136), (77, 328, 264), (150, 72, 136), (300, 200, 264), (40, 4104, 72)])
def test_writes_stay_inside(T, H, F):
    """Exactly sized outputs between canaries, through the C ABI."""
    dev, L = _dev(), gl.lib()
    x, wg, wu = _rand((T, H), 1), _rand((F, H), 2), _rand((F, H), 3)
    cfg = gl.BeamMoeGated(H, F, 0, gl.BEAM_BF16)
    bufs = {n: Guarded(2 * T * F, dev, n) for n in ("h", "gate", "up", "dg", "du")}
    ptr = {n: g.view.data_ptr() for n, g in bufs.items()}
    need = L.beam_moe_gated_linear_workspace_bytes(ctypes.byref(cfg), T)
    fws = Guarded(max(need, 256), dev, "forward workspace")
    st = L.beam_moe_gated_linear(ctypes.byref(cfg), T, x.data_ptr(), wg.data_ptr(), wu.data_ptr(), None, None,
                                 ptr["h"], ptr["gate"], ptr["up"], fws.view.data_ptr(), need, None)
    assert st == gl.BEAM_OK
    fneed = need
    need = L.beam_moe_gated_linear_backward_workspace_bytes(ctypes.byref(cfg), T)
    ws = Guarded(max(need, 256), dev, "workspace")
    out = {"dx": Guarded(2 * T * H, dev, "dx"), "dwg": Guarded(2 * F * H, dev, "dwg"),
           "dwu": Guarded(2 * F * H, dev, "dwu")}
    st = L.beam_moe_gated_linear_backward(
        ctypes.byref(cfg), T, ptr["h"], x.data_ptr(), wg.data_ptr(), wu.data_ptr(), ptr["gate"], ptr["up"],
        ptr["dg"], ptr["du"], *(g.view.data_ptr() for g in out.values()), ws.view.data_ptr(), need, None)
    assert st == gl.BEAM_OK
    for g in [*bufs.values(), *out.values(), ws, fws]:
        g.check()
    fw = gl.gated_linear(x, wg, wu, return_pre=True)
    assert torch.equal(bufs["h"].tensor((T, F), torch.bfloat16), fw["h"])
    bw = gl.gated_linear_backward(fw["h"], x, wg, wu, fw["gate"], fw["up"])
    assert torch.equal(out["dx"].tensor((T, H), torch.bfloat16), bw["dx"])
    assert torch.equal(out["dwu"].tensor((F, H), torch.bfloat16), bw["d_w_up"])
    # in place: gate and up over add_gate and add_up, d_gate and d_up over gate and up
    ag, au = _rand((T, F), 4), _rand((T, F), 5)
    ref = gl.gated_linear(x, wg, wu, add_gate=ag, add_up=au, return_pre=True)
    dh = _rand((T, F), 6)
    bref = gl.gated_linear_backward(dh, x, wg, wu, ref["gate"], ref["up"])
    h = torch.empty_like(ag)
    assert L.beam_moe_gated_linear(ctypes.byref(cfg), T, x.data_ptr(), wg.data_ptr(), wu.data_ptr(), ag.data_ptr(),
                                   au.data_ptr(), h.data_ptr(), ag.data_ptr(), au.data_ptr(), fws.view.data_ptr(),
                                   fneed, None) == gl.BEAM_OK
    assert torch.equal(ag, ref["gate"]) and torch.equal(au, ref["up"]) and torch.equal(h, ref["h"])
    assert L.beam_moe_gated_linear_backward(
        ctypes.byref(cfg), T, dh.data_ptr(), x.data_ptr(), wg.data_ptr(), wu.data_ptr(), ag.data_ptr(),
        au.data_ptr(), ag.data_ptr(), au.data_ptr(), *(g.view.data_ptr() for g in out.values()),
        ws.view.data_ptr(), need, None) == gl.BEAM_OK
    assert torch.equal(ag, bref["d_gate"]) and torch.equal(au, bref["d_up"])
    assert torch.equal(out["dwg"].tensor((F, H), torch.bfloat16), bref["d_w_gate"])


def test_no_tokens():
    x, wg = torch.zeros((0, 64), dtype=torch.bfloat16, device=_dev()), _rand((32, 64), 1)
    r = gl.gated_linear(x, wg, wg, return_pre=True)
    assert r["h"].shape == (0, 32) and r["gate"].shape == (0, 32)
    b = gl.gated_linear_backward(r["h"], x, wg, wg, r["gate"], r["up"])
    assert b["dx"].shape == (0, 64) and not b["d_w_gate"].any() and b["d_w_up"].shape == (32, 64)


def test_deterministic():
    T, H, F = 333, 776, 520
    x, wg, wu = _rand((T, H), 1), _rand((F, H), 2), _rand((F, H), 3)
    a = gl.gated_linear(x, wg, wu, return_pre=True)
    b1 = gl.gated_linear_backward(a["h"], x, wg, wu, a["gate"], a["up"])
    for _ in range(3):
        again = gl.gated_linear(x, wg, wu, return_pre=True)
        assert all(torch.equal(a[k], again[k]) for k in a)
        b2 = gl.gated_linear_backward(a["h"], x, wg, wu, a["gate"], a["up"])
        assert all(torch.equal(b1[k], b2[k]) for k in b1)
