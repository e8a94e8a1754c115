"""GPU parity of the routing of given logits and its gradient, against
oracle.gate in float64.

The chosen experts and their counts have to be equal: both sides decide in 64
bits, and equal keys go to the lower index. A weight is an fp64 value rounded
once: u = 2^-24, plus 2^-40 for the order of the sums. The gradient is fp32:
an exponential whose argument z - m is rounded (|z - m| u, at most 40 u here)
and is itself within 2 u; sums of at most 16 terms in a lane and 6 lane steps;
fewer than 20 further roundings: 100 u on the magnitude f (|df| + sum |df f|)
covers both.
"""

import numpy as np
import pytest
import torch

import group_limited_routing_amd as gl
import oracle

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


def _logits(T, E, seed, dtype="f32", scale=1.5):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=g) * scale).to(DT[dtype]).to(_dev())


def _vec(n, seed, scale):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, generator=g) * scale).to(_dev())


def f64(t):
    return t.detach().cpu().double().numpy()


def _check(z, k, bias=None, valid=None, kind="sigmoid", G=1, keep=1, pick="top2", renorm=True, rsf=1.0):
    r = gl.gate(z, top_k=k, expert_bias=bias, score=kind, n_group=G, topk_group=keep,
                group_score=pick, renormalise=renorm, routed_scaling_factor=rsf, valid=valid,
                return_counts=True)
    idx, w, counts = oracle.gate.gate(
        f64(z), k, None if bias is None else f64(bias), kind, G, keep, pick, renorm, rsf,
        None if valid is None else valid.cpu().numpy())
    assert np.array_equal(r["topk_idx"].cpu().numpy(), idx)
    assert np.array_equal(r["expert_counts"].cpu().numpy(), counts)
    assert (np.abs(f64(r["topk_w"]) - w) <= (U + 2.0 ** -40) * np.abs(w) + 2.0 ** -150).all()
    # the same tokens over and over in a batch of thousands, which other kernels take
    n = 4200 // z.shape[0] + 1
    many = gl.gate(z.repeat(n, 1), top_k=k, expert_bias=bias, score=kind, n_group=G, topk_group=keep,
                   group_score=pick, renormalise=renorm, routed_scaling_factor=rsf,
                   valid=None if valid is None else valid.repeat(n), return_counts=True)
    assert torch.equal(many["topk_idx"], r["topk_idx"].repeat(n, 1))
    assert torch.equal(many["expert_counts"], n * r["expert_counts"])
    # one rounding each of fp64 values that agree to 2^-40
    d = (many["topk_w"].double() - r["topk_w"].repeat(n, 1).double()).abs()
    assert (d <= (2 * U + 2.0 ** -39) * r["topk_w"].repeat(n, 1).abs() + 2.0 ** -149).all()
    return r


# T, E, groups, kept, k: one expert, fewer than a wave, ragged, every width of a lane's share
SHAPES = [(1, 1, 1, 1, 1), (5, 2, 1, 1, 2), (3, 5, 5, 2, 2), (37, 64, 1, 1, 6), (9, 65, 13, 4, 8),
          (130, 100, 4, 2, 7), (37, 160, 8, 3, 6), (66, 256, 8, 4, 8), (33, 256, 64, 9, 32),
          (4, 333, 3, 3, 16), (21, 512, 16, 5, 10), (40, 512, 1, 1, 16),
          (40, 320, 16, 4, 9), (40, 500, 2, 1, 8), (5, 1000, 8, 2, 12), (7, 1024, 1, 1, 32),
          (6, 1024, 64, 8, 8)]


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,G,keep,k", SHAPES)
def test_gate_values(T, E, G, keep, k, kind):
    for i, dtype in enumerate(("f32", "bf16")):
        z = _logits(T, E, 31 + i, dtype)
        bias = _vec(E, 33, 0.1)
        valid = (_vec(T, 34, 1.0) < 0.7)
        _check(z, k, None, None, kind, G, keep, "max", False, 2.5)
        _check(z, k, bias, valid, kind, G, keep, "top2", True, 2.5)
        _check(z, k, bias, None, kind, G, keep, "max", True, 1.0)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G,keep,k", [(256, 8, 4, 8), (160, 8, 3, 6), (60, 1, 1, 4),
                                        (512, 16, 5, 10), (333, 1, 1, 8)])
def test_gate_ties(E, G, keep, k, kind):
    """Logits of few values: equal keys and equal group scores go to the lower index."""
    z = torch.round(_logits(64, E, 35, scale=1.0))
    z[3] = 0.0
    bias = torch.round(_vec(E, 36, 1.0)) / 4
    for b in (None, bias):
        for pick in ("top2", "max"):
            _check(z, k, b, None, kind, G, keep, pick)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_gate_near_ties_are_decided_by_the_values(kind):
    """Neighbouring fp32 logits, whose scores are equal in fp32, and biases
    that bring them within 1e-9 of each other, in any order."""
    for E in (128, 400):
        base = torch.full((40, E), 0.75, device=_dev())
        step = torch.randint(-3, 4, (40, E), generator=torch.Generator().manual_seed(37)).to(_dev())
        z = (base.view(torch.int32) + step.int()).view(torch.float32)
        _check(z, 8, None, None, kind)
        _check(z, 8, _vec(E, 38, 1e-8), None, kind, 8, 3)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
def test_gate_masked_and_extreme_logits(kind):
    """-inf and NaN mask an expert; a row of nothing else has zero weights; +inf
    and far logits saturate; a bias of -inf or NaN sends its expert to the end."""
    inf = float("inf")
    z = _logits(12, 96, 39)
    z[0] = -inf
    z[1] = float("nan")
    z[2, 3:] = -inf          # fewer live experts than slots
    z[3, ::2] = float("nan")
    z[4, 7] = inf
    z[5, [7, 90]] = inf
    z[6] = 200.0
    z[7] = -200.0
    z[8] *= 60.0
    z[9, :] = -inf
    z[9, 95] = 0.0
    for G, keep in ((1, 1), (8, 2), (12, 5)):
        for renorm in (True, False):
            r = _check(z, 6, None, None, kind, G, keep, "top2", renorm)
            assert (r["topk_w"][:2] == 0).all()
    bias = _vec(96, 40, 0.1)
    bias[5], bias[6] = -inf, float("nan")
    _check(z, 6, bias, None, kind)
    _check(z, 6, bias, None, kind, 8, 3)


def test_gate_equals_the_blocks_route():
    """On beam_moe_route's own logits: the same experts and weights."""
    T, H = 200, 256
    g = torch.Generator().manual_seed(41)
    x = torch.randn((T, H), generator=g).to(_dev())
    rw = (torch.randn((256, H), generator=g) * H ** -0.5).to(_dev())
    b = _vec(256, 42, 0.1)
    r = gl.route(x, rw, b, return_logits=True, return_counts=True)
    q = gl.gate(r["router_logits"], top_k=8, expert_bias=b, n_group=8, topk_group=4,
                return_counts=True)
    # the block decides in fp32: tokens whose keys lie further apart have to agree
    far = oracle.route(f64(x), f64(rw), f64(b))["margin"] > 1e-5
    assert far.mean() > 0.9
    same = (r["topk_idx"] == q["topk_idx"]).all(1).cpu().numpy()
    assert same[far].all()
    d = (r["topk_w"] - q["topk_w"]).abs().cpu().numpy()[far]
    assert d.max() < 16 * U


def test_gate_many_tokens_count():
    """More tokens than fit the chip at once: the counts are those of the indices."""
    z = _logits(20011, 256, 43)  # a part of the tokens is decided over in fp64
    valid = torch.arange(20011, device=_dev()) % 7 != 0
    r = gl.gate(z, top_k=8, n_group=8, topk_group=4, valid=valid, return_counts=True)
    live = r["topk_idx"][valid].flatten().long()
    assert torch.equal(torch.bincount(live, minlength=256).int(), r["expert_counts"])
    assert (r["topk_idx"][~valid] == -1).all() and (r["topk_w"][~valid] == 0).all()
    again = gl.gate(z, top_k=8, n_group=8, topk_group=4, valid=valid)
    assert again["expert_counts"] is None
    assert torch.equal(again["topk_idx"], r["topk_idx"]) and torch.equal(again["topk_w"], r["topk_w"])


def _grad_check(dw, z, idx, kind, renorm, rsf):
    got = gl.gate_backward(dw, z, idx, score=kind, renormalise=renorm, routed_scaling_factor=rsf)
    assert got.dtype == z.dtype
    i = idx.cpu().numpy()
    ref = oracle.gate.gate_backward(f64(dw), f64(z), i, kind, renorm, rsf)
    # magnitudes: the same formulas with every term positive
    T, E = z.shape
    mag = np.zeros((T, E))
    for t in range(T):
        f, _ = oracle.gate.scores(f64(z)[t], kind)
        slots = [j for j in range(i.shape[1]) if 0 <= i[t, j] < E]
        e = i[t, slots]
        p, d = f[e], np.abs(f64(dw)[t, slots])
        df = d * rsf
        if renorm:
            S = p.sum()
            df = rsf / S * (d + (d * p).sum() / S) if S > 0 else 0 * d
        full = np.zeros(E)
        np.add.at(full, e, df)
        mag[t] = f * (full + (0 if kind == "sigmoid" or renorm else (df * p).sum()))
    half = 2.0 ** -8 if z.dtype == torch.bfloat16 else U
    # renormalised softmax: the oracle's inner sum is 0 but for fp64 rounding
    tol = half * np.abs(ref) + 100 * U * mag + 1e-15 * np.abs(rsf) * np.abs(f64(dw)).sum(1, keepdims=True) + 1e-37
    err = np.abs(f64(got) - ref)
    assert (err <= tol).all(), float((err / tol).max())
    return got


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,G,keep,k", SHAPES)
def test_gate_gradient(T, E, G, keep, k, kind, renorm):
    for i, dtype in enumerate(("f32", "bf16")):
        z = _logits(T, E, 44 + i, dtype)
        r = gl.gate(z, top_k=k, score=kind, n_group=G, topk_group=keep, renormalise=renorm,
                    valid=_vec(T, 46, 1.0) < 0.9)
        _grad_check(_vec(T * k, 47, 1.0).view(T, k), z, r["topk_idx"], kind, renorm, 2.5)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_gradient_odd_inputs(kind, renorm):
    """Masked and far logits, empty slots, the same expert in two slots."""
    z = _logits(8, 80, 48)
    z[0] = -float("inf")
    z[1, :40] = float("nan")
    z[2] *= 20.0
    idx = torch.stack([torch.randperm(80, generator=torch.Generator().manual_seed(49 + t))[:5]
                       for t in range(8)]).int().to(_dev())
    idx[3, 1:] = -1
    idx[4] = -1
    idx[5, 2], idx[5, 4] = 80, 1 << 30
    idx[6, 3] = idx[6, 0]
    got = _grad_check(_vec(40, 50, 1.0).view(8, 5), z, idx, kind, renorm, 1.5)
    assert (got[0] == 0).all() and (got[4] == 0).all()


def test_gate_gradient_against_differences():
    """Central differences of the forward's weights (fp32)."""
    z, k = _logits(2, 24, 51), 4
    dw = _vec(8, 52, 1.0).view(2, k)
    h = 2.0 ** -7
    for kind in ("sigmoid", "softmax"):
        for renorm in (True, False):
            r = gl.gate(z, top_k=k, score=kind, renormalise=renorm)
            g = gl.gate_backward(dw, z, r["topk_idx"], score=kind, renormalise=renorm)
            for at in [(0, int(r["topk_idx"][0, 1])), (1, int(r["topk_idx"][1, 3])), (0, 3)]:
                side = []
                for sign in (1, -1):
                    v = z.clone()
                    v[at] += sign * h
                    q = gl.gate(v, top_k=k, score=kind, renormalise=renorm)
                    # the same experts in the same order, or no difference can be taken
                    order = [q["topk_idx"][t].tolist().index(e) if e in q["topk_idx"][t].tolist() else None
                             for t in range(2) for e in r["topk_idx"][t].tolist()]
                    assert None not in order
                    w = q["topk_w"].gather(1, torch.tensor(order, device=z.device).view(2, k))
                    side.append(float((w.double() * dw.double()).sum()))
                diff = (side[0] - side[1]) / (2 * h)
                # third derivatives of these weights are below 1 per slot; 8 weights' roundings
                assert abs(diff - float(g[at])) <= 8 * h * h / 6 * 3 + 8 * 3 * U / h, (kind, renorm, at)


def test_gate_no_tokens():
    r = gl.gate(_logits(0, 16, 1), top_k=3, return_counts=True)
    assert r["topk_idx"].shape == (0, 3) and (r["expert_counts"] == 0).all()
    assert gl.gate_backward(torch.zeros((0, 3), device=_dev()), _logits(0, 16, 1),
                            r["topk_idx"]).shape == (0, 16)
