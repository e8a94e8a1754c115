"""GPU parity of the adapters and their gradients, against oracle.mlp in float64.

Tolerances. Products of bf16 values are exact in fp32, and a sum of K in fp32 is at
most 2 K 2^-24 of the magnitudes off (see test_gpu_gated.py). v and dv go into the
second product as a sum of two bf16 values: half a step of the second, 2^-8 of what
half a step of the first leaves, 2^-16. Scaling is one more fp32 rounding. Then half a
step of bf16, 2^-8, of the output.
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
SPLIT = 2.0 ** -16


def _dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


def _rand(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).to(_dev())


def _f(t):
    return t.cpu().double().numpy()


def _index(T, E, how, seed):
    """Adapters of the tokens: "mixed" (some without, some out of range), "runs", "one",
    "none", "last" (the last adapter alone)."""
    g = torch.Generator().manual_seed(seed)
    if how == "mixed":
        i = torch.randint(-1, E + 1, (T,), generator=g)
        i[i == E] = 1 << 30
    elif how == "runs":
        i = torch.randint(0, E, (T // 23 + 1,), generator=g).repeat_interleave(23)[:T]
    elif how == "one":
        i = torch.zeros(T)
    else:
        i = torch.full((T,), -5 if how == "none" else E - 1)
    return i.to(torch.int32).to(_dev())


def _inputs(T, K, N, R, E):
    return dict(x=_rand((T, K), 1), a=_rand((E, R, K), 2, K ** -0.5), b=_rand((E, N, R), 3, R ** -0.5),
                dy=_rand((T, N), 4), base=_rand((T, N), 5), dbase=_rand((T, K), 6),
                scale=(0.5 + torch.rand(E, generator=torch.Generator().manual_seed(7))).to(_dev()))


def _close(got, ref, e, name):
    err = np.abs(_f(got) - ref)
    assert (err <= HALF * (np.abs(ref) + e) + e).all(), (name, (err - HALF * np.abs(ref)).max())


def _check(p, index, scale, base, dbase):
    """Forward and backward on one batch; returns everything."""
    E = p["a"].shape[0]
    plan = gl.lora_plan(index, E)
    fw = gl.lora(p["x"], p["a"], p["b"], plan, scale=scale, base=base, return_v=True)
    idx = index.cpu().numpy()
    f = lambda t: None if t is None else _f(t)
    x, a, b, dy = (_f(p[k]) for k in ("x", "a", "b", "dy"))
    K, N, R = x.shape[1], b.shape[1], a.shape[1]
    out, v = oracle.mlp.lora(x, a, b, idx, f(scale), f(base))
    mag_out, mag_v = oracle.mlp.lora(abs(x), abs(a), abs(b), idx, f(scale))
    assert (np.abs(_f(fw["v"]) - v) <= (2 * K + 8) * U * mag_v).all()
    zero = 0.0 if base is None else np.abs(_f(base)) * 4 * U
    _close(fw["out"], out, ((2 * K + 4 * R + 8) * U + SPLIT) * mag_out + zero, "out")
    bw = gl.lora_backward(p["dy"], p["x"], fw["v"], p["a"], p["b"], plan, scale=scale, base=dbase)
    vs = _f(fw["v"])
    dx, da, db = oracle.mlp.lora_backward(dy, x, vs, a, b, idx, f(scale), f(dbase))
    mdx, mda, mdb = oracle.mlp.lora_backward(abs(dy), abs(x), abs(vs), abs(a), abs(b), idx, f(scale))
    zero = 0.0 if dbase is None else np.abs(_f(dbase)) * 4 * U
    T = x.shape[0]
    _close(bw["dx"], dx, ((2 * N + 4 * R + 8) * U + SPLIT) * mdx + zero, "dx")
    _close(bw["d_a"], da, ((2 * N + 4 * T + 64) * U + SPLIT) * mda, "d_a")
    _close(bw["d_b"], db, ((4 * T + 64) * U + SPLIT) * mdb, "d_b")
    live = (idx >= 0) & (idx < E)
    want = torch.zeros_like(fw["out"]) if base is None else base
    assert torch.equal(fw["out"][~live], want[~live]) and not fw["v"][~live].any()
    for e in set(range(E)) - set(idx[live].tolist()):
        assert not bw["d_a"][e].any() and not bw["d_b"][e].any(), e
    return plan, fw, bw


@pytest.mark.parametrize("how", ["mixed", "runs", "none", "last"])
@pytest.mark.parametrize("T,K,N,R,E", [(1, 8, 8, 8, 1), (1, 1000, 264, 16, 3), (2, 40, 1032, 24, 5), (17, 264, 136, 16, 4),
                                       (64, 520, 264, 32, 40), (65, 128, 520, 8, 2), (130, 328, 72, 64, 3),
                                       (200, 72, 328, 128, 2), (300, 1032, 40, 40, 7)])
def test_lora(T, K, N, R, E, how):
    p = _inputs(T, K, N, R, E)
    _check(p, _index(T, E, how, 11), p["scale"], p["base"], p["dbase"])


@pytest.mark.parametrize("T,R", [(1, 8), (600, 16), (1100, 64), (129, 112), (2100, 24), (4200, 8)])
def test_lora_one_adapter(T, R):
    """Training of one adapter: more tokens than a tile and than a chunk; without scale,
    base or the gradient's base."""
    p = _inputs(T, 264, 328, R, 1)
    _check(p, _index(T, 1, "one", 12), None, None, None)


def test_lora_larger():
    """Sizes of a layer, against fp64 on the GPU."""
    T, K, N, R, E = 1200, 5120, 2568, 16, 6
    p = _inputs(T, K, N, R, E)
    index = _index(T, E, "runs", 13)
    plan = gl.lora_plan(index, E)
    fw = gl.lora(p["x"], p["a"], p["b"], plan, scale=p["scale"], base=p["base"], return_v=True)
    bw = gl.lora_backward(p["dy"], p["x"], fw["v"], p["a"], p["b"], plan, scale=p["scale"], base=p["dbase"])
    out, dx = p["base"].double(), p["dbase"].double()
    for e in range(E):
        at = (index == e).nonzero()[:, 0]
        x, a, b, dy = p["x"][at].double(), p["a"][e].double(), p["b"][e].double(), p["dy"][at].double()
        s = float(p["scale"][e])
        v = x @ a.t().contiguous()
        out[at] += s * v @ b.t().contiguous()
        dv = s * dy @ b
        dx[at] += dv @ a
        for name, want in (("d_a", dv.t().contiguous() @ x), ("d_b", s * dy.t().contiguous() @ v)):
            err = bw[name][e].double() - want
            assert err.norm() <= 1.01 * HALF / 3 ** 0.5 * want.norm(), (name, e)
            assert (err.abs() <= 1.01 * HALF * want.abs() + 2.0 ** -14 * want.abs().max()).all()
    for got, want in ((fw["out"], out), (bw["dx"], dx)):
        err = got.double() - want
        assert err.norm() <= 1.01 * HALF / 3 ** 0.5 * want.norm()
        assert (err.abs() <= 1.01 * HALF * want.abs() + 2.0 ** -12).all()


@pytest.mark.parametrize("T,E,how", [(1, 1, "mixed"), (63, 2, "mixed"), (64, 1024, "mixed"), (1025, 3, "runs"),
                                     (5000, 1024, "mixed"), (20000, 9, "runs"), (9000, 1, "one"), (700, 4, "none")])
def test_plan(T, E, how):
    """The tokens in order of their adapter, stable, those without one last; tiles of at
    most 64 and chunks of at most 1024 tokens of one adapter."""
    index = _index(T, E, how, 14)
    need = gl.lib().beam_moe_lora_plan_bytes(T, E)
    buf = Guarded(need, _dev(), "plan")
    assert gl.lib().beam_moe_lora_plan(index.data_ptr(), T, E, buf.view.data_ptr(), need, None) == gl.BEAM_OK
    buf.check()
    plan = buf.view.view(torch.int32).cpu().numpy()
    i = index.cpu().numpy().astype(np.int64)
    g = np.where((i >= 0) & (i < E), i, E)
    up4 = lambda n: (n + 3) // 4 * 4
    order = plan[16:16 + T]
    assert np.array_equal(order, np.argsort(g, kind="stable"))
    used = min(E, T)
    most = T // 64 + min(E + 1, T)
    tiles = 16 + up4(T)
    tokens, chunks = tiles + 4 * most, tiles + 68 * most
    padded = first = 0
    want_tiles, want_chunks, firsts, slots = [], [], [], []
    for e in range(E + 1):
        c = int((g == e).sum())
        want_tiles += [(e if e < E else -1, first + j, min(64, c - j), padded + j) for j in range(0, c, 64)]
        if e < E:
            firsts.append(len(want_chunks))
            slots.append(sum(n for n in map(int, np.diff(firsts)) if n > 1) if c > 1024 else -1)
            want_chunks += [(e, first + j, min(1024, c - j), padded + j) for j in range(0, c, 1024)]
            padded += (c + 31) // 32 * 32
        first += c
    for at, limit, n, want in ((tiles, most, plan[0], want_tiles),
                               (chunks, T // 1024 + used, plan[1], want_chunks)):
        assert n == len(want) <= limit
        assert np.array_equal(plan[at:at + 4 * n].reshape(n, 4), np.array(want).reshape(n, 4))
    for i, (_, first, c, _) in enumerate(want_tiles):
        row = plan[tokens + 64 * i:tokens + 64 * i + 64]
        assert np.array_equal(row, order[np.minimum(np.arange(first, first + 64), first + c - 1)])
    at = chunks + 4 * (T // 1024 + used)
    assert plan[at:at + E + 1].tolist() == firsts + [len(want_chunks)]
    assert plan[at + up4(E + 1):at + up4(E + 1) + E].tolist() == slots


def test_rows_do_not_touch_each_other():
    """An infinity or a NaN in a token's row reaches that token's outputs, its own
    adapter's gradients, and nothing else; tokens without an adapter keep their base."""
    T, K, N, R, E = 90, 264, 136, 16, 3
    p = _inputs(T, K, N, R, E)
    index = torch.tensor([t % 4 - 1 for t in range(T)], dtype=torch.int32, device=_dev())
    plan = gl.lora_plan(index, E)

    def both(x, dy):
        fw = gl.lora(x, p["a"], p["b"], plan, scale=p["scale"], base=p["base"], return_v=True)
        return fw, gl.lora_backward(dy, x, fw["v"], p["a"], p["b"], plan, scale=p["scale"], base=p["dbase"])

    fw, bw = both(p["x"], p["dy"])
    x = p["x"].clone()
    x[0] = float("nan")      # no adapter
    x[6, 3] = float("inf")   # adapter 1
    fw2, bw2 = both(x, p["dy"])
    keep = [t for t in range(T) if t != 6]
    assert torch.equal(fw["out"][keep], fw2["out"][keep]) and not torch.isfinite(fw2["out"][6]).any()
    assert torch.equal(bw["dx"], bw2["dx"])
    for e in (0, 2):
        assert torch.equal(bw["d_a"][e], bw2["d_a"][e]) and torch.equal(bw["d_b"][e], bw2["d_b"][e])
    cols = [c for c in range(K) if c != 3]
    assert torch.equal(bw["d_a"][1][:, cols], bw2["d_a"][1][:, cols])
    assert not torch.isfinite(bw2["d_a"][1][:, 3]).any()
    dy = p["dy"].clone()
    dy[0] = float("inf")
    dy[9] = float("nan")     # adapter 0
    fw3, bw3 = both(p["x"], dy)
    keep = [t for t in range(T) if t != 9]
    assert torch.equal(bw["dx"][keep], bw3["dx"][keep]) and torch.isnan(bw3["dx"][9]).all()
    assert all(torch.equal(bw[k][1:], bw3[k][1:]) for k in ("d_a", "d_b"))
    # an adapter of NaN: only its own tokens
    a = p["a"].clone()
    a[2] = float("nan")
    out = gl.lora(p["x"], a, p["b"], plan, scale=p["scale"], base=p["base"])["out"]
    mine = (index == 2)
    assert torch.equal(out[~mine], fw["out"][~mine]) and torch.isnan(out[mine]).all()


def test_in_place_and_parts():
    T, K, N, R, E = 150, 328, 264, 24, 4
    p = _inputs(T, K, N, R, E)
    index = _index(T, E, "mixed", 15)
    plan, fw, bw = _check(p, index, p["scale"], p["base"], p["dbase"])
    out = p["base"].clone()
    r = gl.lora(p["x"], p["a"], p["b"], plan, scale=p["scale"], base=out, out=out)
    assert r["out"] is out and r["v"] is None and torch.equal(out, fw["out"])
    dx = p["dbase"].clone()
    args = (p["dy"], p["x"], fw["v"], p["a"], p["b"], plan)
    r = gl.lora_backward(*args, scale=p["scale"], base=dx, dx=dx, weight_grad=False)
    assert r["dx"] is dx and r["d_a"] is None and torch.equal(dx, bw["dx"])
    r = gl.lora_backward(*args, scale=p["scale"], input_grad=False)
    assert r["dx"] is None and torch.equal(r["d_a"], bw["d_a"]) and torch.equal(r["d_b"], bw["d_b"])
    r = gl.lora_backward(*args, scale=p["scale"], input_grad=False, weight_grad=False)
    assert r == {"dx": None, "d_a": None, "d_b": None}
    # a scale of zero switches an adapter off
    off = gl.lora(p["x"], p["a"], p["b"], plan, scale=torch.zeros(E, device=_dev()), base=p["base"])
    assert torch.equal(off["out"], p["base"])
    for _ in range(3):
        again = gl.lora_backward(*args, scale=p["scale"], base=p["dbase"])
        assert all(torch.equal(bw[k], again[k]) for k in bw)


@pytest.mark.parametrize("T,K,N,R,E", [(1, 72, 40, 8, 2), (70, 264, 136, 24, 3), (140, 136, 520, 48, 2)])
def test_writes_stay_inside(T, K, N, R, E):
    """Exactly sized outputs and workspaces between canaries, through the C ABI."""
    dev, L = _dev(), gl.lib()
    p = _inputs(T, K, N, R, E)
    plan = gl.lora_plan(_index(T, E, "mixed", 16), E)
    cfg = ctypes.byref(gl.BeamMoeLoraConfig(K, N, R, E, gl.BEAM_BF16))
    need = L.beam_moe_lora_workspace_bytes(cfg, T), L.beam_moe_lora_backward_workspace_bytes(cfg, T)
    g = {n: Guarded(b, dev, n) for n, b in (("out", 2 * T * N), ("v", 4 * T * R), ("dx", 2 * T * K),
                                            ("da", 2 * E * R * K), ("db", 2 * E * N * R), ("ws", need[0]),
                                            ("bws", need[1]))}
    ptr = {n: b.view.data_ptr() for n, b in g.items()}
    i = {n: t.data_ptr() for n, t in p.items()}
    assert L.beam_moe_lora(cfg, T, i["x"], i["a"], i["b"], i["scale"], plan.buffer.data_ptr(), i["base"], ptr["out"],
                           ptr["v"], ptr["ws"], need[0], None) == gl.BEAM_OK
    assert L.beam_moe_lora_backward(cfg, T, i["dy"], i["x"], ptr["v"], i["a"], i["b"], i["scale"],
                                    plan.buffer.data_ptr(), i["dbase"], ptr["dx"], ptr["da"], ptr["db"], ptr["bws"],
                                    need[1], None) == gl.BEAM_OK
    for b in g.values():
        b.check()
    fw = gl.lora(p["x"], p["a"], p["b"], plan, scale=p["scale"], base=p["base"], return_v=True)
    assert torch.equal(g["out"].tensor((T, N), torch.bfloat16), fw["out"])
    bw = gl.lora_backward(p["dy"], p["x"], fw["v"], p["a"], p["b"], plan, scale=p["scale"], base=p["dbase"])
    assert torch.equal(g["da"].tensor((E, R, K), torch.bfloat16), bw["d_a"])
    assert torch.equal(g["db"].tensor((E, N, R), torch.bfloat16), bw["d_b"])
    assert torch.equal(g["dx"].tensor((T, K), torch.bfloat16), bw["dx"])


def test_large_v():
    """A v beyond the largest bf16 number, and an infinite one: the second part of the
    split must not turn them into NaN."""
    x, a = torch.full((2, 8), 1.5 * 2.0 ** 60), torch.full((1, 8, 8), 2.0 ** 64)
    x[1] = float("inf")
    x[0, 1:] = 0
    x, a = x.to(torch.bfloat16).to(_dev()), a.to(torch.bfloat16).to(_dev())
    b = torch.zeros((1, 8, 8), dtype=torch.bfloat16, device=_dev())
    b[0, :, 0] = 1.0
    b[0, 1, 0] = 2.0 ** -10
    plan = gl.lora_plan(torch.zeros(2, dtype=torch.int32, device=_dev()), 1)
    r = gl.lora(x, a, b, plan, return_v=True)
    assert (r["v"][0] == 1.5 * 2.0 ** 124).all() and torch.isinf(r["v"][1]).all()
    assert r["out"][0, 0] == 1.5 * 2.0 ** 124 and r["out"][0, 1] == 1.5 * 2.0 ** 114
    assert r["out"][1, 0] != r["out"][1, 0] or torch.isinf(r["out"][1, 0])


def test_no_tokens():
    p = _inputs(0, 64, 32, 8, 2)
    plan = gl.lora_plan(torch.zeros(0, dtype=torch.int32, device=_dev()), 2)
    fw = gl.lora(p["x"], p["a"], p["b"], plan, return_v=True)
    assert fw["out"].shape == (0, 32) and fw["v"].shape == (0, 8)
    bw = gl.lora_backward(p["dy"], p["x"], fw["v"], p["a"], p["b"], plan)
    assert bw["dx"].shape == (0, 64) and not bw["d_a"].any() and not bw["d_b"].any()


@pytest.mark.parametrize("R", [16, 64])
@pytest.mark.parametrize("T", [70, 2100])
def test_residual_in_place(T, R):
    """out = x + s B A x in x's own memory, and its gradient in dy's: base and the result
    are also the operand."""
    N, E = 264, 3
    p, index = _inputs(T, N, N, R, E), _index(T, E, "mixed", T)
    plan = gl.lora_plan(index, E)
    x, dy = p["x"], p["dy"]
    a, b, scale = p["a"], p["b"], p["scale"]
    want = gl.lora(x, a, b, plan, scale=scale, base=x, return_v=True)
    x2 = x.clone()
    got = gl.lora(x2, a, b, plan, scale=scale, base=x2, out=x2, return_v=True)
    assert torch.equal(x2, want["out"]) and torch.equal(got["v"], want["v"])
    want = gl.lora_backward(dy, x, got["v"], a, b, plan, scale=scale, base=dy)
    dy2 = dy.clone()
    got2 = gl.lora_backward(dy2, x, got["v"], a, b, plan, scale=scale, base=dy2, dx=dy2)
    assert torch.equal(dy2, want["dx"])
    x3 = x.clone()
    got3 = gl.lora_backward(dy, x3, got["v"], a, b, plan, scale=scale, base=dy, dx=x3)
    assert torch.equal(x3, want["dx"])
    for g in (got2, got3):
        assert torch.equal(g["d_a"], want["d_a"]) and torch.equal(g["d_b"], want["d_b"])


@pytest.mark.parametrize("T", [5, 1030])
@pytest.mark.parametrize("K,N,R", [(72, 136, 8), (200, 72, 72)])
def test_adapters_without_tokens(T, K, N, R):
    """Their gradients are zeros in memory that held other values, whether an adapter can
    have several chunks of tokens or not."""
    E, dev, L = 40, _dev(), gl.lib()
    p = _inputs(T, K, N, R, E)
    index = (torch.arange(T) % 3 * 7).to(torch.int32).to(dev)  # adapters 0, 7 and 14
    plan = gl.lora_plan(index, E)
    v = gl.lora(p["x"], p["a"], p["b"], plan, return_v=True)["v"]
    cfg = ctypes.byref(gl.BeamMoeLoraConfig(K, N, R, E, gl.BEAM_BF16))
    ws = torch.full((L.beam_moe_lora_backward_workspace_bytes(cfg, T),), 255, dtype=torch.uint8, device=dev)
    da, db = (torch.full_like(p[k], float("nan")) for k in "ab")
    assert L.beam_moe_lora_backward(cfg, T, p["dy"].data_ptr(), p["x"].data_ptr(), v.data_ptr(), p["a"].data_ptr(),
                                    p["b"].data_ptr(), None, plan.buffer.data_ptr(), None, None, da.data_ptr(),
                                    db.data_ptr(), ws.data_ptr(), ws.numel(), None) == gl.BEAM_OK
    idle = torch.tensor([e not in (0, 7, 14) for e in range(E)], device=dev)
    for g in (da, db):
        assert (g[idle] == 0).all() and not g.isnan().any() and (g[~idle] != 0).any()
