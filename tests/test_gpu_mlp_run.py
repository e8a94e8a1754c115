"""The dense MLP as a layer uses it: dropout in front of the adapters, adapters on both
projections of the gated product, the down projection on MXFP4 weights with an
adapter beside it, dropout into the stream, and the whole way back; on a side stream,
in HIP graphs that are replayed, and on two streams at once."""

import numpy as np
import pytest
import torch

import group_limited_routing_amd as gl
import oracle

pytestmark = pytest.mark.gpu

R, E, P = 16, 3, 0.2


def _setup(T, H, F, seed):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(seed)

    def r(*shape, scale=1.0):
        return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16).to(dev)

    codes, scales = gl.mx4_quantize(r(H, F, scale=F ** -0.5))
    return dict(x=r(T, H), stream=r(T, H), wg=r(F, H, scale=H ** -0.5), wu=r(F, H, scale=H ** -0.5),
                codes=codes, scales=scales, gain=torch.ones(F, device=dev),
                ag=r(E, R, H, scale=H ** -0.5), bg=r(E, F, R, scale=0.1), au=r(E, R, H, scale=H ** -0.5),
                bu=r(E, F, R, scale=0.1), ad=r(E, R, F, scale=F ** -0.5), bd=r(E, H, R, scale=0.1),
                scale=torch.tensor([0.5, 1.0, 2.0], device=dev),
                index=torch.randint(-1, E, (T,), generator=g).to(torch.int32).to(dev),
                offset=torch.zeros(1, dtype=torch.int64, device=dev))


def _layer(p, stream=None):
    """Forward and backward; every output."""
    kw = dict(stream=stream)
    plan = gl.lora_plan(p["index"], E, **kw)
    xd = gl.dropout(p["x"], P, seed=1, offset=p["offset"], **kw)
    g = gl.lora(xd, p["ag"], p["bg"], plan, scale=p["scale"], return_v=True, **kw)
    u = gl.lora(xd, p["au"], p["bu"], plan, scale=p["scale"], return_v=True, **kw)
    m = gl.gated_linear(p["x"], p["wg"], p["wu"], add_gate=g["out"], add_up=u["out"], return_pre=True, **kw)
    q = gl.add_rms_norm(m["h"], p["gain"], quant="row", **kw)  # the rows of a quantised product
    down = gl.mx4_linear(q["q"], q["q_scale"], p["codes"], p["scales"], **kw)
    y = gl.lora(q["y"], p["ad"], p["bd"], plan, scale=p["scale"], base=down, return_v=True, **kw)
    out = gl.dropout(y["out"], P, seed=2, offset=p["offset"], stream_in=p["stream"], keep=0.75, add=0.5, **kw)
    # back, from out as its own gradient; the frozen product's gradient stands as zeros
    d = gl.dropout_backward(out, P, seed=2, offset=p["offset"], keep=0.75, add=0.5, stream_grad=True, **kw)
    by = gl.lora_backward(d["dx"], q["y"], y["v"], p["ad"], p["bd"], plan, scale=p["scale"], **kw)
    bh = gl.add_rms_norm_backward(by["dx"], m["h"], p["gain"], stream_grad=False, **kw)
    bm = gl.gated_linear_backward(bh["dx"], p["x"], p["wg"], p["wu"], m["gate"], m["up"], **kw)
    bg = gl.lora_backward(bm["d_gate"], xd, g["v"], p["ag"], p["bg"], plan, scale=p["scale"], **kw)
    bu = gl.lora_backward(bm["d_up"], xd, u["v"], p["au"], p["bu"], plan, scale=p["scale"], base=bg["dx"], **kw)
    bx = gl.dropout_backward(bu["dx"], P, seed=1, offset=p["offset"], **kw)
    return [xd, g["out"], g["v"], u["out"], m["h"], m["gate"], m["up"], down, y["out"], y["v"], out, d["dx"],
            d["d_stream_in"], by["dx"], by["d_a"], by["d_b"], bm["dx"], bm["d_w_gate"], bm["d_w_up"], bm["d_gate"],
            bm["d_up"], bg["d_a"], bg["d_b"], bu["dx"], bu["d_a"], bu["d_b"], bx["dx"]]


def _same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("T", [1, 70, 300])
def test_chain_against_float64(T):
    """The adapted gated product of dropped-out rows against the fp64 chain: the
    adapters' shares are rounded to bf16 once (2^-8), then h."""
    p = _setup(T, 264, 160, 91)
    r = _layer(p)
    f = lambda t: t.cpu().double().numpy()
    idx, sc = p["index"].cpu().numpy(), f(p["scale"])
    xd = f(r[0])  # a bf16 rounding of the dropped-out rows, checked in test_gpu_dropout.py
    g, _ = oracle.mlp.lora(xd, f(p["ag"]), f(p["bg"]), idx, sc)
    u, _ = oracle.mlp.lora(xd, f(p["au"]), f(p["bu"]), idx, sc)
    x, wg, wu = f(p["x"]), f(p["wg"]), f(p["wu"])
    h, gate, up = oracle.mlp.gated_linear(x, wg, wu, "silu", g, u)
    for got, ref, share in ((r[5], gate, g), (r[6], up, u)):
        tol = 2.0 ** -8 * (np.abs(ref) + 1.01 * np.abs(share)) + 2.0 ** -12
        assert (np.abs(f(got) - ref) <= tol).all()
    act = oracle.mlp.activation(gate, "silu")[0]
    tol = 2.0 ** -8 * (np.abs(h) + 1.2 * np.abs(g * up) + 1.01 * np.abs(act * u)) + 2.0 ** -12 * (1 + np.abs(up))
    assert (np.abs(f(r[4]) - h) <= 1.02 * tol).all()


@pytest.mark.parametrize("T", [1, 40, 300])
def test_layer_replays_in_graphs(T):
    """Captured layers equal the eager ones on every replay, with new inputs, new
    adapters for the tokens and a new mask in the captured buffers, eager work between
    the replays and a second graph beside it; then both at once."""
    p, q = _setup(T, 264, 256, 92), _setup(T, 264, 256, 93)
    graphs = []
    for s in (p, q):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _layer(s)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _layer(s)
        graphs.append((g, out))
    for i in range(4):
        for (g, out), s in zip(graphs, (p, q)):
            gen = torch.Generator().manual_seed(94 + i)
            s["x"].copy_(torch.randn(s["x"].shape, generator=gen))
            s["index"].copy_(torch.randint(-1, E, (T,), generator=gen))
            s["offset"].fill_(i)
            for o in out:
                o.fill_(7)
            g.replay()
            torch.cuda.synchronize()
            eager = _layer(s)
            torch.cuda.synchronize()
            assert _same(out, eager), i
    eager = [_layer(s) for s in (p, q)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for (g, _), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    assert all(_same(out, e) for (_, out), e in zip(graphs, eager))


def test_layer_on_side_streams():
    """``stream=``: the same bits, with the default stream writing over memory of the
    same sizes in between; two streams at once."""
    p, q = _setup(300, 264, 256, 95), _setup(300, 264, 256, 96)
    eager = [_layer(s) for s in (p, q)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    keep = []
    for _ in range(3):
        got = []
        for s, side in zip((p, q), sides):
            side.wait_stream(torch.cuda.current_stream())
            got.append(_layer(s, stream=side))
            junk = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
            junk.fill_(0xA5)
            keep.append(junk)
        for side in sides:
            side.synchronize()
        torch.cuda.synchronize()
        assert all(_same(a, b) for a, b in zip(got, eager))


def test_long_rows_past_32_bit_offsets():
    """More than 2^31 elements in a tensor: the last rows are those of a call on them
    alone (sums in whatever order a batch of its size takes, then one rounding)."""
    dev = torch.device("cuda:0")
    T, H, F = 270000, 64, 8192  # 2.2e9 outputs
    g = torch.Generator().manual_seed(97)
    x = torch.randn((T, H), generator=g).to(torch.bfloat16).to(dev)
    wg, wu = (torch.randn((F, H), generator=g).to(torch.bfloat16).to(dev) * H ** -0.5 for _ in range(2))
    big = gl.gated_linear(x, wg, wu, return_pre=True)
    few = gl.gated_linear(x[-3:].contiguous(), wg, wu, return_pre=True)
    for k in ("h", "gate", "up"):
        a, b = big[k][-3:].float(), few[k].float()
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -12).all(), k
    del big["h"]
    b = gl.gated_linear_backward(big["up"], x, wg, wu, big["gate"], big["up"], weight_grad=False)
    s = gl.gated_linear_backward(few["up"], x[-3:].contiguous(), wg, wu, few["gate"], few["up"],
                                 weight_grad=False)
    assert ((b["dx"][-3:].float() - s["dx"].float()).abs() <= 2.0 ** -6 * s["dx"].float().abs().max()).all()
    del b
    a, bb = torch.randn((2, 8, H), generator=g), torch.randn((2, F, 8), generator=g)
    a, bb = a.to(torch.bfloat16).to(dev), bb.to(torch.bfloat16).to(dev)
    index = torch.zeros(T, dtype=torch.int32, device=dev)
    index[-2:] = 1
    out = gl.lora(x, a, bb, gl.lora_plan(index, 2), base=big["gate"], out=big["gate"], return_v=True)
    one = gl.lora(x[-3:].contiguous(), a, bb, gl.lora_plan(index[-3:].clone(), 2), base=few["gate"])
    ref = one["out"].float()
    assert ((out["out"][-3:].float() - ref).abs() <= 2.0 ** -6 * (ref.abs() + few["gate"].float().abs() + 1)).all()
    bw = gl.lora_backward(big["up"], x, out["v"], a, bb, gl.lora_plan(index, 2))
    last = index == 1
    want = big["up"][last].double().t().contiguous() @ out["v"][last].double()
    err = bw["d_b"][1].double() - want
    assert (err.abs() <= 1.01 * 2.0 ** -8 * want.abs() + 2.0 ** -14 * want.abs().max()).all()
