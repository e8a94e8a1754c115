"""The operators as a layer uses them together: the stream's update and norm
with E4M3 rows, the dense MXFP4 product on those rows, routing of logits made
from the normalised rows, and the way back; on a side stream, in a HIP graph
that is replayed, and on another stream's memory."""

import numpy as np
import pytest
import torch

import group_limited_routing_amd as gl
import oracle

pytestmark = pytest.mark.gpu


def _setup(T, H, N, seed):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(seed)
    x, st = (torch.randn((T, H), generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    gain = (1 + 0.1 * torch.randn(H, generator=g)).to(dev)
    w = (torch.randn((N, H), generator=g) * H ** -0.5).to(torch.bfloat16).to(dev)
    codes, scales = gl.mx4_quantize(w)
    return dict(x=x, st=st, gain=gain, codes=codes, scales=scales, bias=torch.zeros(96, device=dev))


def _layer(p, quant, stream=None):
    """One layer's operators; every output."""
    n = gl.add_rms_norm(p["x"], p["gain"], stream_in=p["st"], keep=0.75, add=0.5, quant=quant,
                        stream=stream)
    if stream is not None:
        torch.cuda.current_stream().wait_stream(stream)
    logits = n["y"][:, :96].float().contiguous()  # stands for a router's product
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    out = gl.mx4_linear(n["q"], n["q_scale"], p["codes"], p["scales"], stream=stream)
    r = gl.gate(logits, top_k=4, expert_bias=p["bias"], score="softmax", n_group=8, topk_group=3,
                return_counts=True, stream=stream)
    dz = gl.gate_backward(r["topk_w"], logits, r["topk_idx"], score="softmax", stream=stream)
    b = gl.add_rms_norm_backward(n["y"], n["stream_out"], p["gain"], d_stream_out=p["x"], keep=0.75,
                                 add=0.5, stream=stream)
    c4, s4 = gl.mx4_quantize(n["y"], stream=stream)
    out4 = gl.mx4_linear(c4, s4, p["codes"], p["scales"], out_dtype=torch.float32, stream=stream)
    v4 = gl.mx4_dequantize(c4, s4, stream=stream)
    return [n["stream_out"], n["y"], n["q"].view(torch.uint8), n["q_scale"], logits, out, r["topk_idx"],
            r["topk_w"], r["expert_counts"], dz, b["dx"], b["d_stream_in"], b["d_norm_weight"], c4, s4,
            out4, v4]


def _same(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("quant", ["row", "block"])
@pytest.mark.parametrize("T", [1, 70, 400])
def test_layer_against_float64(T, quant):
    """The chain's product against the exact product of the exact norm and the
    dequantised weights: what is left is the E4M3 rounding of the rows (half a
    step, 2^-4 per element, independent signs) and the output's."""
    p = _setup(T, 512, 384, 81)
    out = _layer(p, quant)[5].cpu().double().numpy()
    f = lambda t: t.cpu().double().numpy()
    _, y = oracle.norm.add_rms_norm(f(p["x"]), f(p["gain"]), float(np.float32(1e-6)), f(p["st"]), 0.75, 0.5)
    w = oracle.mxfp4.dequantize(p["codes"].cpu().numpy(), p["scales"].cpu().numpy())
    # a code is at most 2^-4 |y| off (or half the smallest step of its row or block)
    step = 2.0 ** -10 * np.abs(y).max(axis=1, keepdims=True) / 2.0 ** 7
    tol = (2.0 ** -4 * np.abs(y) + step) @ np.abs(w).T + 2.0 ** -8 * np.abs(y @ w.T) * 1.07
    err = np.abs(out - y @ w.T)
    assert (err <= tol).all()
    assert np.linalg.norm(err) <= 0.04 * np.linalg.norm(y @ w.T)


@pytest.mark.parametrize("T", [3, 64, 300])
def test_layer_replays_in_a_graph(T):
    """A captured layer equals the eager one on every replay, with eager work
    between the replays, new inputs in the captured buffers, and a second graph
    captured beside it."""
    p, q = _setup(T, 512, 384, 82), _setup(T, 512, 384, 83)
    graphs = []
    for s in (p, q):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _layer(s, "block")
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _layer(s, "block")
        graphs.append((g, out))
    for i in range(4):
        for (g, out), s in zip(graphs, (p, q)):
            s["x"].copy_(torch.randn(s["x"].shape, generator=torch.Generator().manual_seed(84 + i)))
            for o in out:
                o.fill_(7)
            g.replay()
            torch.cuda.synchronize()
            eager = _layer(s, "block")
            torch.cuda.synchronize()
            assert _same(out, eager), i
    # both at once, on two streams
    eager = [_layer(s, "block") for s in (p, q)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for (g, _), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    assert all(_same(out, e) for (_, out), e in zip(graphs, eager))


def test_layer_on_a_side_stream():
    """``stream=``: the same bits, with the default stream writing over memory of
    the same sizes in between; two streams at once."""
    p, q = _setup(300, 512, 384, 85), _setup(300, 512, 384, 86)
    eager = [_layer(s, "row") for s in (p, q)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    keep = []
    for _ in range(3):
        got = []
        for s, side in zip((p, q), sides):
            side.wait_stream(torch.cuda.current_stream())
            got.append(_layer(s, "row", stream=side))
            junk = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
            junk.fill_(0xA5)
            keep.append(junk)
        for side in sides:
            side.synchronize()
        torch.cuda.synchronize()
        assert all(_same(a, b) for a, b in zip(got, eager))


def test_long_rows_past_32_bit_offsets():
    """More than 2^31 elements in one call: the last rows are those of a call
    on them alone."""
    dev = torch.device("cuda:0")
    T, H = 140000, 16384  # 2.3e9 elements
    x = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    x.copy_(torch.randn((1, H), generator=torch.Generator().manual_seed(87)).to(torch.bfloat16))
    x[-3:] = torch.randn((3, H), generator=torch.Generator().manual_seed(88)).to(torch.bfloat16).to(dev)
    gain = torch.ones(H, device=dev)
    big = gl.add_rms_norm(x, gain, quant="block")
    few = gl.add_rms_norm(x[-3:].contiguous(), gain, quant="block")
    assert torch.equal(big["y"][-3:], few["y"]) and torch.equal(big["q_scale"][-3:], few["q_scale"])
    assert torch.equal(big["q"][-3:].view(torch.uint8), few["q"].view(torch.uint8))
    g = gl.add_rms_norm_backward(x, x, gain, weight_grad=False)["dx"]
    assert torch.equal(g[-3:], gl.add_rms_norm_backward(x[-3:].contiguous(), x[-3:].contiguous(), gain,
                                                        weight_grad=False)["dx"])
    del g
    c, s = gl.mx4_quantize(x)
    c1, s1 = gl.mx4_quantize(x[-3:].contiguous())
    assert torch.equal(c[-3:], c1) and torch.equal(s[-3:], s1)
    assert torch.equal(gl.mx4_dequantize(c, s)[-3:], gl.mx4_dequantize(c1, s1))
    del big, x
    torch.cuda.empty_cache()
    w, ws = c[:16384, :256].contiguous(), s[:16384, :16].contiguous()
    xt, xts = c[:, :256].contiguous(), s[:, :16].contiguous()  # [140000, 512]
    xt[-3:], xts[-3:] = c1[:, :256], s1[:, :16]
    out = gl.mx4_linear(xt, xts, w, ws)  # 2.3e9 outputs
    few = gl.mx4_linear(xt[-200:].contiguous(), xts[-200:].contiguous(), w, ws, out_dtype=torch.float32)
    # fp32 sums in whatever order a batch of its size takes (K / 8 groups), one rounding to bf16
    mag = gl.mx4_dequantize(xt[-3:], xts[-3:]).float().abs() @ gl.mx4_dequantize(w, ws).float().abs().t()
    assert ((out[-3:].float() - few[-3:]).abs() <= 2.0 ** -8 * few[-3:].abs() + 2 * 130 * 2.0 ** -23 * mag).all()
