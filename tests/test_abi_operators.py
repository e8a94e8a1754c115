"""Argument checks of the norm, routing and MXFP4 operators, on the CPU: the C
ABI returns its status before any HIP call (fake pointers stand in for device
memory), and the binding raises before it reaches the library."""

import ctypes
import os

import pytest
import torch

gl = pytest.importorskip("group_limited_routing_amd")

FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gl.LIB_PATH):
        pytest.skip("libbeam_moe.so not built")
    return gl.lib()


def _norm(L, T=8, cfg=(512, gl.BEAM_BF16, 1.0, 1.0, 1e-6, 0), **over):
    p = dict(x=FAKE, si=FAKE, w=FAKE, so=FAKE, y=FAKE, q=None, qs=None)
    p.update(over)
    c = ctypes.byref(gl.BeamMoeNorm(*cfg)) if cfg else None
    return L.beam_moe_add_rms_norm(c, T, p["x"], p["si"], p["w"], p["so"], p["y"], p["q"], p["qs"],
                                   None)


def test_norm_checks(L):
    ok = (512, gl.BEAM_BF16, 1.0, 1.0, 1e-6, 0)
    q = dict(q=FAKE, qs=FAKE)
    assert _norm(L, cfg=None) == gl.BEAM_ERR_NULL
    for i, v, st in [(0, 0, gl.BEAM_ERR_SHAPE), (0, 65537, gl.BEAM_ERR_SHAPE), (1, 2, gl.BEAM_ERR_DTYPE),
                     (2, float("nan"), gl.BEAM_ERR_CONFIG), (3, float("inf"), gl.BEAM_ERR_CONFIG),
                     (4, -1.0, gl.BEAM_ERR_CONFIG), (4, float("nan"), gl.BEAM_ERR_CONFIG),
                     (5, 3, gl.BEAM_ERR_CONFIG), (5, -1, gl.BEAM_ERR_CONFIG)]:
        assert _norm(L, cfg=ok[:i] + (v,) + ok[i + 1:]) == st, (i, v)
    assert _norm(L, T=-1) == gl.BEAM_ERR_SHAPE and _norm(L, T=(1 << 22) + 1) == gl.BEAM_ERR_SHAPE
    # blocks of 32 columns
    assert _norm(L, cfg=(520, gl.BEAM_BF16, 1.0, 1.0, 0.0, 2), **q) == gl.BEAM_ERR_SHAPE
    for name in ("x", "w"):
        assert _norm(L, **{name: None}) == gl.BEAM_ERR_NULL, name
    assert _norm(L, so=None, y=None) == gl.BEAM_ERR_NULL
    for quant in (1, 2):
        for name in ("q", "qs"):
            assert _norm(L, cfg=ok[:5] + (quant,), **dict(q, **{name: None})) == gl.BEAM_ERR_NULL
    for name in ("q", "qs"):  # an 8-bit output that nothing would write
        assert _norm(L, **{name: FAKE}) == gl.BEAM_ERR_CONFIG
    for name in ("x", "si", "w", "so", "y", "q", "qs"):
        assert _norm(L, cfg=ok[:5] + (1,), **dict(q, **{name: FAKE + 8})) == gl.BEAM_ERR_ALIGN, name
    assert _norm(L, T=0, x=None, w=None, y=None) == gl.BEAM_OK


def _norm_bwd(L, T=8, cfg=(512, gl.BEAM_BF16, 1.0, 1.0, 1e-6, 0), ws_bytes=1 << 40, **over):
    p = dict(dy=FAKE, s=FAKE, w=FAKE, dso=FAKE, dx=FAKE, dsi=FAKE, dw=FAKE, ws=FAKE)
    p.update(over)
    c = ctypes.byref(gl.BeamMoeNorm(*cfg)) if cfg else None
    return L.beam_moe_add_rms_norm_backward(c, T, p["dy"], p["s"], p["w"], p["dso"], p["dx"],
                                            p["dsi"], p["dw"], p["ws"], ws_bytes, None)


def test_norm_backward_checks(L):
    assert _norm_bwd(L, cfg=None) == gl.BEAM_ERR_NULL
    assert _norm_bwd(L, cfg=(0, 1, 1.0, 1.0, 0.0, 0)) == gl.BEAM_ERR_SHAPE
    assert _norm_bwd(L, cfg=(64, 3, 1.0, 1.0, 0.0, 0)) == gl.BEAM_ERR_DTYPE
    for name in ("dy", "s", "w", "dx"):
        assert _norm_bwd(L, **{name: None}) == gl.BEAM_ERR_NULL, name
    cfg = gl.BeamMoeNorm(512, gl.BEAM_BF16, 1.0, 1.0, 1e-6, 0)
    need = L.beam_moe_add_rms_norm_backward_workspace_bytes(ctypes.byref(cfg), 8)
    assert need >= 512 * 4
    assert L.beam_moe_add_rms_norm_backward_workspace_bytes(None, 8) == 0
    assert L.beam_moe_add_rms_norm_backward_workspace_bytes(ctypes.byref(cfg), -1) == 0
    assert _norm_bwd(L, ws=None) == gl.BEAM_ERR_WORKSPACE
    assert _norm_bwd(L, ws_bytes=need - 1) == gl.BEAM_ERR_WORKSPACE
    for name in ("dy", "s", "w", "dso", "dx", "dsi", "dw", "ws"):
        assert _norm_bwd(L, **{name: FAKE + 4}) == gl.BEAM_ERR_ALIGN, name
    assert _norm_bwd(L, T=0, dy=None, ws=None) == gl.BEAM_OK


GATE = dict(n_experts=256, n_group=8, topk_group=4, top_k=8, score=0, group_score=0, renormalise=1,
            z_dtype=gl.BEAM_F32, routed_scaling_factor=2.5)


def _gate(L, T=8, cfg=GATE, **over):
    p = dict(z=FAKE, b=FAKE, v=FAKE, idx=FAKE, w=FAKE, cnt=FAKE)
    p.update(over)
    c = ctypes.byref(gl.BeamMoeGateConfig(**cfg)) if cfg else None
    return L.beam_moe_gate(c, T, p["z"], p["b"], p["v"], p["idx"], p["w"], p["cnt"], None)


def _gate_bwd(L, T=8, cfg=GATE, **over):
    p = dict(dw=FAKE, z=FAKE, idx=FAKE, dz=FAKE)
    p.update(over)
    c = ctypes.byref(gl.BeamMoeGateConfig(**cfg)) if cfg else None
    return L.beam_moe_gate_backward(c, T, p["dw"], p["z"], p["idx"], p["dz"], None)


def test_gate_checks(L):
    for call in (_gate, _gate_bwd):
        assert call(L, cfg=None) == gl.BEAM_ERR_NULL
        for kw in (dict(n_experts=0), dict(n_experts=1025), dict(n_group=3), dict(n_group=0),
                   dict(n_group=128), dict(topk_group=0), dict(topk_group=9), dict(top_k=0),
                   dict(top_k=33), dict(topk_group=1, n_group=64, top_k=5), dict(score=2),
                   dict(group_score=2), dict(renormalise=2),
                   dict(routed_scaling_factor=float("nan"))):
            assert call(L, cfg=dict(GATE, **kw)) == gl.BEAM_ERR_CONFIG, kw
        assert call(L, cfg=dict(GATE, z_dtype=2)) == gl.BEAM_ERR_DTYPE
        assert call(L, T=-1) == gl.BEAM_ERR_SHAPE
        assert call(L, T=0, z=None) == gl.BEAM_OK
    for name in ("z", "idx", "w"):
        assert _gate(L, **{name: None}) == gl.BEAM_ERR_NULL, name
    for name in ("z", "b", "v", "idx", "w", "cnt"):
        assert _gate(L, **{name: FAKE + 4}) == gl.BEAM_ERR_ALIGN, name
    for name in ("dw", "z", "idx", "dz"):
        assert _gate_bwd(L, **{name: None}) == gl.BEAM_ERR_NULL, name
        assert _gate_bwd(L, **{name: FAKE + 4}) == gl.BEAM_ERR_ALIGN, name


def test_mx4_row_checks(L):
    for rows, cols, st in [(-1, 64, gl.BEAM_ERR_SHAPE), (4, 0, gl.BEAM_ERR_SHAPE),
                           (4, 48, gl.BEAM_ERR_SHAPE), (1 << 36, 64, gl.BEAM_ERR_SHAPE),
                           (0, 64, gl.BEAM_OK)]:
        assert L.beam_moe_mx4_quantize(FAKE, rows, cols, 1, 0, FAKE, FAKE, None) == st, (rows, cols)
        assert L.beam_moe_mx4_dequantize(FAKE, FAKE, rows, cols, 1, FAKE, None) == st, (rows, cols)
    q = L.beam_moe_mx4_quantize
    assert q(FAKE, 16, 512, 2, 0, FAKE, FAKE, None) == gl.BEAM_ERR_DTYPE
    assert q(FAKE, 16, 512, 1, 2, FAKE, FAKE, None) == gl.BEAM_ERR_CONFIG
    assert q(FAKE, 15, 512, 1, 1, FAKE, FAKE, None) == gl.BEAM_ERR_SHAPE
    assert q(FAKE, 16, 256, 1, 1, FAKE, FAKE, None) == gl.BEAM_ERR_SHAPE
    assert L.beam_moe_mx4_dequantize(FAKE, FAKE, 4, 64, 3, FAKE, None) == gl.BEAM_ERR_DTYPE
    for i in range(3):
        p = [FAKE] * 3
        p[i] = None
        assert q(p[0], 16, 512, 1, 0, p[1], p[2], None) == gl.BEAM_ERR_NULL
        assert L.beam_moe_mx4_dequantize(p[0], p[1], 4, 64, 1, p[2], None) == gl.BEAM_ERR_NULL
        p[i] = FAKE + 8
        assert q(p[0], 16, 512, 1, 0, p[1], p[2], None) == gl.BEAM_ERR_ALIGN
        assert L.beam_moe_mx4_dequantize(p[0], p[1], 4, 64, 1, p[2], None) == gl.BEAM_ERR_ALIGN


def _linear(L, T=8, cfg=(640, 512, 0, gl.BEAM_BF16), **over):
    p = dict(x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, out=FAKE)
    p.update(over)
    c = ctypes.byref(gl.BeamMoeLinear(*cfg)) if cfg else None
    return L.beam_moe_mx4_linear(c, T, p["x"], p["xs"], p["w"], p["ws"], p["out"], None)


def test_linear_checks(L):
    assert _linear(L, cfg=None) == gl.BEAM_ERR_NULL
    for cfg, st in [((0, 512, 0, 1), gl.BEAM_ERR_SHAPE), (((1 << 20) + 1, 512, 0, 1), gl.BEAM_ERR_SHAPE),
                    ((640, 0, 0, 1), gl.BEAM_ERR_SHAPE), ((640, 48, 0, 1), gl.BEAM_ERR_SHAPE),
                    ((640, 65568, 0, 1), gl.BEAM_ERR_SHAPE), ((640, 512, 3, 1), gl.BEAM_ERR_CONFIG),
                    ((640, 512, -1, 1), gl.BEAM_ERR_CONFIG), ((640, 512, 0, 2), gl.BEAM_ERR_DTYPE)]:
        assert _linear(L, cfg=cfg) == st, cfg
    assert _linear(L, T=-1) == gl.BEAM_ERR_SHAPE
    for name in ("x", "xs", "w", "ws", "out"):
        assert _linear(L, **{name: None}) == gl.BEAM_ERR_NULL, name
    for name in ("x", "xs", "w", "ws", "out"):
        assert _linear(L, **{name: FAKE + 8}) == gl.BEAM_ERR_ALIGN, name
    assert _linear(L, T=0, x=None) == gl.BEAM_OK


def test_binding_refuses_bad_tensors():
    """Wrong shapes, types, strides and devices raise before the library is called."""
    bf, f8, u8 = torch.bfloat16, torch.float8_e4m3fn, torch.uint8
    x, w = torch.zeros(4, 64, dtype=bf), torch.zeros(64)
    bad = [
        lambda: gl.add_rms_norm(x.half(), w),
        lambda: gl.add_rms_norm(x, w.to(bf)),
        lambda: gl.add_rms_norm(x, w[:32]),
        lambda: gl.add_rms_norm(x.t(), torch.zeros(4)),
        lambda: gl.add_rms_norm(x, w, stream_in=x.float()),
        lambda: gl.add_rms_norm(x, w, stream_in=x[:3]),
        lambda: gl.add_rms_norm(x, w, stream_in=x, stream_out=x.float()),
        lambda: gl.add_rms_norm(x, w, quant="fp8"),
        lambda: gl.add_rms_norm_backward(x, x.float(), w),
        lambda: gl.add_rms_norm_backward(x, x, w, d_stream_out=x[:, :32]),
        lambda: gl.gate(x.half(), top_k=2),
        lambda: gl.gate(x, top_k=2, score="relu"),
        lambda: gl.gate(x, top_k=2, group_score="sum"),
        lambda: gl.gate(x, top_k=2, expert_bias=w[:8]),
        lambda: gl.gate(x, top_k=2, valid=torch.ones(3, dtype=torch.bool)),
        lambda: gl.gate(x, top_k=2, valid=torch.ones(4)),
        lambda: gl.gate_backward(torch.zeros(4, 2), x, torch.zeros(4, 2, dtype=torch.int64)),
        lambda: gl.gate_backward(torch.zeros(4, 2), x, torch.zeros(4, 3, dtype=torch.int32)),
        lambda: gl.gate_backward(torch.zeros(4, 2, dtype=bf), x, torch.zeros(4, 2, dtype=torch.int32)),
        lambda: gl.mx4_quantize(x.half()),
        lambda: gl.mx4_quantize(x[:, :33].contiguous()),
        lambda: gl.mx4_quantize(x, packed=True),
        lambda: gl.mx4_quantize(torch.zeros(2, 8, 512), packed=True),
        lambda: gl.mx4_dequantize(torch.zeros(4, 32, dtype=u8), torch.zeros(4, 3, dtype=u8)),
        lambda: gl.mx4_dequantize(torch.zeros(4, 32, dtype=u8), torch.zeros(4, 2, dtype=u8),
                                  dtype=torch.float16),
    ]
    xq, xs, xb = torch.zeros(4, 64).to(f8), torch.zeros(4), torch.zeros(4, 2, dtype=u8)
    wq, ws = torch.zeros(8, 32, dtype=u8), torch.zeros(8, 2, dtype=u8)
    bad += [
        lambda: gl.mx4_linear(x, xs, wq, ws),
        lambda: gl.mx4_linear(xq, xs, wq, ws[:4]),
        lambda: gl.mx4_linear(xq, xs[:3], wq, ws),
        lambda: gl.mx4_linear(xq, xb[:, :1], wq, ws),
        lambda: gl.mx4_linear(xb, xs, wq, ws),
        lambda: gl.mx4_linear(xq[:, :32], xs, wq, ws),
        lambda: gl.mx4_linear(xq, xs, wq, ws, out=torch.zeros(4, 9, dtype=bf)),
        lambda: gl.mx4_linear(xq, xs, wq, ws, out_dtype=torch.float16),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was not refused")
    # what is right but for its device
    for f in (lambda: gl.add_rms_norm(x, w), lambda: gl.add_rms_norm_backward(x, x, w),
              lambda: gl.gate(x, top_k=2), lambda: gl.mx4_quantize(x),
              lambda: gl.mx4_linear(xq, xs, wq, ws)):
        with pytest.raises(ValueError, match="expected a GPU"):
            f()


def test_binding_refuses_sizes_past_32_bits():
    """Sizes that would wrap in the library's 32-bit arguments are refused."""
    big, bf, u8 = (1 << 32) + 4, torch.bfloat16, torch.uint8
    rows, w = torch.empty(big, 0, dtype=bf), torch.empty(0)
    for f in (lambda: gl.add_rms_norm(rows, w), lambda: gl.add_rms_norm_backward(rows, rows, w),
              lambda: gl.gate(rows, top_k=1),
              lambda: gl.gate(torch.zeros(4, 8), top_k=big),
              lambda: gl.gate(torch.zeros(4, 8), top_k=1, n_group=big),
              lambda: gl.gate_backward(torch.empty(big, 0), rows, torch.empty(big, 0, dtype=torch.int32)),
              lambda: gl.mx4_linear(torch.empty(big, 0, dtype=u8), torch.empty(big, 0, dtype=u8),
                                    torch.empty(4, 0, dtype=u8), torch.empty(4, 0, dtype=u8))):
        with pytest.raises(gl.BeamMoeError) as e:
            f()
        assert e.value.status == gl.BEAM_ERR_SHAPE
