"""Argument checks of the gated product, the adapters and dropout, on the CPU: the C
ABI returns its status before any HIP call (fake pointers stand in for device
memory), and the binding raises before it reaches the library."""

import ctypes
import os

import pytest
import torch

gl = pytest.importorskip("group_limited_routing_amd")

FAKE = 0x7F0000000000  # 16-byte aligned, never dereferenced
HUGE = 1 << 50


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gl.LIB_PATH):
        pytest.skip("libbeam_moe.so not built")
    return gl.lib()


GATED = dict(hidden=512, intermediate=264, activation=0, dtype=gl.BEAM_BF16)


def _gated(L, T=8, cfg=GATED, ws_bytes=HUGE, **over):
    p = dict(x=FAKE, wg=FAKE, wu=FAKE, ag=FAKE, au=FAKE, h=FAKE, g=FAKE, u=FAKE, ws=FAKE)
    p.update(over)
    c = ctypes.byref(gl.BeamMoeGated(**cfg)) if cfg else None
    return L.beam_moe_gated_linear(c, T, *p.values(), ws_bytes, None)


def _gated_bwd(L, T=8, cfg=GATED, ws_bytes=HUGE, **over):
    p = dict(dh=FAKE, x=FAKE, wg=FAKE, wu=FAKE, g=FAKE, u=FAKE, dg=FAKE, du=FAKE, dx=FAKE, dwg=FAKE,
             dwu=FAKE, ws=FAKE)
    p.update(over)
    c = ctypes.byref(gl.BeamMoeGated(**cfg)) if cfg else None
    return L.beam_moe_gated_linear_backward(c, T, *p.values(), ws_bytes, None)


def test_gated_checks(L):
    for call in (_gated, _gated_bwd):
        assert call(L, cfg=None) == gl.BEAM_ERR_NULL
        for kw, st in [(dict(hidden=0), gl.BEAM_ERR_SHAPE), (dict(hidden=12), gl.BEAM_ERR_SHAPE),
                       (dict(hidden=65544), gl.BEAM_ERR_SHAPE), (dict(intermediate=4), gl.BEAM_ERR_SHAPE),
                       (dict(intermediate=-8), gl.BEAM_ERR_SHAPE), (dict(intermediate=262152), gl.BEAM_ERR_SHAPE),
                       (dict(activation=2), gl.BEAM_ERR_CONFIG), (dict(activation=-1), gl.BEAM_ERR_CONFIG),
                       (dict(dtype=gl.BEAM_F32), gl.BEAM_ERR_DTYPE), (dict(dtype=9), gl.BEAM_ERR_DTYPE)]:
            assert call(L, cfg=dict(GATED, **kw)) == st, kw
        assert call(L, T=-1) == gl.BEAM_ERR_SHAPE and call(L, T=(1 << 22) + 1) == gl.BEAM_ERR_SHAPE
        assert call(L, T=0, x=None) == gl.BEAM_OK
    for name in ("x", "wg", "wu", "h"):
        assert _gated(L, **{name: None}) == gl.BEAM_ERR_NULL, name
    for name in ("x", "wg", "wu", "ag", "au", "h", "g", "u", "ws"):
        assert _gated(L, **{name: FAKE + 8}) == gl.BEAM_ERR_ALIGN, name
    for name in ("dh", "g", "u", "dg", "du", "wg", "wu", "x", "dwg", "dwu"):
        assert _gated_bwd(L, **{name: None}) == gl.BEAM_ERR_NULL, name
    for name in ("dh", "x", "wg", "wu", "g", "u", "dg", "du", "dx", "dwg", "dwu", "ws"):
        assert _gated_bwd(L, **{name: FAKE + 8}) == gl.BEAM_ERR_ALIGN, name
    c = gl.BeamMoeGated(**dict(GATED, hidden=4096))
    for call, size in ((_gated, L.beam_moe_gated_linear_workspace_bytes),
                       (_gated_bwd, L.beam_moe_gated_linear_backward_workspace_bytes)):
        assert size(None, 8) == 0 and size(ctypes.byref(c), -1) == 0 and size(ctypes.byref(c), 0) == 0
        seen = 0
        for T in (1, 8, 100, 4096):
            need = size(ctypes.byref(c), T)
            if need:
                seen += 1
                assert call(L, T=T, cfg=dict(GATED, hidden=4096), ws=None) == gl.BEAM_ERR_WORKSPACE
                assert call(L, T=T, cfg=dict(GATED, hidden=4096), ws_bytes=need - 1) == gl.BEAM_ERR_WORKSPACE
        assert seen


LORA = dict(k=512, n=264, rank=16, n_adapters=5, dtype=gl.BEAM_BF16)


def _lora(L, T=8, cfg=LORA, ws_bytes=HUGE, **over):
    p = dict(x=FAKE, a=FAKE, b=FAKE, s=FAKE, plan=FAKE, base=FAKE, out=FAKE, v=FAKE, ws=FAKE)
    p.update(over)
    c = ctypes.byref(gl.BeamMoeLoraConfig(**cfg)) if cfg else None
    return L.beam_moe_lora(c, T, *p.values(), ws_bytes, None)


def _lora_bwd(L, T=8, cfg=LORA, ws_bytes=HUGE, **over):
    p = dict(dy=FAKE, x=FAKE, v=FAKE, a=FAKE, b=FAKE, s=FAKE, plan=FAKE, base=FAKE, dx=FAKE, da=FAKE,
             db=FAKE, ws=FAKE)
    p.update(over)
    c = ctypes.byref(gl.BeamMoeLoraConfig(**cfg)) if cfg else None
    return L.beam_moe_lora_backward(c, T, *p.values(), ws_bytes, None)


def test_lora_checks(L):
    for call in (_lora, _lora_bwd):
        assert call(L, cfg=None) == gl.BEAM_ERR_NULL
        for kw, st in [(dict(k=0), gl.BEAM_ERR_SHAPE), (dict(k=20), gl.BEAM_ERR_SHAPE),
                       (dict(k=65544), gl.BEAM_ERR_SHAPE), (dict(n=4), gl.BEAM_ERR_SHAPE),
                       (dict(n=262152), gl.BEAM_ERR_SHAPE), (dict(rank=0), gl.BEAM_ERR_CONFIG),
                       (dict(rank=12), gl.BEAM_ERR_CONFIG), (dict(rank=136), gl.BEAM_ERR_CONFIG),
                       (dict(n_adapters=0), gl.BEAM_ERR_CONFIG), (dict(n_adapters=1025), gl.BEAM_ERR_CONFIG),
                       (dict(dtype=gl.BEAM_F32), gl.BEAM_ERR_DTYPE)]:
            assert call(L, cfg=dict(LORA, **kw)) == st, kw
        assert call(L, T=-1) == gl.BEAM_ERR_SHAPE and call(L, T=(1 << 22) + 1) == gl.BEAM_ERR_SHAPE
        assert call(L, T=0, a=None) == gl.BEAM_OK
        assert call(L, ws=None) == gl.BEAM_ERR_WORKSPACE
    c = ctypes.byref(gl.BeamMoeLoraConfig(**LORA))
    for call, size in ((_lora, L.beam_moe_lora_workspace_bytes),
                       (_lora_bwd, L.beam_moe_lora_backward_workspace_bytes)):
        assert size(c, 8) >= 8 * 16 * 4 and size(None, 8) == 0 and size(c, -1) == 0
        assert call(L, ws_bytes=size(c, 8) - 1) == gl.BEAM_ERR_WORKSPACE
    for name in ("x", "a", "b", "plan", "out"):
        assert _lora(L, **{name: None}) == gl.BEAM_ERR_NULL, name
    for name in ("x", "a", "b", "s", "plan", "base", "out", "v", "ws"):
        assert _lora(L, **{name: FAKE + 4}) == gl.BEAM_ERR_ALIGN, name
    for name in ("dy", "x", "v", "a", "b", "plan", "da", "db"):
        assert _lora_bwd(L, **{name: None}) == gl.BEAM_ERR_NULL, name
    assert _lora_bwd(L, dx=None, da=None, db=None) == gl.BEAM_ERR_NULL
    for name in ("dy", "x", "v", "a", "b", "s", "plan", "base", "dx", "da", "db", "ws"):
        assert _lora_bwd(L, **{name: FAKE + 4}) == gl.BEAM_ERR_ALIGN, name


def test_lora_plan_checks(L):
    size, plan = L.beam_moe_lora_plan_bytes, L.beam_moe_lora_plan
    for T, E, st in [(8, 0, gl.BEAM_ERR_CONFIG), (8, 1025, gl.BEAM_ERR_CONFIG), (-1, 4, gl.BEAM_ERR_SHAPE),
                     ((1 << 22) + 1, 4, gl.BEAM_ERR_SHAPE)]:
        assert size(T, E) == 0 and plan(FAKE, T, E, FAKE, HUGE, None) == st
    assert plan(None, 0, 4, None, 0, None) == gl.BEAM_OK
    assert plan(None, 8, 4, FAKE, HUGE, None) == gl.BEAM_ERR_NULL
    assert plan(FAKE, 8, 4, None, HUGE, None) == gl.BEAM_ERR_NULL
    assert plan(FAKE, 8, 4, FAKE, size(8, 4) - 1, None) == gl.BEAM_ERR_WORKSPACE
    assert plan(FAKE + 4, 8, 4, FAKE, HUGE, None) == gl.BEAM_ERR_ALIGN
    assert plan(FAKE, 8, 4, FAKE + 4, HUGE, None) == gl.BEAM_ERR_ALIGN


def _drop(L, n=64, cfg=(0.1, 1.0, 1.0, gl.BEAM_BF16), **over):
    p = dict(x=FAKE, st=FAKE, off=FAKE, out=FAKE)
    p.update(over)
    c = ctypes.byref(gl.BeamMoeDropoutConfig(*cfg)) if cfg else None
    return L.beam_moe_dropout(c, n, p["x"], p["st"], 1, 2, p["off"], p["out"], None)


def _drop_bwd(L, n=64, cfg=(0.1, 1.0, 1.0, gl.BEAM_BF16), **over):
    p = dict(x=FAKE, off=FAKE, out=FAKE, dst=FAKE)
    p.update(over)
    c = ctypes.byref(gl.BeamMoeDropoutConfig(*cfg)) if cfg else None
    return L.beam_moe_dropout_backward(c, n, p["x"], 1, 2, p["off"], p["out"], p["dst"], None)


def test_dropout_checks(L):
    ok, nan = (0.1, 1.0, 1.0, gl.BEAM_BF16), float("nan")
    for call in (_drop, _drop_bwd):
        assert call(L, cfg=None) == gl.BEAM_ERR_NULL
        for i, v, st in [(0, -0.1, gl.BEAM_ERR_CONFIG), (0, 1.01, gl.BEAM_ERR_CONFIG), (0, nan, gl.BEAM_ERR_CONFIG),
                         (1, nan, gl.BEAM_ERR_CONFIG), (2, float("inf"), gl.BEAM_ERR_CONFIG),
                         (3, gl.BEAM_FP8_E4M3, gl.BEAM_ERR_DTYPE)]:
            assert call(L, cfg=ok[:i] + (v,) + ok[i + 1:]) == st, (i, v)
        assert call(L, n=-1) == gl.BEAM_ERR_SHAPE and call(L, n=(1 << 40) + 1) == gl.BEAM_ERR_SHAPE
        assert call(L, n=0, x=None) == gl.BEAM_OK
        for name in ("x", "out"):
            assert call(L, **{name: None}) == gl.BEAM_ERR_NULL, name
            assert call(L, **{name: FAKE + 4}) == gl.BEAM_ERR_ALIGN, name
        assert call(L, off=FAKE + 4) == gl.BEAM_ERR_ALIGN
    assert _drop(L, st=FAKE + 2) == gl.BEAM_ERR_ALIGN and _drop_bwd(L, dst=FAKE + 2) == gl.BEAM_ERR_ALIGN


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _plan(T=4, E=2):
    return gl.LoraPlan(torch.zeros(4096, dtype=torch.uint8), T, E)


def test_binding_refuses_before_the_library():
    x, wg = _bf(4, 16), _bf(24, 16)
    with pytest.raises(ValueError, match="expected a GPU"):
        gl.gated_linear(x, wg, wg)
    with pytest.raises(ValueError, match="w_up has shape"):
        gl.gated_linear(x, wg, _bf(16, 16))
    with pytest.raises(ValueError, match="x has dtype"):
        gl.gated_linear(x.float(), wg, wg)
    with pytest.raises(ValueError, match="contiguous"):
        gl.gated_linear(_bf(16, 4).t(), wg, wg)
    with pytest.raises(ValueError, match="activation is"):
        gl.gated_linear(x, wg, wg, activation="tanh")
    with pytest.raises(ValueError, match="add_up has shape"):
        gl.gated_linear(x, wg, wg, add_up=_bf(4, 16))
    with pytest.raises(ValueError, match="gate has shape"):
        gl.gated_linear_backward(_bf(4, 24), x, wg, wg, _bf(3, 24), _bf(4, 24))
    for H, F in ((12, 24), (16, 20)):
        with pytest.raises(gl.BeamMoeError) as e:
            gl.gated_linear(_bf(4, H), _bf(F, H), _bf(F, H))
        assert e.value.status == gl.BEAM_ERR_SHAPE
    a, b = _bf(2, 8, 16), _bf(2, 24, 8)
    with pytest.raises(ValueError, match="expected a GPU"):
        gl.lora(x, a, b, _plan())
    with pytest.raises(ValueError, match="plan is for"):
        gl.lora(x, a, b, _plan(E=3))
    with pytest.raises(ValueError, match="plan is for"):
        gl.lora(x, a, b, _plan(T=5))
    with pytest.raises(ValueError, match="b has shape"):
        gl.lora(x, a, _bf(3, 24, 8), _plan())
    with pytest.raises(ValueError, match="scale has"):
        gl.lora(x, a, b, _plan(), scale=torch.ones(2, dtype=torch.float64))
    with pytest.raises(ValueError, match="base has shape"):
        gl.lora(x, a, b, _plan(), base=_bf(4, 16))
    with pytest.raises(ValueError, match="v has dtype"):
        gl.lora_backward(_bf(4, 24), x, _bf(4, 8), a, b, _plan())
    for aa, bb in ((_bf(2, 12, 16), _bf(2, 24, 12)), (_bf(2, 136, 16), _bf(2, 24, 136))):
        with pytest.raises(gl.BeamMoeError) as e:
            gl.lora(x, aa, bb, _plan())
        assert e.value.status == gl.BEAM_ERR_CONFIG
    with pytest.raises(gl.BeamMoeError) as e:
        gl.lora(x, a, _bf(2, 20, 8), _plan())
    assert e.value.status == gl.BEAM_ERR_SHAPE
    for n in (0, -1):
        with pytest.raises(gl.BeamMoeError) as e:
            gl.lora_plan(torch.zeros(4, dtype=torch.int32), n)
        assert e.value.status == gl.BEAM_ERR_CONFIG
    with pytest.raises(ValueError, match="index has dtype"):
        gl.lora_plan(torch.zeros(4, dtype=torch.int64), 2)
    with pytest.raises(ValueError, match="expected a GPU"):
        gl.dropout(x, 0.1, seed=1)
    for kw in (dict(seed=-1), dict(seed=1 << 64), dict(seed=0, offset=-1), dict(seed=0, offset=1 << 64)):
        with pytest.raises(ValueError, match="64 bits"):
            gl.dropout(x, 0.1, **kw)
    with pytest.raises(ValueError, match="offset has dtype"):
        gl.dropout(x, 0.1, seed=0, offset=torch.zeros(1))
    with pytest.raises(ValueError, match="offset has 2 elements"):
        gl.dropout(x, 0.1, seed=0, offset=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="stream_in has dtype"):
        gl.dropout(x, 0.1, seed=0, stream_in=x.float())
