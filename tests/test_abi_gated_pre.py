"""gate and up in fp32: argument checks of the C ABI and of the binding, on the CPU
(fake pointers, as in test_abi_mlp.py)."""

import pytest
import torch

from test_abi_mlp import FAKE, GATED, L, _bf, _gated, _gated_bwd, gl  # noqa: F401

F32 = dict(GATED, pre_f32=1)


def test_pre_f32_is_a_truth_value(L):  # noqa: F811
    for v in (-1, 2):
        assert _gated(L, cfg=dict(GATED, pre_f32=v)) == gl.BEAM_ERR_CONFIG
        assert _gated_bwd(L, cfg=dict(GATED, pre_f32=v)) == gl.BEAM_ERR_CONFIG


def test_fp32_rows_do_not_share_memory_with_bf16_ones(L):  # noqa: F811
    own = dict(g=FAKE + 0x1000000, u=FAKE + 0x2000000)
    for name in ("g", "u"):  # the other arguments stand at FAKE
        assert _gated(L, cfg=F32, **dict(own, **{name: FAKE})) == gl.BEAM_ERR_CONFIG
        assert _gated_bwd(L, cfg=F32, **dict(own, **{name: FAKE})) == gl.BEAM_ERR_CONFIG
        assert _gated(L, cfg=F32, **dict(own, **{name: FAKE + 8})) == gl.BEAM_ERR_ALIGN


def test_binding_takes_a_pair_of_one_type():
    x, w, f = _bf(4, 16), _bf(24, 16), _bf(4, 24)
    with pytest.raises(ValueError, match="gate and up have dtype"):
        gl.gated_linear(x, w, w, return_pre=True, pre_dtype=torch.float16)
    with pytest.raises(ValueError, match="gate and up have dtype"):
        gl.gated_linear_backward(f, x, w, w, f.double(), f.double())
    with pytest.raises(ValueError, match="up has dtype"):
        gl.gated_linear_backward(f, x, w, w, f.float(), f)
    with pytest.raises(ValueError, match="dh has dtype"):
        gl.gated_linear_backward(f.float(), x, w, w, f.float(), f.float())
    with pytest.raises(ValueError, match="expected a GPU"):
        gl.gated_linear(x, w, w, return_pre=True, pre_dtype=torch.float32)
    with pytest.raises(ValueError, match="expected a GPU"):
        gl.gated_linear_backward(f, x, w, w, f.float(), f.float())
