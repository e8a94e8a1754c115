"""Sizes that the binding of the operators has to refuse before it allocates
outputs of them, on the CPU."""

import pytest
import torch

gl = pytest.importorskip("group_limited_routing_amd")


@pytest.mark.parametrize("top_k", [0, -1, -(1 << 31), 17, 1 << 30, 1 << 40])
def test_gate_top_k(top_k):
    z = torch.zeros(4, 16)
    with pytest.raises(gl.BeamMoeError) as e:
        gl.gate(z, top_k=top_k)
    assert e.value.status == (gl.BEAM_ERR_SHAPE if top_k > 0x7fffffff else gl.BEAM_ERR_CONFIG)


@pytest.mark.parametrize("kw", [dict(n_group=-1), dict(topk_group=-1), dict(n_group=-(1 << 40)),
                                dict(topk_group=-(1 << 33) + 1), dict(n_group=0), dict(topk_group=0)])
def test_gate_groups(kw):
    with pytest.raises(gl.BeamMoeError) as e:
        gl.gate(torch.zeros(4, 16), top_k=2, **kw)
    assert e.value.status == gl.BEAM_ERR_CONFIG


def test_gate_backward_slots():
    """More slots than experts, or none."""
    for k in (0, 17):
        with pytest.raises(gl.BeamMoeError) as e:
            gl.gate_backward(torch.zeros(4, k), torch.zeros(4, 16), torch.zeros(4, k, dtype=torch.int32))
        assert e.value.status == gl.BEAM_ERR_CONFIG
