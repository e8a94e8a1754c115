"""Gradients with frozen weights or adapters: the input's gradient without x (or v),
which only the weights' gradients read."""

import pytest
import torch

gl = pytest.importorskip("group_limited_routing_amd")


def _bf(*shape, seed=1, dev="cpu"):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).to(dev)


def test_binding_asks_for_x_where_it_is_read():
    w, f = _bf(24, 16), _bf(4, 24)
    a, b, plan = _bf(2, 8, 16), _bf(2, 24, 8), gl.LoraPlan(torch.zeros(4096, dtype=torch.uint8), 4, 2)
    v = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="x is None"):
        gl.gated_linear_backward(f, None, w, w, f, f)
    with pytest.raises(ValueError, match="x is None"):
        gl.lora_backward(f, None, v, a, b, plan)
    # without the weights' gradients the next check is the device's
    with pytest.raises(ValueError, match="expected a GPU"):
        gl.gated_linear_backward(f, None, w, w, f, f, weight_grad=False)
    with pytest.raises(ValueError, match="expected a GPU"):
        gl.lora_backward(f, None, None, a, b, plan, weight_grad=False)
    # and the other rows are held against dh, dy and the weights
    with pytest.raises(ValueError, match="up has shape"):
        gl.gated_linear_backward(f, None, w, w, f, _bf(3, 24), weight_grad=False)
    with pytest.raises(ValueError, match="x has shape"):
        gl.gated_linear_backward(f, _bf(4, 24), w, w, f, f)
    with pytest.raises(ValueError, match="dy has shape"):
        gl.lora_backward(_bf(4, 16), None, None, a, b, plan, weight_grad=False)
    with pytest.raises(ValueError, match="plan is for"):
        gl.lora_backward(_bf(5, 24), None, None, a, b, plan, weight_grad=False)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [0, 1, 70, 300])
def test_gradients_without_x(T):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dev, H, F, R, E = torch.device("cuda:0"), 264, 136, 16, 3
    x, wg, wu = _bf(T, H, dev=dev), _bf(F, H, seed=2, dev=dev), _bf(F, H, seed=3, dev=dev)
    dh, gate, up = (_bf(T, F, seed=s, dev=dev) for s in (4, 5, 6))
    want = gl.gated_linear_backward(dh, x, wg, wu, gate, up)
    got = gl.gated_linear_backward(dh, None, wg, wu, gate, up, weight_grad=False)
    assert got["d_w_gate"] is None and all(torch.equal(got[k], want[k]) for k in ("dx", "d_gate", "d_up"))
    a, b = _bf(E, R, H, seed=7, dev=dev), _bf(E, F, R, seed=8, dev=dev)
    index = (torch.arange(T, device=dev) % (E + 1)).to(torch.int32)
    plan = gl.lora_plan(index, E)
    v = gl.lora(x, a, b, plan, return_v=True)["v"]
    want = gl.lora_backward(dh, x, v, a, b, plan, base=x)
    got = gl.lora_backward(dh, None, None, a, b, plan, base=x, weight_grad=False)
    assert got["d_a"] is None and torch.equal(got["dx"], want["dx"])
