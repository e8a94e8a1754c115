"""Every tile of the gated product and its gradient, whole, cut along the reduction and
both (a test of each combination that the cost rule can choose, at small sizes that make
it), and both products of the gradient in one launch for every pair of tiles; the
borders of the kernel for few tokens. Against fp64 on the GPU, with the bounds of
test_gpu_gated.py."""

import pytest
import torch

import group_limited_routing_amd as gl
from test_gpu_gated import _near, _rand

pytestmark = pytest.mark.gpu

FORWARD = [(2552, 488, 3272), (6369, 3944, 336), (8231, 128, 464), (7293, 1248, 552), (67, 3984, 5592),
           (196, 128, 8440), (11130, 1768, 152), (17, 720, 128), (17, 128, 128), (16, 512, 5120), (16, 512, 5128),
           (8, 264, 10240), (9, 264, 10240), (1, 5120, 2568)]
BACKWARD = [(9367, 1688, 216), (10893, 144, 2552), (9434, 784, 128), (7293, 1048, 600), (5569, 152, 1896),
            (11028, 264, 128), (10961, 272, 728), (1, 128, 328), (6698, 136, 6152), (340, 3760, 1864), (1, 392, 8344),
            (494, 1256, 6552), (5620, 136, 5416), (1415, 696, 5384), (655, 136, 128), (1, 128, 128)]


@pytest.mark.parametrize("T,H,F", FORWARD)
def test_forward(T, H, F):
    x, wg, wu = _rand((T, H), 1), _rand((F, H), 2, H ** -0.5), _rand((F, H), 3, H ** -0.5)
    ag, au = _rand((T, F), 4), _rand((T, F), 5)
    g = x.double() @ wg.double().t().contiguous() + ag.double()
    u = x.double() @ wu.double().t().contiguous() + au.double()
    r = gl.gated_linear(x, wg, wu, activation="gelu", add_gate=ag, add_up=au, return_pre=True)
    phi = 0.5 * torch.special.erfc(-g / 2 ** 0.5)
    for name, want in (("gate", g), ("up", u), ("h", g * phi * u)):
        _near(r[name], want, H + 1, name)
    again = gl.gated_linear(x, wg, wu, activation="gelu", add_gate=ag, add_up=au)
    assert torch.equal(again["h"], r["h"])


@pytest.mark.parametrize("T,H,F", BACKWARD)
def test_backward(T, H, F):
    x, wg, wu = _rand((T, H), 1), _rand((F, H), 2, H ** -0.5), _rand((F, H), 3, H ** -0.5)
    dh, gate, up = _rand((T, F), 6), _rand((T, F), 7), _rand((T, F), 8)
    r = gl.gated_linear_backward(dh, x, wg, wu, gate, up)
    dg, du, xd = r["d_gate"].double(), r["d_up"].double(), x.double()
    for name, want, K in (("dx", dg @ wg.double() + du @ wu.double(), 2 * F),
                          ("d_w_gate", dg.t().contiguous() @ xd, T), ("d_w_up", du.t().contiguous() @ xd, T)):
        _near(r[name], want, K, name)
    # one product at a time: the same sums
    part = gl.gated_linear_backward(dh, x, wg, wu, gate, up, weight_grad=False)
    assert torch.equal(part["dx"], r["dx"])
    part = gl.gated_linear_backward(dh, x, wg, wu, gate, up, input_grad=False)
    assert torch.equal(part["d_w_gate"], r["d_w_gate"]) and torch.equal(part["d_w_up"], r["d_w_up"])
