"""Routing of given logits and its gradient where values run out of fp32's
range, stand in masked places or tie, against oracle.gate in float64. The
tolerances are those of test_gpu_gate.py, whose checks are used."""

import numpy as np
import pytest
import torch

import group_limited_routing_amd as gl
from test_gpu_gate import DT, _check, _dev, _grad_check, _logits, _vec

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("k", [1, 2, 8])
def test_gradient_of_far_negative_sigmoids(k, renorm, dtype):
    """Scores that fp32 holds as subnormals or not at all still share their sum.
    Differences of a row's chosen logits are at most 6, so that an exponential's
    rounded argument is 6 u off, below the 40 u that the tolerance has for it."""
    level = torch.tensor([-80.0, -87.0, -88.0, -90.0, -100.0, -104.0, -120.0, -200.0, -600.0])
    g = torch.Generator().manual_seed(61)
    z = (level[:, None] - 5 * torch.rand((9, 40), generator=g)).to(DT[dtype]).to(_dev())
    z[:, 30:] -= 1000.0
    r = gl.gate(z, top_k=k, renormalise=renorm, routed_scaling_factor=2.5)
    if renorm:
        assert torch.allclose(r["topk_w"].sum(1), torch.full((9,), 2.5, device=_dev()), rtol=1e-6)
    got = _grad_check(_vec(9 * k, 62, 1.0).view(9, k), z, r["topk_idx"], "sigmoid", renorm, 2.5)
    if renorm and k > 1:
        assert (got.abs().amax(1) > 1e-4).all()


def test_gradient_of_mixed_sigmoids():
    """One slot far above the others, positive and negative logits in one row."""
    z = torch.tensor([[40.0, -40.0, 0.0, -100.0], [-90.0, -91.0, -120.0, -300.0],
                      [100.0, 90.0, -100.0, 3.0], [-INF, -95.0, -95.0, -INF],
                      [INF, 2.0, -3.0, -200.0]], device=_dev())
    idx = torch.arange(4, dtype=torch.int32, device=_dev()).repeat(5, 1)
    _grad_check(_vec(20, 63, 1.0).view(5, 4), z, idx, "sigmoid", True, 2.5)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("junk", [float("nan"), INF, -INF])
def test_gradient_passes_over_masked_slots(kind, renorm, junk):
    """What arrives at a slot of a masked expert does not reach the others."""
    z = _logits(6, 24, 64)
    z[:, 5], z[:, 11] = -INF, float("nan")
    idx = torch.tensor([[5, 1, 2], [3, 11, 4], [5, 11, 7], [0, 1, 5], [5, 11, -1], [11, 23, 24]],
                       dtype=torch.int32, device=_dev())
    dw = _vec(18, 65, 1.0).view(6, 3)
    masked = (idx == 5) | (idx == 11) | (idx < 0) | (idx > 23)
    clean = _grad_check(torch.where(masked, torch.zeros_like(dw), dw), z, idx, kind, renorm, 1.5)
    got = gl.gate_backward(torch.where(masked, torch.full_like(dw, junk), dw), z, idx, score=kind,
                           renormalise=renorm, routed_scaling_factor=1.5)
    assert torch.equal(got, clean) and (got[4] == 0).all()


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinite_bias_in_a_masked_group(kind, dtype):
    """A group whose two best keys are +inf and -inf has no score: it comes last,
    in batches of any size."""
    z = _logits(10, 96, 66, dtype)
    bias = _vec(96, 67, 0.1)
    bias[13] = INF
    z[::2, 12:24] = -INF
    z[::2, 13] = 0.5
    for keep in (1, 2, 5):
        with np.errstate(invalid="ignore"):
            _check(z, 6, bias, None, kind, 8, keep, "top2")
            _check(z, 6, bias, None, kind, 8, keep, "max")
    bias[40] = INF
    with np.errstate(invalid="ignore"):
        _check(z, 6, bias, None, kind, 8, 2, "top2")


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E,G,keep", [(64, 1, 1), (256, 8, 3), (500, 4, 2)])
def test_ties_of_tiny_logits(E, G, keep, kind, dtype):
    """Logits so small that their fp64 scores are equal, in twos and threes, and
    zeros of either sign: the lower index comes first, wherever top_k cuts them."""
    rows = []
    for values in ([1e-30, 1e-30, 0.0], [1e-30, 0.0, 0.0], [0.0, -0.0, 0.0], [-0.0, 0.0, 1e-20],
                   [2e-25, 2e-25, 1e-25], [-1e-30, -1e-30, -2e-30], [0.0, -1e-30, -0.0]):
        for at in ([5, 7, 3], [9, 5, 7], [3, 5, 7], [40, 20, 60], [60, 40, 20]):
            for ahead in (0, 2):
                row = torch.full((E,), -2.0)
                row[at] = torch.tensor(values)
                row[50:50 + ahead] = 1.0
                rows.append(row)
    rows.append(torch.zeros(E))
    rows.append(-torch.zeros(E))
    z = torch.stack(rows).to(DT[dtype]).to(_dev())
    for k in (1, 2, 3, 4, 5):
        _check(z, k, None, None, kind, G, keep, "max")
        _check(z, k, None, None, kind, G, keep, "top2")
