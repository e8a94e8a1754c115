"""GPU parity of dropout, against oracle.mlp: the mask has to be equal, the values are
a few fp32 roundings (x by the factor, by add, the stream by keep, the sum: each at
most 2^-24 of the magnitudes) and one to the type (fp32 2^-24, bf16 2^-8) off."""

import numpy as np
import pytest
import torch

import group_limited_routing_amd as gl
import oracle
from parity import Guarded

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24


def _dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


def _rand(shape, seed, dtype):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).to(_dev())


def _f(t):
    return t.cpu().double().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (3, 5), (2, 3, 11), (33, 67), (64, 512)])
@pytest.mark.parametrize("p,seed,offset", [(0.1, 0, 0), (0.5, (1 << 64) - 1, 3), (0.75, 1 << 33, (1 << 64) - 1)])
def test_dropout(shape, p, seed, offset, dtype):
    x, st = _rand(shape, 1, dtype), _rand(shape, 2, dtype)
    f = oracle.mlp.dropout_factor(x.numel(), p, seed, offset).reshape(shape)
    keep, add = (float(np.float32(v)) for v in (0.8, 0.6))
    for stream in (None, st):
        out = gl.dropout(x, p, seed=seed, offset=offset, stream_in=stream, keep=keep, add=add)
        assert out.dtype == x.dtype and out.shape == x.shape
        part = add * f * _f(x)
        ref = part if stream is None else part + keep * _f(st)
        mag = np.abs(part) + (0.0 if stream is None else np.abs(keep * _f(st)))
        assert (np.abs(_f(out) - ref) <= HALF[dtype] * np.abs(ref) + 5 * U * mag).all()
        if stream is None:
            assert np.array_equal(_f(out) == 0, (f == 0) | (_f(x) == 0))
    b = gl.dropout_backward(x, p, seed=seed, offset=offset, keep=keep, add=add, stream_grad=True)
    assert torch.equal(b["dx"], gl.dropout(x, p, seed=seed, offset=offset, add=add))
    assert (np.abs(_f(b["d_stream_in"]) - keep * _f(x)) <= (HALF[dtype] + U) * np.abs(keep * _f(x))).all()
    # the gradient against the difference quotient of the (linear) forward
    d = _f(gl.dropout(torch.ones_like(x), p, seed=seed, offset=offset, add=add))
    assert (np.abs(_f(b["dx"]) - d * _f(x)) <= (2 * HALF[dtype] + 4 * U) * np.abs(d * _f(x))).all()


def test_default_gradient():
    x = _rand((5, 9), 1, "bf16")
    b = gl.dropout_backward(x, 0.3, seed=4)
    assert b["d_stream_in"] is None and torch.equal(b["dx"], gl.dropout(x, 0.3, seed=4))
    assert gl.dropout_backward(x, 0.3, seed=4, stream_grad=True)["d_stream_in"] is x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ends_of_p(dtype):
    x, st = _rand((13, 21), 1, dtype), _rand((13, 21), 2, dtype)
    assert torch.equal(gl.dropout(x, 0.0, seed=1), x) and not gl.dropout(x, 1.0, seed=1).any()
    assert torch.equal(gl.dropout(x, 1.0, seed=1, stream_in=st), st)
    assert torch.equal(gl.dropout(x, 2.0 ** -18, seed=1), x)  # rounds to 0 of 65536
    f = oracle.mlp.dropout_factor(x.numel(), 65535 / 65536, 1).reshape(x.shape)
    assert np.array_equal(_f(gl.dropout(torch.ones_like(x), 65535 / 65536, seed=1)), f)


def test_dropped_values_reach_nothing():
    """Infinities and NaN in dropped places."""
    n = 4096
    f = oracle.mlp.dropout_factor(n, 0.5, 9)
    x, st = _rand((n,), 1, "f32"), _rand((n,), 2, "f32")
    bad = x.clone()
    bad[torch.from_numpy(f == 0).to(_dev())] = float("nan")
    bad[int(np.flatnonzero(f == 0)[0])] = float("inf")
    for kw in (dict(), dict(stream_in=st)):
        assert torch.equal(gl.dropout(bad, 0.5, seed=9, **kw), gl.dropout(x, 0.5, seed=9, **kw))
    bad = x.clone()
    bad[int(np.flatnonzero(f)[0])] = float("nan")
    assert torch.isnan(gl.dropout(bad, 0.5, seed=9)).sum() == 1


def test_offset_on_the_device_and_other_masks():
    x = torch.ones((200, 64), device=_dev())
    at = torch.tensor(7, device=_dev())
    a = gl.dropout(x, 0.4, seed=3, offset=at)
    assert torch.equal(a, gl.dropout(x, 0.4, seed=3, offset=7))
    at += 1
    b = gl.dropout(x, 0.4, seed=3, offset=at)
    assert torch.equal(b, gl.dropout(x, 0.4, seed=3, offset=8))
    # other offsets and seeds: independent masks, five standard deviations
    n = x.numel()
    for other in (b, gl.dropout(x, 0.4, seed=4, offset=7)):
        both = float(((a != 0) & (other != 0)).double().mean())
        assert abs(both - 0.36) <= 5 * (0.36 * 0.64 / n) ** 0.5
    assert abs(float((a != 0).double().mean()) - 0.6) <= 5 * (0.24 / n) ** 0.5
    at.fill_(-1)
    assert torch.equal(gl.dropout(x, 0.4, seed=3, offset=at), gl.dropout(x, 0.4, seed=3, offset=(1 << 64) - 1))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 5, 8, 1001, 4099])
def test_in_place_and_inside(n, dtype):
    x, st = _rand((n,), 1, dtype), _rand((n,), 2, dtype)
    ref = gl.dropout(x, 0.3, seed=2, stream_in=st, keep=0.5)
    g = Guarded(n * x.element_size(), _dev(), "out")
    out = g.tensor((n,), x.dtype)
    assert gl.dropout(x, 0.3, seed=2, stream_in=st, keep=0.5, out=out) is out
    g.check()
    assert torch.equal(out, ref)
    for target in (x.clone(), st.clone()):
        mine = dict(x=x, st=st)
        if torch.equal(target, x):
            mine["x"] = target
        else:
            mine["st"] = target
        gl.dropout(mine["x"], 0.3, seed=2, stream_in=mine["st"], keep=0.5, out=target)
        assert torch.equal(target, ref)


def test_past_32_bit_offsets():
    """More than 2^32 elements: the last ones are those of their place in the tensor."""
    n = (1 << 32) + 8 * 1000 + 3
    x = torch.ones(n, dtype=torch.bfloat16, device=_dev())
    gl.dropout(x, 0.5, seed=6, out=x)
    for first, count in ((0, 64), ((1 << 31) - 8, 24), ((1 << 32) - 16, 64), (n - 40, 40)):
        f = oracle.mlp.dropout_factor(count, 0.5, 6, first=first)
        assert np.array_equal(_f(x[first:first + count]), f)


def test_empty():
    x = torch.zeros((0, 8), device=_dev())
    assert gl.dropout(x, 0.5, seed=1).shape == (0, 8)
    assert gl.dropout_backward(x, 0.5, seed=1, keep=0.5, stream_grad=True)["d_stream_in"].shape == (0, 8)
