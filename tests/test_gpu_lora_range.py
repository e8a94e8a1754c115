"""The adapters at the ends of the number range, against oracle.mlp in float64: a v beyond
the largest bf16 number, and infinities in the rows and the adapters."""

import numpy as np
import pytest
import torch

import group_limited_routing_amd as gl
import oracle
from test_gpu_lora import HALF, SPLIT, U, _dev, _f

pytestmark = pytest.mark.gpu


def _bf(a):
    return torch.as_tensor(a, dtype=torch.float64).to(torch.bfloat16).to(_dev())


def _matches(got, want, mag, terms, name):
    """A NaN where the definition has one, an infinity where it has one or the value
    rounds to one, else the bound of test_gpu_lora.py with ``mag``, the same sum of
    magnitudes (infinite ones are not asked)."""
    got = _f(got)
    assert np.array_equal(np.isnan(got), np.isnan(want)), name
    rounded = torch.from_numpy(want).to(torch.bfloat16).double().numpy()
    ends = np.isinf(rounded)
    assert np.array_equal(got[ends], rounded[ends]), name
    at = np.isfinite(rounded)
    e = (terms * U + SPLIT) * mag[at]
    assert (np.abs(got[at] - want[at]) <= HALF * (np.abs(want[at]) + e) + e).all(), name


def _check(x, a, b, index, dy, v=None):
    """Forward, and the gradients from ``v`` (None: the forward's own)."""
    xs, As, bs, dys = (_bf(t) for t in (x, a, b, dy))
    x, a, b, dy = (_f(t) for t in (xs, As, bs, dys))
    plan = gl.lora_plan(torch.as_tensor(index, dtype=torch.int32, device=_dev()), a.shape[0])
    fw = gl.lora(xs, As, bs, plan, return_v=True)
    T, K, N, R = x.shape[0], x.shape[1], b.shape[1], a.shape[1]
    with np.errstate(invalid="ignore", over="ignore"):
        out, _ = oracle.mlp.lora(x, a, b, index)
        mag, _ = oracle.mlp.lora(abs(x), abs(a), abs(b), index)
        _matches(fw["out"], out, mag, 2 * K + 4 * R + 8, "out")
        vs = fw["v"] if v is None else torch.as_tensor(v, dtype=torch.float32, device=_dev())
        bw = gl.lora_backward(dys, xs, vs, As, bs, plan)
        want = oracle.mlp.lora_backward(dy, x, _f(vs), a, b, index)
        mags = oracle.mlp.lora_backward(abs(dy), abs(x), abs(_f(vs)), abs(a), abs(b), index)
        for name, w, m in zip(("dx", "d_a", "d_b"), want, mags):
            _matches(bw[name], w, m, 2 * N + 4 * max(R, T) + 64, name)
    return fw, bw


BIG = 2.0 ** 128 - 2.0 ** 112  # sums of powers of two, exact in fp32; bf16 rounds it to an infinity


@pytest.mark.parametrize("R", [8, 16, 24, 64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_v_beyond_the_largest_bf16(R, sign):
    """v, and dv of the gradients, of 2^128 - 2^112: the products have their values,
    and are infinite only where they are beyond bf16. An infinite v gives infinities."""
    K = N = 16
    parts, falling = 2.0 ** (63 - np.arange(K)), 2.0 ** -np.arange(K)
    x, a, b = np.zeros((3, K)), np.zeros((2, R, K)), np.zeros((2, N, R))
    x[0], x[1, 0], x[2, 0] = sign * parts, np.inf, 1.0
    a[0, 0] = 2.0 ** 64
    a[1, :, 0] = 1.0  # every rank of token 1 is infinite
    b[0, :, 0] = falling
    b[1] = 1.0
    index = [0, 1, 0]
    fw, _ = _check(x, a, b, index, np.zeros((3, N)), v=np.zeros((3, R)))
    assert fw["v"][0, 0] == sign * BIG and not fw["v"][0, 1:].any() and (fw["v"][1] == np.inf).all()
    assert (fw["out"][1] == np.inf).all() and fw["out"][0, 0] == sign * np.inf
    # dv the same way; d_b from a v of that size
    dy, x = np.zeros((3, N)), np.zeros((3, K))
    dy[0], dy[1], dy[2] = sign * parts, 2.0 ** -60 * falling, 2.0 ** -70 * falling
    x[0] = falling
    a, b = np.zeros((2, R, K)), np.zeros((2, N, R))
    a[0, 0] = falling
    b[0, :, 0] = 2.0 ** 64
    v = np.zeros((3, R))
    v[1, 0], v[1, 3] = sign * BIG, -sign * BIG
    _, bw = _check(x, a, b, index, dy, v=v)
    assert bw["dx"][0, 0] == sign * np.inf and torch.isfinite(bw["dx"][0, 1:]).all()
    assert bw["d_a"][0, 0, 0] == sign * np.inf and torch.isfinite(bw["d_a"][0, 0, 1:]).all()


@pytest.mark.parametrize("value", [np.inf, -np.inf])
@pytest.mark.parametrize("where", ["x", "a", "b", "dy"])
@pytest.mark.parametrize("T,R,whole", [(5, 8, True), (70, 16, False), (1100, 24, True), (1100, 64, False),
                                       (40, 128, False)])
def test_infinite_operands(T, R, whole, where, value):
    """One infinity in a row or an adapter: infinities of the definition's sign, not NaN, in
    what it reaches, and nothing else changes. v and dv of few bits (``whole``, so that a
    second part of them is 0) and of many (so that it has either sign)."""
    K, N, E = 24, 40, 2
    rng = np.random.default_rng(T + R)
    # whole numbers from 1 to 3 of either sign: sums below 2^8 of the K products of a v
    some = lambda *s: (rng.integers(1, 4, s) * rng.choice([-1.0, 1.0], s)) if whole else rng.standard_normal(s)
    p = dict(x=some(T, K), a=some(E, R, K), b=some(E, N, R), dy=some(T, N))
    index = rng.integers(-1, E, T)
    index[T // 2] = 0
    v = some(T, R)
    p[where][{"x": (T // 2, 3), "dy": (T // 2, 37), "a": (0, R - 1, 5), "b": (0, 17, 2)}[where]] = value
    fw, bw = _check(p["x"], p["a"], p["b"], index, p["dy"], v=v)
    hit = {"x": (bw["d_a"][0, :, 3],), "dy": (bw["d_b"][0, 37],), "a": (fw["out"][T // 2], bw["dx"][T // 2, 5]),
           "b": (fw["out"][T // 2, 17], bw["dx"][T // 2])}[where]
    assert any(t.isinf().any() for t in hit)
