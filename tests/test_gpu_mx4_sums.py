"""Sums of the dense MXFP4 product keep 32 bits, with E4M3 rows as with 4-bit rows.

An E4M3 value is a multiple of 2^-9 and an E2M1 value of 2^-1, so with equal
scales every product is a multiple of one unit, 2^-10 of them. Where the magnitudes of a
sum stay below 2^24 units, each partial sum is an fp32 number, in any order and
any grouping: the output has to be the exact sum, and in bf16 its one rounding.
In general the reduction adds K / 8 groups, twice with E4M3 rows, each addition
at most one step (2^-23) of the sum of magnitudes off, and its splits fewer than
64 more; then one rounding to the output type and one for a row's scale.
"""

import pytest
import torch

import group_limited_routing_amd as gl
import test_gpu_mx4 as product

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
UNIT = 2.0 ** -10
# every kernel of the product with E4M3 rows: streams of 16, 32 and 64 tokens, 32 and 64
# columns wide, and the tiles of 64, 128 and 256
STREAMS = [(5, 70), (5, 16000), (20, 5100), (30, 16000), (50, 700), (60, 16001), (250, 5121)]
TILES = [(384, 5121), (500, 5100), (2020, 5115), (2900, 5100)]


def _dev():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return torch.device("cuda:0")


def _gen(seed):
    return torch.Generator(device=_dev()).manual_seed(seed)


def _bytes(shape, seed):
    return torch.randint(0, 256, shape, generator=_gen(seed), device=_dev(), dtype=torch.int32).to(torch.uint8)


def _any_e4m3(shape, seed):
    """Every finite E4M3 code, subnormals and the largest among them, alike often."""
    c = torch.randint(0, 127, shape, generator=_gen(seed), device=_dev(), dtype=torch.int32)
    sign = torch.randint(0, 2, shape, generator=_gen(seed + 1), device=_dev(), dtype=torch.int32)
    return (c + 128 * sign).to(torch.uint8).view(torch.float8_e4m3fn)


@pytest.mark.parametrize("fmt", ["row", "block"])
@pytest.mark.parametrize("T,N,K", [(T, N, K) for T, N in STREAMS for K in (32, 160, 512, 1120)] +
                         [(T, N, K) for T, N in TILES for K in (32, 96, 160, 384, 416, 448, 512, 544, 672, 1120)])
def test_linear_sums_are_exact(T, N, K, fmt):
    dev = _dev()
    x = _any_e4m3((T, K), 1).float()
    # up to 40 values of a row are not zero, in whole groups of 8
    groups = torch.rand((T, K // 8), generator=_gen(3), device=dev)
    x = (x.view(T, K // 8, 8) * (groups <= groups.sort(1)[0][:, min(4, K // 8 - 1), None])[:, :, None]).view(T, K)
    x = x.to(torch.float8_e4m3fn)
    w, ws = _bytes((N, K // 2), 4), torch.full((N, K // 32), 125, dtype=torch.uint8, device=dev)
    xv, wv = x.double(), gl.mx4_dequantize(w, ws, dtype=torch.float32).double()
    if fmt == "row":
        xs = torch.exp2(torch.arange(T, device=dev) % 5 - 2.0)
        xv, unit = xv * xs.double()[:, None], UNIT / 4 * xs.double()[:, None]
    else:
        xs = torch.full((T, K // 32), 130, dtype=torch.uint8, device=dev)
        xv, unit = xv * 8, torch.full((T, 1), UNIT / 4 * 8, dtype=torch.float64, device=dev)
    ref = xv @ wv.t().contiguous()
    small = xv.abs() @ wv.abs().t().contiguous() < 2.0 ** 24 * unit
    assert float(small.double().mean()) > 0.7
    got = gl.mx4_linear(x, xs, w, ws, out_dtype=torch.float32).double()
    assert torch.equal(got[small], ref[small]), float((got - ref)[small].abs().max())
    got = gl.mx4_linear(x, xs, w, ws)
    assert torch.equal(got[small], ref.to(torch.float32).to(torch.bfloat16)[small])


@pytest.mark.parametrize("fmt", ["row", "block", "mx4"])
@pytest.mark.parametrize("T,N,K", [(3, 130, 5120), (60, 512, 5152), (300, 300, 2080), (1111, 640, 5120),
                                   (2020, 5115, 1024)])
def test_linear_sums_in_general(T, N, K, fmt):
    dev = _dev()
    w, ws = _bytes((N, K // 2), 5), (118 + _bytes((N, K // 32), 6) % 8).to(torch.uint8)
    wv = gl.mx4_dequantize(w, ws, dtype=torch.float32).double()
    xs = (118 + _bytes((T, K // 32), 7) % 8).to(torch.uint8)
    if fmt == "mx4":
        x = _bytes((T, K // 2), 8)
        xv = gl.mx4_dequantize(x, xs, dtype=torch.float32).double()
    else:
        x = (torch.randn((T, K), generator=_gen(8), device=dev) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
        xv = (x.double().view(T, -1, 32) * torch.exp2(xs.double() - 127)[:, :, None]).view(T, K)
        if fmt == "row":
            xs = 0.01 + 0.1 * torch.rand(T, generator=_gen(9), device=dev)
            xv = x.double() * xs.double()[:, None]
    ref = xv @ wv.t().contiguous()
    mag = xv.abs() @ wv.abs().t().contiguous()
    adds = (K // 8 if fmt == "mx4" else K // 4) + 66
    for out, half in ((torch.float32, U), (torch.bfloat16, 2.0 ** -8)):
        err = (gl.mx4_linear(x, xs, w, ws, out_dtype=out).double() - ref).abs()
        assert bool((err <= half * ref.abs() + adds * 2 * U * mag).all())
        # independent roundings of partial sums, which in the norm are no larger than the
        # whole: they add up as the root of their number
        if out == torch.float32:
            assert float(err.norm() / ref.norm()) <= 2 * U * adds ** 0.5


@pytest.mark.parametrize("fmt", ["row", "block"])
@pytest.mark.parametrize("T,N", TILES[::3])
def test_linear_tiles_keep_to_their_rows(T, N, fmt):
    """The tiles of 64 and 256 with E4M3 rows: a NaN scale at a row's start is its
    own row's alone, and not a byte around the output changes."""
    for K in (160, 416, 544, 608):
        product.test_linear_scales_behind_a_row_stay_out(T, N, K, fmt)
    product.test_linear_writes_its_rows_only(T, N, fmt)
