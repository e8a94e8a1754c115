"""The adapters on batches of more than 65536 tokens, whose chunks are longer than 1024
tokens: the plan's records, and every gradient against fp64 on the GPU."""

import numpy as np
import pytest
import torch

import group_limited_routing_amd as gl
from parity import Guarded
from test_gpu_lora import HALF, _dev, _index, _inputs

pytestmark = pytest.mark.gpu


def _chunk(T):
    """Tokens of a chunk: 1024, or a 64th of the batch, rounded up to 512 tokens."""
    return 1024 if T <= 65536 else (T // 64 + 511) // 512 * 512


@pytest.mark.parametrize("T,E,how", [(65536, 1, "one"), (65537, 1, "one"), (70000, 3, "mixed"), (98305, 1, "one"),
                                     (98305, 200, "runs"), (270000, 2, "mixed")])
def test_plan_of_a_long_batch(T, E, how):
    index = _index(T, E, how, 17)
    need = gl.lib().beam_moe_lora_plan_bytes(T, E)
    buf = Guarded(need, _dev(), "plan")
    assert gl.lib().beam_moe_lora_plan(index.data_ptr(), T, E, buf.view.data_ptr(), need, None) == gl.BEAM_OK
    buf.check()
    plan = buf.view.view(torch.int32).cpu().numpy()
    i = index.cpu().numpy().astype(np.int64)
    g = np.where((i >= 0) & (i < E), i, E)
    order = np.argsort(g, kind="stable")
    up4 = lambda n: (n + 3) // 4 * 4
    chunk, used = _chunk(T), min(E, T)
    most_tiles, most_chunks = T // 64 + min(E + 1, T), T // chunk + used
    o_tiles = 16 + up4(T)
    o_tokens = o_tiles + 4 * most_tiles
    o_chunks = o_tokens + 64 * most_tiles
    o_first = o_chunks + 4 * most_chunks
    o_slot = o_first + up4(E + 1)
    assert need == 4 * (o_slot + up4(E)) and np.array_equal(plan[16:16 + T], order)
    tiles, chunks, first_chunk, slot, slots = [], [], [], [], 0
    first = padded = 0
    for e, c in enumerate(np.bincount(g, minlength=E + 1).tolist()):
        tiles += [(e if e < E else -1, first + j, min(64, c - j), padded + j) for j in range(0, c, 64)]
        if e < E:
            mine = [(e, first + j, min(chunk, c - j), padded + j) for j in range(0, c, chunk)]
            first_chunk.append(len(chunks))
            chunks += mine
            slot.append(slots if len(mine) > 1 else -1)
            slots += len(mine) if len(mine) > 1 else 0
            padded += (c + 31) // 32 * 32
        first += c
    assert plan[0] == len(tiles) <= most_tiles and plan[1] == len(chunks) <= most_chunks
    assert slots <= 2 * (T // chunk) and max(np.bincount([c[0] for c in chunks])) <= 65
    tiles = np.array(tiles)
    assert np.array_equal(plan[o_tiles:o_tokens].reshape(-1, 4)[:len(tiles)], tiles)
    assert np.array_equal(plan[o_chunks:o_first].reshape(-1, 4)[:len(chunks)], np.array(chunks).reshape(-1, 4))
    at = tiles[:, 1:2] + np.minimum(np.arange(64), tiles[:, 2:3] - 1)
    assert np.array_equal(plan[o_tokens:o_chunks].reshape(-1, 64)[:len(tiles)], order[at])
    assert plan[o_first:o_first + E + 1].tolist() == first_chunk + [len(chunks)]
    assert plan[o_slot:o_slot + E].tolist() == slot


@pytest.mark.parametrize("T,K,N,R,E,how", [(70000, 40, 72, 16, 1, "one"), (70000, 72, 40, 40, 3, "mixed"),
                                           (98305, 136, 40, 8, 1, "one"), (98305, 40, 136, 64, 3, "runs")])
def test_gradients_of_a_long_batch(T, K, N, R, E, how):
    """The rounding to bf16 has a root mean square of at most 2^-8 / sqrt(3) of a value; the
    rounding of a sum of T in fp32 is as good as random, T^0.5 2^-24 < 2^-15 of the largest sums,
    and the parts of 16 bits are 2^-16 of them."""
    p, index = _inputs(T, K, N, R, E), _index(T, E, how, 18)
    plan = gl.lora_plan(index, E)
    fw = gl.lora(p["x"], p["a"], p["b"], plan, scale=p["scale"], base=p["base"], return_v=True)
    bw = gl.lora_backward(p["dy"], p["x"], fw["v"], p["a"], p["b"], plan, scale=p["scale"], base=p["dbase"])
    want = dict(out=p["base"].double(), dx=p["dbase"].double(), d_a=torch.zeros_like(p["a"], dtype=torch.float64),
                d_b=torch.zeros_like(p["b"], dtype=torch.float64))
    for e in range(E):
        at = (index == e).nonzero()[:, 0]
        x, a, b, dy = p["x"][at].double(), p["a"][e].double(), p["b"][e].double(), p["dy"][at].double()
        v, s = fw["v"][at].double(), float(p["scale"][e])
        exact = torch.mm(x, a.t().contiguous())
        assert ((v - exact).abs() <= 2.0 ** -18 * exact.abs().max()).all()
        dv = s * torch.mm(dy, b)
        want["out"][at] += s * torch.mm(v, b.t().contiguous())
        want["dx"][at] += torch.mm(dv, a)
        want["d_a"][e] = torch.mm(dv.t().contiguous(), x)
        want["d_b"][e] = s * torch.mm(dy.t().contiguous(), v)
    for name, w in want.items():
        for got, ref in zip(*((t if name[:2] == "d_" else t[None]) for t in ({**fw, **bw}[name], w))):
            err = got.double() - ref
            assert err.norm() <= 1.01 * HALF / 3 ** 0.5 * ref.norm(), name
            assert (err.abs() <= 1.01 * HALF * ref.abs() + 2.0 ** -14 * ref.abs().max()).all(), name
