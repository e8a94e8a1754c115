"""Measured cases of the operators around the MoE block: the RMS norm with the
residual's addition and its gradient, the routing of given logits and its
gradient, and the MXFP4 quantisation and dense product.

``run`` computes a case in plain torch operations, or, with ``own`` set, with
the library's entry points; ``exact`` states the same results in 64 bits,
from the operators' definitions alone.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # The pre-norm of a decode step's MoE block: 64 sequences, the stream
        # update and the norm in one pass, E4M3 rows for quantised experts and
        # the bf16 rows that the router reads.
        dict(name="norm decode row", op="norm", T=64, H=5120, dtype="bf16", quant="row", y=True),
        # The same step of a long prompt in front of a block-scaled product:
        # only the 8-bit rows are needed.
        dict(name="norm prefill block", op="norm", T=8192, H=5120, dtype="bf16", quant="block",
             y=False),
        # Training: the gradient of the norm and the stream over one packed
        # sequence batch at the block's width.
        dict(name="norm backward train", op="norm_bwd", T=16384, H=5120, dtype="bf16"),
        # A small fp32 fine-tune of a width that no vector length divides.
        dict(name="norm backward odd", op="norm_bwd", T=1537, H=1001, dtype="f32"),
        # A decode batch with a softmax router: 160 experts in 8 groups ranked
        # by their best expert, weights as they are; some rows are padding.
        dict(name="gate decode softmax", op="gate", T=37, E=160, dtype="bf16", score="softmax",
             groups=8, keep=3, pick="max", k=6, renorm=False, bias=False, pad=True),
        # A long prompt with the block's own routing: sigmoid scores, balance
        # bias, 8 groups of 32 ranked by their two best, top 8 of the best 4.
        dict(name="gate prefill sigmoid", op="gate", T=16384, E=256, dtype="f32", score="sigmoid",
             groups=8, keep=4, pick="top2", k=8, renorm=True, bias=True, pad=False),
        # Training of a softmax router: the gradient of every logit.
        dict(name="gate backward softmax", op="gate_bwd", T=16384, E=256, dtype="f32",
             score="softmax", k=8, renorm=False),
        # Token rows quantised for a 4-bit product: a ragged batch.
        dict(name="quantize tokens", op="quantize", R=1003, C=5120, dtype="bf16"),
        # Expert weights quantised at load time: 8 experts of one shard.
        dict(name="quantize experts", op="quantize", R=8 * 2560, C=5120, dtype="bf16"),
        # A decode step's projection: 64 E4M3 rows against 4-bit weights.
        dict(name="linear decode a8", op="linear", T=64, N=5120, K=5120, a="row"),
        # A ragged prompt chunk with 4-bit rows and 4-bit weights.
        dict(name="linear ragged a4", op="linear", T=1111, N=2560, K=5120, a="mx4"),
        # A long prompt's projection with block-scaled E4M3 rows.
        dict(name="linear prefill a8", op="linear", T=8192, N=5120, K=5120, a="block"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "gate", "gate", "gate_bwd", "quantize", "linear",
                     "linear", "linear"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_bwd"):
        quant = rng.choice(["none", "row", "block"]) if op == "norm" else "none"
        H = _spread(rng, 64, 16384)
        if quant == "block":
            H = max(32, H // 32 * 32)
        elif rng.random() < 0.6:
            H = max(64, H // 64 * 64)
        T = _spread(rng, 1, max(1, min(16384, (8192 if op == "norm" else 16384) * 5120 // H // 2)))
        case = dict(op=op, T=T, H=H, dtype=dtype)
        if op == "norm":
            case.update(quant=quant, y=quant == "none" or rng.random() < 0.5)
        return case
    if op in ("gate", "gate_bwd"):
        groups = rng.choice([1, 1, 4, 8, 16])
        size = rng.choice([4, 8, 10, 16, 20, 32]) if groups > 1 else _spread(rng, 8, 512)
        E = groups * size
        keep = rng.randint(1, groups) if groups > 1 else 1
        k = rng.randint(1, min(16, keep * size))
        score = rng.choice(["softmax", "sigmoid"])
        renorm = rng.random() < 0.6
        T = _spread(rng, 1, max(1, 16384 * 256 // max(E, 256)))
        if op == "gate_bwd":
            return dict(op=op, T=T, E=E, dtype=dtype, score=score, k=k, renorm=renorm)
        return dict(op=op, T=T, E=E, dtype=dtype, score=score, groups=groups, keep=keep,
                    pick=rng.choice(["top2", "max"]), k=k, renorm=renorm,
                    bias=rng.random() < 0.6, pad=rng.random() < 0.3)
    if op == "quantize":
        C = 32 * _spread(rng, 2, 512)
        return dict(op=op, R=_spread(rng, 1, 8 * 2560 * 5120 // C // 2), C=C, dtype=dtype)
    K = 32 * _spread(rng, 8, 320)
    N = _spread(rng, 64, 10240)
    T = _spread(rng, 1, max(1, min(8192, 8192 * 5120 * 5120 // (N * K))))
    return dict(op="linear", T=T, N=N, K=K, a=rng.choice(["row", "block", "mx4"]))


# ------------------------------------------------------------------ the inputs
def _codes(gen, shape):
    return torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.int32).to(torch.uint8)


def _scales(gen, shape, lo, hi):
    return torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.int32).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    op = case["op"]
    s = {"case": dict(case)}
    if op in ("norm", "norm_bwd"):
        T, H, dt = case["T"], case["H"], _DTYPES[case["dtype"]]
        # a few channels of the stream are much larger than the others
        wide = 1.0 + 9.0 * (torch.rand(H, generator=gen, device="cuda") < 0.01)
        s["w"] = 1.0 + 0.1 * normal(H)
        s["eps"] = 1e-6
        # step 11 of the depth-scaled stream, the two weights as fp32 holds them
        s["keep"], s["add"] = torch.tensor([10.0 / 11.0, 1.0 / 11.0]).sqrt().tolist()
        s["stream"] = (normal(T, H) * wide).to(dt)
        if op == "norm":
            s["x"] = normal(T, H).to(dt)
        else:
            s["dy"] = normal(T, H).to(dt)
            s["d_stream"] = normal(T, H).to(dt)
    elif op in ("gate", "gate_bwd"):
        T, E = case["T"], case["E"]
        s["z"] = normal(T, E).to(_DTYPES[case["dtype"]])
        if op == "gate":
            s["bias"] = 0.05 * normal(E) if case["bias"] else None
            s["valid"] = (torch.rand(T, generator=gen, device="cuda") < 0.8) if case["pad"] else None
        else:
            s["dw"] = normal(T, case["k"])
            s["idx"] = s["z"].float().argsort(1, descending=True)[:, :case["k"]].int().contiguous()
        s["rsf"] = 2.5
    elif op == "quantize":
        s["x"] = (normal(case["R"], case["C"]) * torch.exp(normal(case["R"], 1))).to(
            _DTYPES[case["dtype"]])
    else:
        T, N, K = case["T"], case["N"], case["K"]
        s["w"] = _codes(gen, (N, K // 2))
        s["ws"] = _scales(gen, (N, K // 32), 118, 122)
        if case["a"] == "mx4":
            s["x"] = _codes(gen, (T, K // 2))
        else:
            s["x"] = (normal(T, K) * 110.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        if case["a"] == "row":
            s["xs"] = 0.005 + 0.01 * torch.rand(T, generator=gen, device="cuda")
        else:
            s["xs"] = _scales(gen, (T, K // 32), 118, 122)
    return s


# ------------------------------------------------------------------ one pass
def _block_exponent(amax, top):
    """floor(log2 amax) - top per block of 32, at least -127; 0 for a block of zeros."""
    e = torch.frexp(amax)[1] - 1 - top
    return torch.where(amax > 0, e.clamp(min=-127), -127)


def _two_to(e):
    """2^e in fp32 for -127 <= e <= 127."""
    return torch.where(e > -127, ((e + 127) << 23), 1 << 22).to(torch.int32).view(torch.float32)


def _plain_norm(s):
    c = s["case"]
    dt = _DTYPES[c["dtype"]]
    h = s["keep"] * s["stream"].float() + s["add"] * s["x"].float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + s["eps"]) * s["w"]
    out = {"stream": h.to(dt)}
    if c["y"]:
        out["y"] = y.to(dt)
    if c["quant"] == "row":
        amax = y.abs().amax(1)
        live = amax > 0
        amax = torch.where(live, amax, 448.0)
        out["q"] = (y * (448.0 / amax)[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        out["scale"] = amax / 448.0
    elif c["quant"] == "block":
        b = y.view(c["T"], -1, 32)
        sc = _two_to(_block_exponent(b.abs().amax(2), 8))
        q = (b / sc[:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        # a code times its power of two is a bf16 value
        out["q"] = (q.float() * sc[:, :, None]).view(c["T"], c["H"]).to(torch.bfloat16)
    return out


def _own_norm(s):
    import group_limited_routing_amd as gl
    c = s["case"]
    r = gl.add_rms_norm(s["x"], s["w"], stream_in=s["stream"], keep=s["keep"], add=s["add"],
                        norm_eps=s["eps"], return_y=c["y"],
                        quant=None if c["quant"] == "none" else c["quant"])
    out = {"stream": r["stream_out"]}
    if c["y"]:
        out["y"] = r["y"]
    if c["quant"] == "row":
        out["q"], out["scale"] = r["q"], r["q_scale"]
    elif c["quant"] == "block":
        sc = r["q_scale"].view(torch.float8_e8m0fnu).to(torch.bfloat16)
        q = r["q"].to(torch.bfloat16).view(c["T"], -1, 32)
        out["q"] = (q * sc[:, :, None]).view(c["T"], c["H"])
    return out


def _plain_norm_bwd(s):
    h, dy, w = s["stream"].float(), s["dy"].float(), s["w"]
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + s["eps"])
    g = dy * w
    n = h * r
    ds = s["d_stream"].float() + r * (g - n * (g * n).mean(1, keepdim=True))
    dt = s["stream"].dtype
    return {"dx": (s["add"] * ds).to(dt), "d_stream_in": (s["keep"] * ds).to(dt),
            "dw": (dy * n).sum(0)}


def _own_norm_bwd(s):
    import group_limited_routing_amd as gl
    r = gl.add_rms_norm_backward(s["dy"], s["stream"], s["w"], d_stream_out=s["d_stream"],
                                 keep=s["keep"], add=s["add"], norm_eps=s["eps"])
    return {"dx": r["dx"], "d_stream_in": r["d_stream_in"], "dw": r["d_norm_weight"]}


def _plain_gate(s):
    c = s["case"]
    T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
    # 64 bits: the order of two keys decides which expert a token goes to
    z = s["z"].double()
    f = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, 1)
    key = f if s["bias"] is None else f + s["bias"].double()
    if G > 1:
        g = key.view(T, G, E // G).sort(2, descending=True)[0]
        g = g[:, :, 0] + g[:, :, 1] if c["pick"] == "top2" else g[:, :, 0]
        best = g.sort(dim=1, descending=True, stable=True)[1][:, :c["keep"]]
        live = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, best, True)
        key = torch.where(live.repeat_interleave(E // G, 1), key, -math.inf)
    idx = key.sort(dim=1, descending=True, stable=True)[1][:, :k]
    w = f.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = (s["rsf"] * w).float()
    idx = idx.int()
    if s["valid"] is not None:
        idx = torch.where(s["valid"][:, None], idx, -1)
        w = torch.where(s["valid"][:, None], w, 0.0)
    counts = torch.zeros(E + 1, dtype=torch.int32, device=z.device)
    counts.index_add_(0, (idx.view(-1) + 1).long(), torch.ones(T * k, dtype=torch.int32, device=z.device))
    return {"idx": idx, "w": w, "counts": counts[1:]}


def _own_gate(s):
    import group_limited_routing_amd as gl
    c = s["case"]
    r = gl.gate(s["z"], expert_bias=s["bias"], score=c["score"], n_group=c["groups"],
                topk_group=c["keep"], group_score=c["pick"], top_k=c["k"],
                renormalise=c["renorm"], routed_scaling_factor=s["rsf"], valid=s["valid"],
                return_counts=True)
    return {"idx": r["topk_idx"], "w": r["topk_w"], "counts": r["expert_counts"]}


def _plain_gate_bwd(s):
    c = s["case"]
    z, idx, dw = s["z"].float(), s["idx"].long(), s["dw"]
    f = torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, 1)
    p = f.gather(1, idx)
    if c["renorm"]:
        total = p.sum(1, keepdim=True)
        w = p / total
        df = s["rsf"] / total * (dw - (dw * w).sum(1, keepdim=True))
    else:
        df = s["rsf"] * dw
    dz = torch.zeros_like(z).scatter_(1, idx, df)
    if c["score"] == "sigmoid":
        dz = dz * f * (1.0 - f)
    elif c["renorm"]:  # the sum over the chosen df * p is zero: nothing flows to the others
        dz = dz * f
    else:
        dz = f * (dz - (df * p).sum(1, keepdim=True))
    return {"dz": dz.to(s["z"].dtype)}


def _own_gate_bwd(s):
    import group_limited_routing_amd as gl
    c = s["case"]
    return {"dz": gl.gate_backward(s["dw"], s["z"], s["idx"], score=c["score"],
                                   renormalise=c["renorm"], routed_scaling_factor=s["rsf"])}


def _plain_quantize(s):
    b = s["x"].float().view(s["x"].shape[0], -1, 32)
    sc = _two_to(_block_exponent(b.abs().amax(2), 2))[:, :, None]
    v = b / sc
    a = v.abs()
    # E2M1 magnitudes are 0.5 apart below 2, 1 apart below 4, 2 apart up to 6
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    q = (torch.round(a / step) * step).clamp(max=6.0)
    return {"values": (torch.copysign(q, v) * sc).view(s["x"].shape).to(torch.bfloat16)}


def _own_quantize(s):
    import group_limited_routing_amd as gl
    codes, scales = gl.mx4_quantize(s["x"])
    return {"values": gl.mx4_dequantize(codes, scales, dtype=torch.bfloat16)}


def _values_mx4(codes, scales):
    """fp32 values of row-major E2M1 codes (two to a byte) and E8M0 block scales."""
    lut = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    lut = torch.cat((lut, -lut))
    v = torch.stack((lut[(codes & 15).int()], lut[(codes >> 4).int()]), 2)
    return (v.view(codes.shape[0], -1, 32) * _two_to(scales.int() - 127)[:, :, None]).view(
        codes.shape[0], -1)


def _plain_linear(s):
    a = s["case"]["a"]
    if a == "mx4":
        x = _values_mx4(s["x"], s["xs"])
    elif a == "block":
        x = (s["x"].float().view(s["x"].shape[0], -1, 32)
             * _two_to(s["xs"].int() - 127)[:, :, None]).view(s["x"].shape)
    else:
        x = s["x"].float()
    out = x @ _values_mx4(s["w"], s["ws"]).t()
    if a == "row":
        out = out * s["xs"][:, None]
    return {"out": out.to(torch.bfloat16)}


def _own_linear(s):
    import group_limited_routing_amd as gl
    return {"out": gl.mx4_linear(s["x"], s["xs"], s["w"], s["ws"])}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "gate": _own_gate,
                "gate_bwd": _own_gate_bwd, "quantize": _own_quantize, "linear": _own_linear}[op](state)
    return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "gate": _plain_gate,
            "gate_bwd": _plain_gate_bwd, "quantize": _plain_quantize, "linear": _plain_linear}[op](state)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        n, b = case["T"] * case["H"], 2 if case["dtype"] == "bf16" else 4
        if op == "norm_bwd":  # dy, stream, d_stream; dx, d_stream_in; w and dw
            return {"bytes": 5 * n * b + 8 * case["H"], "flops": 14 * n}
        out = n * b + (n * b if case["y"] else 0) + 4 * case["H"]  # the stream, y; w
        out += {"none": 0, "row": n + 4 * case["T"], "block": n + n // 32}[case["quant"]]
        return {"bytes": 2 * n * b + out, "flops": 10 * n}
    if op in ("gate", "gate_bwd"):
        n, b = case["T"] * case["E"], 2 if case["dtype"] == "bf16" else 4
        slots = case["T"] * case["k"] * 8
        if op == "gate_bwd":  # every logit is read only where every logit has a gradient
            full = case["score"] == "softmax" and not case["renorm"]
            return {"bytes": slots + n * b + (n if full else case["T"] * case["k"]) * b,
                    "flops": 8 * n}
        return {"bytes": n * b + slots + 4 * case["E"] + (4 * case["E"] if case["bias"] else 0)
                + (case["T"] if case["pad"] else 0), "flops": 12 * n}
    if op == "quantize":  # the input; codes and scales; the values they stand for
        n = case["R"] * case["C"]
        return {"bytes": n * (2 if case["dtype"] == "bf16" else 4) + n // 2 + n // 32 + 2 * n,
                "flops": 6 * n}
    T, N, K = case["T"], case["N"], case["K"]
    x = {"row": T * K + 4 * T, "block": T * K + T * K // 32, "mx4": T * K // 2 + T * K // 32}[case["a"]]
    return {"bytes": x + N * K // 2 + N * K // 32 + 2 * T * N, "flops": 2 * T * N * K}


# ------------------------------------------------------------------ 64 bits
def _exact_power(v):
    """The largest power of two that is at most each v > 0 (v over its mantissa, exactly)."""
    return v / torch.frexp(v)[0] / 2


def _exact_scale(blocks, largest):
    """The E8M0 scale of each block: the power of two that brings its largest
    magnitude into the top binade of the element format, ``largest`` = its exponent."""
    top = blocks.abs().max(-1).values
    live = top > 0
    p = _exact_power(torch.where(live, top, 1.0)) / 2.0 ** largest
    return torch.where(live, p.clamp(min=2.0 ** -127), 2.0 ** -127)


def _exact_e4m3(v):
    """The nearest E4M3 value, ties to even, magnitudes beyond 448 to 448."""
    a = v.abs()
    quantum = _exact_power(a.clamp(min=2.0 ** -6)) / 8
    return torch.sign(v) * (torch.round(a / quantum) * quantum).clamp(max=448.0)


def _exact_e2m1(v):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 by its borders; a value on a
    border goes to the even code."""
    a = v.abs()
    code = torch.zeros_like(a, dtype=torch.int8)
    for border, up in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        code += (a >= border) if up else (a > border)
    m = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=v.device)[code.int()]
    return torch.where(torch.signbit(v), -m, m)


def _exact_e8m0(scales):
    """One value per element of the blocks of 32."""
    powers = torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device=scales.device)
    return powers[scales.int()].repeat_interleave(32, 1)


def _exact_mx4(codes, scales):
    c = torch.stack((codes % 16, codes // 16), -1).flatten(1).int()
    # code s ee m: m / 2 for ee = 0, else (1 + m / 2) 2^(ee - 1)
    mag = [0.5 * m if e == 0 else (1 + 0.5 * m) * 2.0 ** (e - 1) for e in range(4) for m in range(2)]
    table = torch.tensor(mag + [-m for m in mag], dtype=torch.float64, device=codes.device)
    return table[c] * _exact_e8m0(scales)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["keep"] * s["stream"].double() + s["add"] * s["x"].double()
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["H"] + s["eps"]) * s["w"].double()
        out = {"stream": h}
        if case["y"]:
            out["y"] = y
        if case["quant"] == "row":
            scale = y.abs().max(1, keepdim=True).values / 448
            out["q"], out["scale"] = _exact_e4m3(y / scale), scale[:, 0]
        elif case["quant"] == "block":
            b = y.unflatten(1, (-1, 32))
            scale = _exact_scale(b, 8)[..., None]
            out["q"] = (_exact_e4m3(b / scale) * scale).flatten(1)
        return out
    if op == "norm_bwd":
        h, dy, w = s["stream"].double(), s["dy"].double(), s["w"].double()
        v = (h * h).sum(1, keepdim=True) / case["H"] + s["eps"]
        g = dy * w
        ds = s["d_stream"].double() + g / v.sqrt() - h * (g * h).sum(1, keepdim=True) / (case["H"] * v * v.sqrt())
        return {"dx": s["add"] * ds, "d_stream_in": s["keep"] * ds, "dw": (dy * h / v.sqrt()).sum(0)}
    if op in ("gate", "gate_bwd"):
        z = s["z"].double()
        if case["score"] == "sigmoid":
            f = 1 / (1 + torch.exp(-z))
        else:
            f = torch.exp(z - z.max(1, keepdim=True).values)
            f = f / f.sum(1, keepdim=True)
        if op == "gate":
            T, E, G = case["T"], case["E"], case["groups"]
            left = f if s["bias"] is None else f + s["bias"].double()

            def best(v):
                """The lowest index of each row's largest value."""
                at = torch.arange(v.shape[1], device=v.device)
                return torch.where(v == v.max(1, keepdim=True).values, at, E).min(1, keepdim=True).values

            if G > 1:
                g = left.view(T * G, E // G)
                rank = g.max(1).values
                if case["pick"] == "top2":
                    rank = rank + g.scatter(1, best(g), -math.inf).max(1).values
                rank = rank.view(T, G)
                kept = torch.zeros(T, G, device=z.device)
                for _ in range(case["keep"]):
                    g = best(rank)
                    kept.scatter_(1, g, 1.0)
                    rank = rank.scatter(1, g, -math.inf)
                left = torch.where((kept > 0).repeat_interleave(E // G, 1), left, -math.inf)
            idx = []
            for _ in range(case["k"]):
                idx.append(best(left))
                left = left.scatter(1, idx[-1], -math.inf)
            p = f.gather(1, torch.cat(idx, 1))
            if case["renorm"]:
                p = p / p.sum(1, keepdim=True)
            if s["valid"] is not None:
                p = p * s["valid"][:, None]
            return {"idx": None, "w": s["rsf"] * p, "counts": None}
        idx = s["idx"].long()
        chosen = torch.zeros_like(f).scatter_(1, idx, 1.0)
        dw = torch.zeros_like(f).scatter_(1, idx, s["dw"].double())
        if case["renorm"]:
            total = (f * chosen).sum(1, keepdim=True)
            df = chosen * s["rsf"] * (dw * total - (dw * f * chosen).sum(1, keepdim=True)) / total ** 2
        else:
            df = s["rsf"] * dw
        if case["score"] == "sigmoid":
            return {"dz": df * f * (1 - f)}
        return {"dz": f * df - f * (f * df).sum(1, keepdim=True)}
    if op == "quantize":
        out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        rows = max(1, (1 << 24) // case["C"])
        for r in range(0, case["R"], rows):
            b = s["x"][r:r + rows].double().unflatten(1, (-1, 32))
            scale = _exact_scale(b, 2)[..., None]
            out[r:r + rows] = (_exact_e2m1(b / scale) * scale).flatten(1)
        return {"values": out}
    w = _exact_mx4(s["w"], s["ws"])
    if case["a"] == "mx4":
        x = _exact_mx4(s["x"], s["xs"])
    elif case["a"] == "block":
        x = s["x"].double() * _exact_e8m0(s["xs"])
    else:
        x = s["x"].double() * s["xs"].double()[:, None]
    return {"out": x @ w.t()}
