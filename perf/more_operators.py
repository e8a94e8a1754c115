"""Measured cases of the dense MLP's operators: the gated product (both
projections, the activation and the product) with its gradient, the low-rank
adapters of many requests with their gradient, and dropout from a counter-based
generator.

``run`` computes a case in plain torch operations, or, with ``own`` set, with
the library's entry points; ``exact`` states the same results in 64 bits,
from the operators' definitions alone.
"""

import math

import numpy
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # One sequence's decode step through a narrow dense layer: the latency of a call.
        dict(name="gated one token", op="gated", T=1, H=5120, F=2560, act="silu", adapters=False,
             pre=False),
        # A decode batch through a dense layer: the weights' stream.
        dict(name="gated decode", op="gated", T=64, H=5120, F=10240, act="silu", adapters=False,
             pre=False),
        # A ragged prompt chunk with adapters on both projections, kept for the gradient.
        dict(name="gated ragged adapters", op="gated", T=1111, H=2560, F=5000, act="gelu",
             adapters=True, pre=True),
        # A long prompt.
        dict(name="gated prefill", op="gated", T=8192, H=5120, F=10240, act="silu",
             adapters=False, pre=False),
        # Training: the gradient over one packed batch.
        dict(name="gated backward train", op="gated_bwd", T=4096, H=5120, F=10240, act="silu"),
        # A small fine-tune of sizes that no tile divides.
        dict(name="gated backward ragged", op="gated_bwd", T=777, H=1288, F=1000, act="gelu"),
        # A decode batch of 64 sequences that use 32 adapters between them.
        dict(name="lora decode", op="lora", T=64, K=5120, N=5120, R=16, E=32, mixed=True, v=False),
        # Prompts of several requests, one after the other, with an adapter each.
        dict(name="lora prefill", op="lora", T=8192, K=5120, N=10240, R=16, E=8, mixed=False, v=False),
        # Training of one adapter of a wide rank on a packed batch of odd length.
        dict(name="lora backward train", op="lora_bwd", T=8191, K=5120, N=5120, R=64, E=1, mixed=False),
        # The gradients of several small adapters, tokens in any order.
        dict(name="lora backward mixed", op="lora_bwd", T=515, K=1000, N=2504, R=8, E=5, mixed=True),
        # Training: the block's output dropped out on its way into the stream.
        dict(name="dropout stream train", op="dropout", T=16384, H=5120, dtype="bf16", p=0.1,
             stream=True),
        # Its gradient for fp32 rows of an odd width.
        dict(name="dropout backward odd", op="dropout_bwd", T=1537, H=1001, dtype="f32", p=0.25,
             stream=False),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _eights(rng, lo, hi):
    return 8 * _spread(rng, lo // 8, hi // 8)


def draw(rng):
    op = rng.choice(["gated", "gated", "gated", "gated_bwd", "gated_bwd", "lora", "lora",
                     "lora_bwd", "dropout", "dropout_bwd"])
    if op in ("gated", "gated_bwd"):
        H, F = _eights(rng, 256, 8192), _eights(rng, 256, 12288)
        most = (8192 if op == "gated" else 4096) * 5120 * 10240 // (H * F)
        T = _spread(rng, 1, min(16384, max(1, most)))
        case = dict(op=op, T=T, H=H, F=F, act=rng.choice(["silu", "silu", "gelu"]))
        if op == "gated":
            case.update(adapters=rng.random() < 0.3, pre=rng.random() < 0.3)
        return case
    if op in ("lora", "lora_bwd"):
        E = _spread(rng, 1, 64)
        return dict(op=op, T=_spread(rng, 1, 8192), K=_eights(rng, 256, 5120),
                    N=_eights(rng, 256, 5120 if op == "lora_bwd" else 10240),
                    R=rng.choice([8, 16, 16, 32, 64]) if E <= 32 else rng.choice([8, 16]), E=E,
                    mixed=rng.random() < 0.5, **({"v": rng.random() < 0.3} if op == "lora" else {}))
    H = _spread(rng, 64, 16384)
    if rng.random() < 0.6:
        H = max(64, H // 64 * 64)
    return dict(op=op, T=_spread(rng, 1, min(16384, 16384 * 5120 // H // 2)), H=H,
                dtype=rng.choice(["bf16", "bf16", "f32"]), p=rng.choice([0.05, 0.1, 0.25, 0.5]),
                stream=rng.random() < 0.5)


# ------------------------------------------------------------------ the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)

    op, T = case["op"], case["T"]
    s = {"case": dict(case)}
    if op in ("gated", "gated_bwd"):
        H, F = case["H"], case["F"]
        s["x"] = normal(T, H)
        s["wg"], s["wu"] = normal(F, H, scale=H ** -0.5), normal(F, H, scale=H ** -0.5)
        if op == "gated" and case["adapters"]:
            s["ag"], s["au"] = normal(T, F, scale=0.1), normal(T, F, scale=0.1)
        if op == "gated_bwd":
            s["gate"], s["up"], s["dh"] = normal(T, F), normal(T, F), normal(T, F)
    elif op in ("lora", "lora_bwd"):
        K, N, R, E = case["K"], case["N"], case["R"], case["E"]
        if case["mixed"]:  # a request per token, some of them without an adapter
            index = torch.randint(0, 10 * E, (T,), generator=gen, device="cuda") // 9
            index = torch.where(index < E, index, -1)
        else:  # requests one after the other
            starts = torch.rand(2 * E - 1, generator=gen, device="cuda").sort()[0] * T
            at = torch.searchsorted(starts, torch.arange(T, device="cuda", dtype=torch.float32))
            index = torch.randint(0, E, (2 * E,), generator=gen, device="cuda")[at]
        s["index"] = index.to(torch.int32)
        s["x"] = normal(T, K)
        s["a"], s["b"] = normal(E, R, K, scale=K ** -0.5), normal(E, N, R, scale=R ** -0.5)
        s["scale"] = 0.5 + torch.rand(E, generator=gen, device="cuda")
        if op == "lora":
            s["base"] = normal(T, N)
        else:
            s["base"], s["dy"] = normal(T, K), normal(T, N)
            s["v"] = torch.randn((T, R), generator=gen, device="cuda")
            s["v"][s["index"] < 0] = 0.0
        if own:  # once for all products of a batch
            import group_limited_routing_amd as gl
            s["plan"] = gl.lora_plan(s["index"], E)
    else:
        dt = _DTYPES[case["dtype"]]
        s["x"] = torch.randn((T, case["H"]), generator=gen, device="cuda").to(dt)
        s["stream"] = (torch.randn((T, case["H"]), generator=gen, device="cuda").to(dt)
                       if op == "dropout" and case["stream"] else None)
        # step 11 of the depth-scaled stream, the two weights as fp32 holds them
        s["keep"], s["add"] = torch.tensor([10.0 / 11.0, 1.0 / 11.0]).sqrt().tolist()
        s["seed"], s["offset"] = 0x9D3A5 * (int(seed) + 1) + (1 << 40), 3 * int(seed) + 1
    return s


# ------------------------------------------------------------------ one pass
def _act(g, act):
    """act(g) and its derivative, in fp32."""
    if act == "silu":
        q = torch.sigmoid(g)
        return g * q, q * (1.0 + g * (1.0 - q))
    q = 0.5 * (1.0 + torch.erf(g * 0.5 ** 0.5))
    return g * q, q + g * torch.exp(-0.5 * g * g) * (2.0 * math.pi) ** -0.5


def _plain_gated(s):
    c = s["case"]
    x = s["x"].float()
    gate, up = x @ s["wg"].float().t(), x @ s["wu"].float().t()
    if c["adapters"]:
        gate, up = gate + s["ag"].float(), up + s["au"].float()
    out = {"h": (_act(gate, c["act"])[0] * up).to(torch.bfloat16)}
    if c["pre"]:
        out["gate"], out["up"] = gate.to(torch.bfloat16), up.to(torch.bfloat16)
    return out


def _own_gated(s):
    import group_limited_routing_amd as gl
    c = s["case"]
    r = gl.gated_linear(s["x"], s["wg"], s["wu"], activation=c["act"], add_gate=s.get("ag"),
                        add_up=s.get("au"), return_pre=c["pre"])
    return r if c["pre"] else {"h": r["h"]}


def _plain_gated_bwd(s):
    x, dh, up = s["x"].float(), s["dh"].float(), s["up"].float()
    f, df = _act(s["gate"].float(), s["case"]["act"])
    d_gate, d_up = dh * up * df, dh * f
    dx = d_gate @ s["wg"].float() + d_up @ s["wu"].float()
    out = {"dx": dx, "d_w_gate": d_gate.t() @ x, "d_w_up": d_up.t() @ x, "d_gate": d_gate, "d_up": d_up}
    return {k: v.to(torch.bfloat16) for k, v in out.items()}


def _own_gated_bwd(s):
    import group_limited_routing_amd as gl
    return gl.gated_linear_backward(s["dh"], s["x"], s["wg"], s["wu"], s["gate"], s["up"],
                                    activation=s["case"]["act"])


def _chosen(s):
    """[T, E]: the scale of each token's own adapter, 0 at the others'."""
    e = torch.arange(s["case"]["E"], device=s["index"].device)
    return (s["index"][:, None] == e) * s["scale"]


def _plain_lora(s):
    c = s["case"]
    T, K, N, R, E = c["T"], c["K"], c["N"], c["R"], c["E"]
    own_scale = _chosen(s)[:, :, None]
    v = (s["x"].float() @ s["a"].float().view(E * R, K).t()).view(T, E, R)
    sv = (v * own_scale).view(T, E * R)
    out = {"out": (s["base"].float() + sv @ s["b"].float().transpose(1, 2).reshape(E * R, N)).to(
        torch.bfloat16)}
    if c["v"]:
        out["v"] = (v * (own_scale > 0)).sum(1)
    return out


def _own_lora(s):
    import group_limited_routing_amd as gl
    r = gl.lora(s["x"], s["a"], s["b"], s["plan"], scale=s["scale"], base=s["base"],
                return_v=s["case"]["v"])
    return r if s["case"]["v"] else {"out": r["out"]}


def _plain_lora_bwd(s):
    c = s["case"]
    T, K, N, R, E = c["T"], c["K"], c["N"], c["R"], c["E"]
    own_scale = _chosen(s)[:, :, None]
    x, dy = s["x"].float(), s["dy"].float()
    dv = (dy @ s["b"].float().transpose(1, 2).reshape(E * R, N).t()).view(T, E, R) * own_scale
    dv = dv.view(T, E * R)
    sv = (s["v"][:, None, :] * own_scale).view(T, E * R)
    return {"dx": (s["base"].float() + dv @ s["a"].float().view(E * R, K)).to(torch.bfloat16),
            "d_a": (dv.t() @ x).view(E, R, K).to(torch.bfloat16),
            "d_b": (sv.t() @ dy).view(E, R, N).transpose(1, 2).to(torch.bfloat16)}


def _own_lora_bwd(s):
    import group_limited_routing_amd as gl
    return gl.lora_backward(s["dy"], s["x"], s["v"], s["a"], s["b"], s["plan"], scale=s["scale"],
                            base=s["base"])


def _mul_hi(c, m):
    """The upper 32 bits of c * m, both below 2^32, in int64 that cannot overflow."""
    return (c * (m >> 16) + ((c * (m & 0xffff)) >> 16)) >> 16


def _random16(n, seed, offset, device):
    """16 random bits for each of n elements: Philox4x32-10 at the counter
    (element / 8, offset) under the key ``seed``; two elements to a word."""
    low = 0xffffffff
    j = torch.arange((n + 7) // 8, device=device)
    c0, c1 = j & low, j >> 32
    c2, c3 = torch.full_like(j, offset & low), torch.full_like(j, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        h0, l0 = _mul_hi(c0, 0xD2511F53), (c0 * 0xD2511F53) & low
        h1, l1 = _mul_hi(c2, 0xCD9E8D57), (c2 * 0xCD9E8D57) & low
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((c0, c1, c2, c3), 1)
    return torch.stack((words & 0xffff, words >> 16), 2).view(-1)[:n]


def _plain_dropout(s):
    c, x = s["case"], s["x"]
    border = math.floor(c["p"] * 65536 + 0.5)
    kept = (_random16(x.numel(), s["seed"], s["offset"], x.device) >= border).view(x.shape)
    out = s["add"] * torch.where(kept, x.float() * (65536.0 / (65536 - border)), 0.0)
    if s["stream"] is not None:
        out = out + s["keep"] * s["stream"].float()
    if c["op"] == "dropout":
        return {"out": out.to(x.dtype)}
    r = {"dx": out.to(x.dtype)}
    if c["stream"]:
        r["d_stream_in"] = (s["keep"] * x.float()).to(x.dtype)
    return r


def _own_dropout(s):
    import group_limited_routing_amd as gl
    c = s["case"]
    how = dict(seed=s["seed"], offset=s["offset"], keep=s["keep"], add=s["add"])
    if c["op"] == "dropout":
        return {"out": gl.dropout(s["x"], c["p"], stream_in=s["stream"], **how)}
    r = gl.dropout_backward(s["x"], c["p"], stream_grad=c["stream"], **how)
    return r if c["stream"] else {"dx": r["dx"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"gated": _own_gated, "gated_bwd": _own_gated_bwd, "lora": _own_lora,
                "lora_bwd": _own_lora_bwd, "dropout": _own_dropout, "dropout_bwd": _own_dropout}[op](state)
    return {"gated": _plain_gated, "gated_bwd": _plain_gated_bwd, "lora": _plain_lora,
            "lora_bwd": _plain_lora_bwd, "dropout": _plain_dropout,
            "dropout_bwd": _plain_dropout}[op](state)


# ------------------------------------------------------------------ work
def work(case):
    op, T = case["op"], case["T"]
    if op == "gated":  # x, both weights, the adapters' shares; h and both pre-activations
        H, F = case["H"], case["F"]
        rows = 1 + 2 * case["adapters"] + 2 * case["pre"]
        return {"bytes": 2 * (T * H + 2 * F * H + rows * T * F), "flops": 4 * T * F * H}
    if op == "gated_bwd":  # x, weights, dh, gate, up; dx, the weights' gradients, d_gate, d_up
        H, F = case["H"], case["F"]
        return {"bytes": 2 * (2 * T * H + 4 * F * H + 5 * T * F), "flops": 8 * T * F * H}
    if op in ("lora", "lora_bwd"):
        K, N, R, E = case["K"], case["N"], case["R"], min(case["E"], T)
        if op == "lora":  # x, base, out; the adapters; v
            return {"bytes": 2 * T * (K + 2 * N) + 2 * E * R * (K + N) + 4 * T * (1 + R * case["v"]),
                    "flops": 2 * T * R * (K + N)}
        # dy, x, base, dx; v; the adapters and their gradients
        return {"bytes": 2 * T * (N + 3 * K) + 4 * T * (R + 1) + 2 * R * (K + N) * (E + case["E"]),
                "flops": 4 * T * R * (K + N)}
    n, b = T * case["H"], 2 if case["dtype"] == "bf16" else 4
    return {"bytes": (3 if case["stream"] else 2) * n * b, "flops": 4 * n}


# ------------------------------------------------------------------ 64 bits
def _exact_random16(n, seed, offset):
    """The generator again, in numpy's unsigned 64-bit integers."""
    u = numpy.uint64
    j = numpy.arange((n + 7) // 8, dtype=u)
    word = [j & u(0xffffffff), j >> u(32), numpy.full_like(j, offset % 2 ** 32),
            numpy.full_like(j, offset // 2 ** 32)]
    key = [seed % 2 ** 32, seed // 2 ** 32]
    for _ in range(10):
        a, b = word[0] * u(0xD2511F53), word[2] * u(0xCD9E8D57)
        word = [(b >> u(32)) ^ word[1] ^ u(key[0]), b & u(0xffffffff),
                (a >> u(32)) ^ word[3] ^ u(key[1]), a & u(0xffffffff)]
        key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
    out = numpy.empty((j.size, 4, 2), dtype=numpy.int32)
    for i in range(4):
        out[:, i, 0], out[:, i, 1] = word[i] % u(65536), word[i] // u(65536)
    return torch.from_numpy(out.reshape(-1)[:n])


def exact(case, seed):
    s = prepare(case, seed)
    op, T = case["op"], case["T"]
    if op in ("gated", "gated_bwd"):
        x, wg, wu = s["x"].double(), s["wg"].double(), s["wu"].double()
        if op == "gated":
            g, u = torch.mm(x, wg.mT.contiguous()), torch.mm(x, wu.mT.contiguous())
            if case["adapters"]:
                g += s["ag"].double()
                u += s["au"].double()
        else:
            g, u = s["gate"].double(), s["up"].double()
        if case["act"] == "silu":  # g / (1 + e^-g), and its derivative by the quotient rule
            e = torch.exp(-g)
            f, df = g / (1 + e), (1 + e + g * e) / (1 + e) ** 2
        else:  # g Phi(g), Phi by the complementary error function
            phi = torch.special.erfc(-g / math.sqrt(2)) / 2
            f, df = g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        if op == "gated":
            return {"h": f * u, "gate": g, "up": u} if case["pre"] else {"h": f * u}
        dh = s["dh"].double()
        dg, du = dh * u * df, dh * f
        xt = x.mT.contiguous()
        return {"dx": torch.mm(dg, wg) + torch.mm(du, wu), "d_w_gate": torch.mm(xt, dg).mT,
                "d_w_up": torch.mm(xt, du).mT, "d_gate": dg, "d_up": du}
    if op in ("lora", "lora_bwd"):
        x, base = s["x"].double(), s["base"].double()
        if op == "lora":
            out, v = base.clone(), torch.zeros(T, case["R"], dtype=torch.float64, device=x.device)
        else:
            dx = base.clone()
            da = torch.zeros(s["a"].shape, dtype=torch.float64, device=x.device)
            db = torch.zeros(s["b"].shape, dtype=torch.float64, device=x.device)
        for e in range(case["E"]):  # one adapter's tokens after the other's
            at = (s["index"] == e).nonzero()[:, 0]
            a, b, f = s["a"][e].double(), s["b"][e].double(), float(s["scale"][e])
            if op == "lora":
                v[at] = torch.mm(x[at], a.mT.contiguous())
                out[at] += f * torch.mm(v[at], b.mT.contiguous())
            else:
                dy, v = s["dy"][at].double(), s["v"][at].double()
                dv = f * torch.mm(dy, b)
                dx[at] += torch.mm(dv, a)
                da[e] = torch.mm(dv.mT.contiguous(), x[at])
                db[e] = f * torch.mm(dy.mT.contiguous(), v)
        if op == "lora":
            return {"out": out, "v": v} if case["v"] else {"out": out}
        return {"dx": dx, "d_a": da, "d_b": db}
    x = s["x"].double()
    border = round(case["p"] * 65536)
    kept = _exact_random16(x.numel(), s["seed"], s["offset"]).view(x.shape).cuda() >= border
    out = s["add"] * kept * x / (1 - border / 65536)
    if op == "dropout":
        return {"out": out if s["stream"] is None else out + s["keep"] * s["stream"].double()}
    return {"dx": out, "d_stream_in": s["keep"] * x} if case["stream"] else {"dx": out}
