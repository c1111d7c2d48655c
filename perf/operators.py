"""Measured cases of the Mixture-of-Experts token movement and of the 8-bit
integer products.

Each case is one call (or one short chain of calls) that a layer makes:

* ``sort``         -- expert choices -> slots and counts, rows copied to their experts
* ``sort_grad``    -- the gradient of that copy: each token sums its rows' gradients
* ``combine``      -- each token sums its rows, weighted
* ``combine_grad`` -- the gradients of that sum: of the rows and of the weights
* ``product``      -- int8 x int8 with a scale per row and per column
* ``linear``       -- activations quantised per row, then the int8 product
* ``experts``      -- the int8 product of every expert with its own rows

``run`` computes a case in plain torch operations in 32 bits, or, with
``own``, through the library's entry points.  ``exact`` gives the result in
64 bits.  Inputs are drawn from the seed alone.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"f16": 2, "bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def _moe(op, tokens, topk, groups, capacity, width, dtype, name=None):
    case = {"op": op, "tokens": tokens, "topk": topk, "groups": groups, "capacity": capacity,
            "width": width, "dtype": dtype}
    if name:
        case["name"] = name
    return case


def _product(op, M, N, K, dtype, act="none", bias=False, name=None):
    case = {"op": op, "M": M, "N": N, "K": K, "dtype": dtype, "act": act, "bias": bias}
    if name:
        case["name"] = name
    return case


def _experts(tokens, topk, groups, capacity, N, K, dtype, act, name=None):
    case = {"op": "experts", "tokens": tokens, "topk": topk, "groups": groups, "capacity": capacity,
            "N": N, "K": K, "dtype": dtype, "act": act}
    if name:
        case["name"] = name
    return case


def listed():
    return [
        # one decode step of 16 sequences through 8 experts of width 4096: latency
        _moe("sort", 16, 2, 8, 16, 4096, "f16", "sort_decode"),
        # a whole prompt through the same experts, as the grouped product's 8-expert layout
        _moe("sort", 8192, 2, 8, 4096, 4096, "f16", "sort_prompt"),
        # training through 64 small experts, the gradient towards the tokens
        _moe("sort_grad", 4096, 6, 64, 512, 2048, "bf16", "sort_grad"),
        # the way back of one decode step through 64 experts: latency
        _moe("combine", 16, 6, 64, 16, 2048, "f16", "combine_decode"),
        # the way back of a whole prompt
        _moe("combine", 8192, 2, 8, 4096, 4096, "bf16", "combine_prompt"),
        # training, an odd number of tokens: the gradients of rows and weights
        _moe("combine_grad", 4095, 6, 64, 512, 2048, "f16", "combine_grad"),
        # a projection in a decode step of 16 sequences, activations quantised on the way
        _product("linear", 16, 14336, 4096, "f16", name="linear_decode"),
        # the same over a long prompt with an odd number of tokens: the largest product
        _product("linear", 8191, 8192, 8192, "bf16", name="linear_prompt"),
        # one token through a square projection: the smallest product, latency
        _product("product", 1, 4096, 4096, "f32", name="product_token"),
        # a batch of decoded tokens, every size odd, with bias and activation
        _product("product", 97, 14333, 4095, "f32", "gelu", True, name="product_batch"),
        # a decode step of 32 sequences through 64 experts
        _experts(32, 6, 64, 32, 1408, 2048, "f16", "silu", "experts_decode"),
        # a prompt through 64 experts, as the grouped product's 64-expert layout
        _experts(4096, 6, 64, 512, 1408, 2048, "f16", "silu", "experts_prompt"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    """One more case: tokens from 1 to 8192, widths and depths from a few
    hundred to 8192 with odd ones among them, 4 to 64 experts."""
    op = rng.choice(["sort", "sort_grad", "combine", "combine_grad", "product", "product", "linear",
                     "linear", "experts", "experts"])
    dtype = rng.choice(["f16", "bf16"])
    if op in ("product", "linear"):
        M = _log(rng, 1, 8192)
        K = _log(rng, 256, 8192)
        N = _log(rng, 256, 8192)
        if rng.random() < 0.5:
            N = max(16, N // 16 * 16)
        act = rng.choice(["none", "none", "gelu", "silu", "relu"])
        return _product(op, M, N, K, rng.choice(["f16", "bf16", "f32"]), act, rng.random() < 0.5)
    groups = _log(rng, 4, 64)
    topk = rng.randint(1, min(6, groups))
    tokens = _log(rng, 1, 8192)
    fair = tokens * topk / groups
    capacity = max(1, min(tokens, int(fair * rng.uniform(1.0, 2.0)) + 8))
    if op == "experts":
        tokens = min(tokens, 4096)
        capacity = min(capacity, 512)
        return _experts(tokens, topk, groups, capacity, _log(rng, 256, 2048), _log(rng, 256, 2048),
                        dtype, rng.choice(["none", "silu", "gelu"]))
    width = _log(rng, 256, 4096)
    if rng.random() < 0.75:
        width = max(8, width // 8 * 8)
    return _moe(op, tokens, topk, groups, capacity, width, dtype)


# ------------------------------------------------------------------ inputs

def _popularity(groups):
    """Log-weights of a router whose busiest expert gets about three times
    what its least busy one gets."""
    return np.linspace(0.55, -0.55, groups)


def _choices(tokens, topk, groups, seed):
    """topk different experts per token (tokens x topk, int32), drawn by the
    experts' popularity, and each token's normalised weights (f32)."""
    g = np.random.default_rng(seed)
    z = _popularity(groups)[None, :] + g.gumbel(size=(tokens, groups))
    ids = np.argsort(-z, axis=1)[:, :topk].astype(np.int32)
    w = np.exp(g.standard_normal((tokens, topk)))
    w = (w / w.sum(axis=1, keepdims=True)).astype(np.float32)
    return np.ascontiguousarray(ids), w


def _slots_of(ids, groups, capacity):
    """Slots and counts in numpy: the rows of an expert in token order, those
    past the capacity dropped."""
    flat = ids.reshape(-1)
    slots = np.full(flat.shape, -1, dtype=np.int32)
    counts = np.zeros(groups, dtype=np.int32)
    for e in range(groups):
        at = np.flatnonzero(flat == e)[:capacity]
        slots[at] = e * capacity + np.arange(at.size)
        counts[e] = at.size
    return slots.reshape(ids.shape), counts


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)


def _normal(shape, g, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _int8(batch, rows, cols, g):
    """Codes of quantised normal values (most of them small, up to +-127), the
    row pitch a multiple of 16 bytes."""
    pitch = -(-cols // 16) * 16
    x = torch.randn((batch, rows, pitch), generator=g, device="cuda", dtype=torch.float32) * 36.0
    return x.round_().clamp_(-127, 127).to(torch.int8)[:, :, :cols]


def _scales(shape, g):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32) * 0.01 + 0.002


def _empty_out(batch, rows, cols, dtype):
    return torch.zeros((batch, rows, -(-cols // 8) * 8), device="cuda", dtype=dtype)[:, :, :cols]


def prepare(case, seed):
    op = case["op"]
    dtype = _TYPES[case["dtype"]]
    g = _generator(seed)
    s = dict(case)
    if op in ("product", "linear"):
        M, N, K = case["M"], case["N"], case["K"]
        if op == "product":
            s["A"] = _int8(1, M, K, g)[0]
            s["scale_a"] = _scales((M,), g)
        else:
            # activations with a spread of row magnitudes and a few large channels
            x = torch.randn((M, K), generator=g, device="cuda") * torch.exp(
                torch.randn((M, 1), generator=g, device="cuda"))
            x[:, ::97] *= 6.0
            s["x"] = x.to(dtype)
        s["B"] = _int8(1, K, N, g)[0]
        s["scale_b"] = _scales((N,), g)
        s["bias_v"] = torch.randn((N,), generator=g, device="cuda") if case["bias"] else None
        s["out"] = _empty_out(1, M, N, dtype)[0]
    elif op == "experts":
        G, cap, N, K = case["groups"], case["capacity"], case["N"], case["K"]
        ids, _ = _choices(case["tokens"], case["topk"], G, seed)
        _, counts = _slots_of(ids, G, cap)
        s["counts"] = torch.from_numpy(counts).cuda()
        s["A"] = _int8(G, cap, K, g)
        s["scale_a"] = _scales((G, cap), g)
        s["B"] = _int8(G, K, N, g)
        s["scale_b"] = _scales((G, N), g)
        s["out"] = _empty_out(G, cap, N, dtype)
    else:
        T, G, cap, H = case["tokens"], case["groups"], case["capacity"], case["width"]
        ids, w = _choices(T, case["topk"], G, seed)
        slots, counts = _slots_of(ids, G, cap)
        s["ids"] = torch.from_numpy(ids).cuda()
        s["weights"] = torch.from_numpy(w).cuda()
        if op == "sort":
            s["x"] = _normal((T, H), g, dtype)
            # one row past the experts' rows takes what the plain form drops
            s["buffer"] = torch.zeros((G * cap + 1, H), device="cuda", dtype=dtype)
        else:
            s["slots"] = torch.from_numpy(slots).cuda()
            s["rows"] = _normal((G, cap, H), g, dtype)
        if op == "combine_grad":
            s["dout"] = _normal((T, H), g, dtype)
            s["buffer"] = torch.zeros((G * cap + 1, H), device="cuda", dtype=dtype)
    return s


# ------------------------------------------------------------------ the pass

def _act(v, act):
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * 0.7071067811865476))
    if act == "silu":
        return v * (1.0 / (1.0 + torch.exp(-v)))
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    return v


def _plain_route(ids, groups, capacity):
    flat = ids.reshape(-1).long()
    hot = (flat[:, None] == torch.arange(groups, device=flat.device)[None, :]).to(torch.int32)
    rank = (hot.cumsum(0, dtype=torch.int32) * hot).sum(1, dtype=torch.int32) - 1
    slots = torch.where(rank < capacity, flat.to(torch.int32) * capacity + rank,
                        torch.full_like(rank, -1))
    counts = hot.sum(0, dtype=torch.int32).clamp(max=capacity)
    return slots.reshape(ids.shape), counts


def _plain_quantize(x):
    x = x.float()
    scale = x.abs().amax(dim=-1) / 127.0
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    return torch.round(x / safe[..., None]).clamp(-127, 127), scale


def _run_plain(s):
    op = s["op"]
    if op in ("product", "linear"):
        if op == "product":
            a, sa = s["A"].float(), s["scale_a"]
        else:
            a, sa = _plain_quantize(s["x"])
        v = (a @ s["B"].float()) * sa[:, None] * s["scale_b"][None, :]
        if s["bias_v"] is not None:
            v = v + s["bias_v"][None, :]
        s["out"].copy_(_act(v, s["act"]))
        return s["out"]
    if op == "experts":
        v = torch.bmm(s["A"].float(), s["B"].float()) * s["scale_a"][:, :, None] * s["scale_b"][:, None, :]
        used = torch.arange(s["capacity"], device="cuda")[None, :] < s["counts"][:, None]
        s["out"].copy_(torch.where(used[:, :, None], _act(v, s["act"]), s["out"].float()))
        return s["out"]
    G, cap, H = s["groups"], s["capacity"], s["width"]
    if op == "sort":
        slots, counts = _plain_route(s["ids"], G, cap)
        to = torch.where(slots >= 0, slots, torch.full_like(slots, G * cap)).reshape(-1).long()
        s["buffer"][to] = s["x"].repeat_interleave(s["topk"], dim=0)
        return {"rows": s["buffer"][:-1].view(G, cap, H), "slots": slots, "counts": counts}
    slots = s["slots"].long()
    kept = (slots >= 0).float()
    at = slots.clamp(min=0)
    flat = s["rows"].view(-1, H)
    if op == "sort_grad":
        return (flat[at].float() * kept[:, :, None]).sum(1).to(flat.dtype)
    w = s["weights"] * kept
    if op == "combine":
        return (flat[at].float() * w[:, :, None]).sum(1).to(flat.dtype)
    d = s["dout"].float()
    to = torch.where(slots >= 0, slots, torch.full_like(slots, G * cap)).reshape(-1)
    s["buffer"][to] = (d[:, None, :] * w[:, :, None]).to(flat.dtype).view(-1, H)
    dw = (flat[at].float() * d[:, None, :]).sum(2) * kept
    return {"rows": s["buffer"][:-1].view(G, cap, H), "weights": dw}


def _run_own(s):
    from tiled_staged_matmul_gb300 import binding as lib
    op = s["op"]
    if op == "product":
        return lib.gemm_s8(s["A"], s["B"], s["scale_a"], s["scale_b"], s["out"], bias=s["bias_v"],
                           activation=s["act"])
    if op == "linear":
        q, scale = lib.quantize_rows(s["x"])
        return lib.gemm_s8(q, s["B"], scale, s["scale_b"], s["out"], bias=s["bias_v"],
                           activation=s["act"])
    if op == "experts":
        return lib.grouped_gemm_s8(s["A"], s["B"], s["scale_a"], s["scale_b"], s["counts"], s["out"],
                                   activation=s["act"])
    G, cap, H = s["groups"], s["capacity"], s["width"]
    if op == "sort":
        slots, counts = lib.moe_route(s["ids"], G, cap)
        rows = lib.moe_dispatch(s["x"], slots, G, cap, s["buffer"][:-1].view(G, cap, H))
        return {"rows": rows, "slots": slots, "counts": counts}
    if op == "sort_grad":
        return lib.moe_dispatch_grad(s["rows"], s["slots"])
    if op == "combine":
        return lib.moe_combine(s["rows"], s["slots"], s["weights"])
    rows, dw = lib.moe_combine_grad(s["dout"], s["rows"], s["slots"], s["weights"],
                                    s["buffer"][:-1].view(G, cap, H))
    return {"rows": rows, "weights": dw}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass needs

def _kept(case):
    """Rows that find room, for the router above (one fixed draw)."""
    ids, _ = _choices(case["tokens"], case["topk"], case["groups"], 0)
    _, counts = _slots_of(ids, case["groups"], case["capacity"])
    return int(counts.sum()), int((counts > 0).sum())


def work(case):
    op = case["op"]
    es = _BYTES[case["dtype"]]
    if op in ("product", "linear"):
        M, N, K = case["M"], case["N"], case["K"]
        read = K * N + 4 * N + (4 * N if case["bias"] else 0)
        read += M * K + 4 * M if op == "product" else M * K * es
        return {"bytes": read + M * N * es, "flops": 2 * M * N * K}
    rows, used = _kept(case)
    if op == "experts":
        N, K = case["N"], case["K"]
        return {"bytes": used * (K * N + 4 * N) + rows * (K + 4 + N * es) + 4 * case["groups"],
                "flops": 2 * rows * N * K}
    T, k, H = case["tokens"], case["topk"], case["width"]
    if op == "sort":
        return {"bytes": (T + rows) * H * es + 8 * T * k + 4 * case["groups"], "flops": 0}
    if op == "sort_grad":
        return {"bytes": (T + rows) * H * es + 4 * T * k, "flops": rows * H}
    if op == "combine":
        return {"bytes": (T + rows) * H * es + 8 * T * k, "flops": 2 * rows * H}
    return {"bytes": (T + 2 * rows) * H * es + 12 * T * k, "flops": 3 * rows * H}


# ------------------------------------------------------------------ in 64 bits

def _act64(v, act):
    if act == "gelu":
        return v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "relu":
        return v.clamp(min=0)
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("product", "linear"):
        if op == "product":
            a, sa = s["A"].double(), s["scale_a"].double()
        else:
            # the scale is an f32 value by definition, and so are the codes' quotients
            sa = (s["x"].float().abs().max(dim=1).values / 127.0).double()
            q = (s["x"].float() / sa.float()[:, None]).double()
            a = torch.round(q).clamp(-127, 127)
        out = torch.empty((case["M"], case["N"]), device="cuda", dtype=torch.float64)
        step = 2048
        for r in range(0, case["M"], step):
            v = torch.mm(a[r:r + step], s["B"].double())
            v = v * (sa[r:r + step, None] * s["scale_b"].double()[None, :])
            if s["bias_v"] is not None:
                v = v + s["bias_v"].double()
            out[r:r + step] = _act64(v, case["act"])
        return out
    if op == "experts":
        out = torch.zeros((case["groups"], case["capacity"], case["N"]), device="cuda",
                          dtype=torch.float64)
        for e, n in enumerate(s["counts"].tolist()):
            v = torch.mm(s["A"][e, :n].double(), s["B"][e].double())
            out[e, :n] = _act64(v * (s["scale_a"][e, :n, None].double() * s["scale_b"][e].double()),
                                case["act"])
        return out
    ids, w = _choices(case["tokens"], case["topk"], case["groups"], seed)
    slots, counts = _slots_of(ids, case["groups"], case["capacity"])
    G, cap, H, T = case["groups"], case["capacity"], case["width"], case["tokens"]
    at = torch.from_numpy(slots).cuda().long()
    if op == "sort":
        rows = torch.zeros((G * cap, H), device="cuda", dtype=torch.float64)
        for j in range(case["topk"]):
            t = torch.nonzero(at[:, j] >= 0)[:, 0]
            rows[at[t, j]] = s["x"][t].double()
        return {"rows": rows.view(G, cap, H), "slots": None, "counts": None}
    flat = s["rows"].reshape(-1, H)
    if op in ("sort_grad", "combine"):
        out = torch.zeros((T, H), device="cuda", dtype=torch.float64)
        for j in range(case["topk"]):
            t = torch.nonzero(at[:, j] >= 0)[:, 0]
            c = s["weights"][t, j].double()[:, None] if op == "combine" else 1.0
            out[t] += flat[at[t, j]].double() * c
        return out
    rows = torch.zeros((G * cap, H), device="cuda", dtype=torch.float64)
    dw = torch.zeros((T, case["topk"]), device="cuda", dtype=torch.float64)
    for j in range(case["topk"]):
        t = torch.nonzero(at[:, j] >= 0)[:, 0]
        rows[at[t, j]] = s["dout"][t].double() * s["weights"][t, j].double()[:, None]
        dw[t, j] = (s["dout"][t].double() * flat[at[t, j]].double()).sum(1)
    return {"rows": rows.view(G, cap, H), "weights": dw}
