"""Measured cases of the choice of experts and of the microscaled 4-bit products.

Each case is one call (or one short chain of calls) that a layer makes:

* ``choose``      -- router logits -> each token's experts and their weights
* ``choose_grad`` -- the weights' gradient -> the logits' gradient
* ``product``     -- 4-bit floating point x 4-bit, a scale for every block of 16 or 32
* ``linear``      -- activations quantised to 4 bits, then the product
* ``experts``     -- the product of every expert with its own rows

A 4-bit operand is rows of codes along the product's inner dimension, two to a
byte (the even one in the low half), with an 8-bit scale per block.  Blocks of
16 have e4m3 scales and an f32 scale per row, blocks of 32 have powers of two
(e8m0) and no other.  The scales are kept 128 rows x 4 blocks at a time, 512
bytes each: byte 16 * (row % 32) + 4 * (row / 32) + block % 4.

``run`` computes a case in plain torch operations in 32 bits (experts are
chosen in 64: two scores may differ by less than 32 bits hold), or, with
``own``, through the library's entry points.  ``exact`` gives the result in 64
bits.  Inputs are drawn from the seed alone.
"""
import math

import numpy as np
import torch

own = False

_DEVICE = "cuda"
_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"f16": 2, "bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def _choose(op, tokens, experts, topk, dtype, score, renormalize, bias=False, groups=1, keep=1, best=2, scale=1.0,
            name=None):
    case = {"op": op, "tokens": tokens, "experts": experts, "topk": topk, "dtype": dtype, "score": score,
            "renormalize": renormalize, "bias": bias, "groups": groups, "keep": keep, "best": best, "scale": scale}
    if name:
        case["name"] = name
    return case


def _product(op, M, N, K, block, dtype, act="none", bias=False, name=None):
    case = {"op": op, "M": M, "N": N, "K": K, "block": block, "dtype": dtype, "act": act, "bias": bias}
    if name:
        case["name"] = name
    return case


def _experts(tokens, topk, groups, capacity, N, K, block, dtype, act, name=None):
    case = {"op": "experts", "tokens": tokens, "topk": topk, "groups": groups, "capacity": capacity,
            "N": N, "K": K, "block": block, "dtype": dtype, "act": act}
    if name:
        case["name"] = name
    return case


def listed():
    return [
        # one decode step of 32 sequences before 64 experts: the smallest call, latency
        _choose("choose", 32, 64, 6, "f32", "softmax", True, name="choose_decode"),
        # a long prompt before 256 experts in eight groups, balanced by a bias: the largest choice
        _choose("choose", 8192, 256, 8, "f32", "sigmoid", True, True, 8, 4, 2, 2.5, name="choose_prompt"),
        # a training step of an odd number of tokens, 16-bit logits, weights not renormalised
        _choose("choose", 4095, 64, 6, "bf16", "softmax", False, name="choose_train"),
        # the gradient of that step's weights: the whole row's softmax takes part
        _choose("choose_grad", 4095, 64, 6, "bf16", "softmax", False, name="choose_grad_train"),
        # the gradient at the largest choice
        _choose("choose_grad", 8192, 256, 8, "f32", "sigmoid", True, True, 8, 4, 2, 2.5, name="choose_grad_long"),
        # one token through a square projection: the smallest product, latency
        _product("product", 1, 4096, 4096, 16, "f16", name="product_token"),
        # a batch of decoded tokens, every size ragged, with bias and activation
        _product("product", 97, 14333, 4010, 32, "bf16", "gelu", True, name="product_batch"),
        # a projection in a decode step of 16 sequences, activations quantised on the way
        _product("linear", 16, 14336, 4096, 16, "f16", name="linear_decode"),
        # the same over a long prompt with an odd number of tokens: the largest product
        _product("linear", 8191, 8192, 8192, 16, "bf16", name="linear_prompt"),
        # a chunk of a prompt, blocks of 32
        _product("linear", 512, 14336, 4096, 32, "bf16", "silu", name="linear_chunk"),
        # a decode step of 32 sequences through 64 experts
        _experts(32, 6, 64, 32, 1408, 2048, 32, "f16", "silu", "experts_decode"),
        # a prompt through the same experts, as the grouped product's 64-expert layout
        _experts(4096, 6, 64, 512, 1408, 2048, 16, "f16", "silu", "experts_prompt"),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    """One more case: tokens from 1 to 8192, widths and depths from a few
    hundred to 8192 with ragged ones among them, 4 to 256 experts."""
    op = rng.choice(["choose", "choose", "choose_grad", "choose_grad", "product", "product", "linear", "linear",
                     "experts", "experts"])
    if op in ("choose", "choose_grad"):
        groups = rng.choice([1, 1, 1, 2, 4, 8])
        experts = groups * _log(rng, max(1, 8 // groups), 256 // groups)
        keep = rng.randint(max(1, groups // 2), groups)
        score = rng.choice(["softmax", "sigmoid"])
        renormalize = rng.random() < 0.5
        # (the one weight of a single choice, renormalised, has no gradient)
        topk = rng.randint(1 + renormalize, min(8, keep * (experts // groups)))
        return _choose(op, _log(rng, 1, 8192), experts, topk, rng.choice(["f16", "bf16", "f32"]), score,
                       renormalize, rng.random() < 0.5, groups, keep, rng.choice([1, 2]), rng.choice([1.0, 2.5]))
    block = rng.choice([16, 32])
    if op in ("product", "linear"):
        M = _log(rng, 1, 8192)
        K = 2 * _log(rng, 128, 4096)
        N = _log(rng, 256, 8192)
        if rng.random() < 0.5:
            N = max(16, N // 16 * 16)
        if rng.random() < 0.5:
            K = K // 64 * 64
        act = rng.choice(["none", "none", "gelu", "silu", "relu"])
        return _product(op, M, N, K, block, rng.choice(["f16", "bf16"]), act, rng.random() < 0.5)
    groups = _log(rng, 4, 64)
    topk = rng.randint(1, min(6, groups))
    tokens = _log(rng, 1, 4096)
    fair = tokens * topk / groups
    capacity = max(1, min(tokens, int(fair * rng.uniform(1.0, 2.0)) + 8, 512))
    return _experts(tokens, topk, groups, capacity, _log(rng, 256, 2048), 2 * _log(rng, 128, 1024), block,
                    rng.choice(["f16", "bf16"]), rng.choice(["none", "silu", "gelu"]))


# ------------------------------------------------------------------ 4-bit operands

# The magnitudes of the eight codes, and the midpoints between them.
_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
_MIDDLES = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)


def _power(e):
    """2 ** e for whole e, exactly (an f64 of that exponent)."""
    return ((e.long() + 1023) << 52).view(torch.float64).float()


def _codes_of(v):
    """Codes 0 ... 15 nearest to v; a middle goes to the even code."""
    a = v.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for i, m in enumerate(_MIDDLES):
        code += (a > m) if i % 2 == 0 else (a >= m)
    return code + 8 * (v < 0).to(torch.uint8)


def _blocks(x, block):
    """Rows cut into blocks, the last one filled with zeros."""
    pad = -x.shape[-1] % block
    if pad:
        x = torch.cat([x, x.new_zeros((*x.shape[:-1], pad))], dim=-1)
    return x.reshape(*x.shape[:-1], -1, block)


def _plain_quantize(x, block):
    """(codes, block scales as values, row scales) of rows x."""
    b = _blocks(x.float(), block)
    top = b.abs().amax(dim=-1)
    if block == 32:
        # the largest power of two in the block over 4, the largest one a code holds
        e = torch.frexp(top).exponent - 3
        s = _power(torch.where(top > 0, e, torch.full_like(e, -127)).clamp(min=-127))
        return _codes_of(b / s[..., None]), s, None
    most = top.amax(dim=-1)
    # the smallest power of two that lets 6 * 448 of it reach the row's largest
    part, e = torch.frexp(most)
    e = torch.where(part <= 0.65625, e - 12, e - 11).clamp(min=-126)
    r = torch.where(most > 0, _power(e), torch.zeros_like(most))
    inv = torch.where(most > 0, _power(-e), torch.zeros_like(most))
    t = top * inv[..., None] / torch.full_like(top, 6.0)  # (by a number it would be a product)
    # to e4m3: four significant bits, the smallest step 2 ** -9
    step = _power((torch.frexp(t).exponent - 4).clamp(min=-9))
    s = torch.round(t / step) * step
    safe = torch.where(s > 0, s, torch.ones_like(s))
    v = torch.where((s > 0)[..., None], b * inv[..., None, None] / safe[..., None], torch.zeros_like(b))
    return _codes_of(v), s, r


def _pack(codes, s, K):
    """Codes two to a byte (16-byte pitch), scales in 512-byte tiles."""
    flat = codes.reshape(*codes.shape[:-2], -1)[..., :K + K % 2]
    bytes_ = flat[..., 0::2] | (flat[..., 1::2] << 4)
    pitch = -(-bytes_.shape[-1] // 16) * 16
    held = bytes_.new_zeros((*bytes_.shape[:-1], pitch))
    held[..., :bytes_.shape[-1]] = bytes_
    if codes.shape[-1] == 16:
        raw = s.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        raw = (torch.frexp(s).exponent + 126).to(torch.uint8)
    *lead, rows, blocks = raw.shape
    R, B = -(-rows // 128), -(-blocks // 4)
    full = raw.new_zeros((*lead, R * 128, B * 4))
    full[..., :rows, :blocks] = raw
    n = len(lead)
    tiles = full.view(*lead, R, 4, 32, B, 4).permute(*range(n), n, n + 3, n + 2, n + 1, n + 4)
    return held[..., :bytes_.shape[-1]], tiles.reshape(*lead, R, B, 512).contiguous()


def _plain_values(codes, tiles, row_scales, block):
    """The numbers that an operand stands for, f32 (with the row scales)."""
    *lead, rows, width = codes.shape
    low = (codes & 15).long()
    high = (codes >> 4).long()
    table = torch.tensor(_VALUES + tuple(-v for v in _VALUES), device=codes.device)
    v = torch.stack([table[low], table[high]], dim=-1).reshape(*lead, rows, 2 * width)
    n = len(lead)
    R, B = tiles.shape[n], tiles.shape[n + 1]
    raw = tiles.view(*lead, R, B, 32, 4, 4).permute(*range(n), n, n + 3, n + 2, n + 1, n + 4)
    raw = raw.reshape(*lead, R * 128, B * 4)[..., :rows, :].contiguous()
    s = raw.view(torch.float8_e4m3fn).float() if block == 16 else _power(raw.int() - 127)
    v = v * s.repeat_interleave(block, dim=-1)[..., :2 * width]
    return v if row_scales is None else v * row_scales[..., None]


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device=_DEVICE).manual_seed(seed * 7919 + 29)


def _normal(shape, g):
    return torch.randn(shape, generator=g, device=_DEVICE, dtype=torch.float32)


def _operand(shape, block, g):
    """A 4-bit operand of values with a spread of row magnitudes, as a program keeps it."""
    x = _normal(shape, g) * torch.exp(0.5 * _normal((*shape[:-1], 1), g)) * 0.02
    codes, s, r = _plain_quantize(x, block)
    return (*_pack(codes, s, shape[-1]), r)


def _counts(tokens, topk, groups, capacity, seed):
    """Rows of each expert, for a router whose busiest expert gets about three
    times what its least busy one gets."""
    g = np.random.default_rng(seed)
    z = np.linspace(0.55, -0.55, groups)[None, :] + g.gumbel(size=(tokens, groups))
    ids = np.argsort(-z, axis=1)[:, :topk]
    return np.minimum(np.bincount(ids.reshape(-1), minlength=groups), capacity).astype(np.int32)


def _empty_out(shape, dtype):
    *lead, cols = shape
    return torch.zeros((*lead, -(-cols // 8) * 8), device=_DEVICE, dtype=dtype)[..., :cols]


def prepare(case, seed):
    op = case["op"]
    dtype = _TYPES[case["dtype"]]
    g = _generator(seed)
    s = dict(case)
    if op in ("choose", "choose_grad"):
        T, E = case["tokens"], case["experts"]
        # logits with favourite experts; a balance bias of the size of the scores' differences
        s["logits"] = (1.5 * _normal((T, E), g) + 0.5 * _normal((1, E), g)).to(dtype)
        s["bias_v"] = 0.05 * _normal((E,), g) if case["bias"] else None
        if op == "choose_grad":
            s["ids"], _ = _plain_choose(s)
            s["dweights"] = _normal((T, case["topk"]), g)
        return s
    N, K, block = case["N"], case["K"], case["block"]
    if op == "experts":
        G, cap = case["groups"], case["capacity"]
        s["counts"] = torch.from_numpy(_counts(case["tokens"], case["topk"], G, cap, seed)).to(_DEVICE)
        s["A"] = _operand((G, cap, K), block, g)
        s["B"] = _operand((G, N, K), block, g)
        s["out"] = _empty_out((G, cap, N), dtype)
        return s
    M = case["M"]
    if op == "product":
        s["A"] = _operand((M, K), block, g)
    else:
        # activations with a spread of row magnitudes and a few large channels
        x = _normal((M, K), g) * torch.exp(_normal((M, 1), g))
        x[:, ::97] *= 6.0
        s["x"] = x.to(dtype)
    s["B"] = _operand((N, K), block, g)
    s["bias_v"] = _normal((N,), g) if case["bias"] else None
    s["out"] = _empty_out((M, N), dtype)
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


def _plain_scores(s):
    x = s["logits"].double()
    if s["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    p = torch.exp(x - x.amax(dim=1, keepdim=True))
    return p / p.sum(dim=1, keepdim=True)


def _first_largest(c):
    """The lowest index of each row's largest value."""
    n = c.shape[1]
    at = torch.arange(n, device=c.device)
    return torch.where(c == c.amax(dim=1, keepdim=True), at[None, :], n).amin(dim=1)


def _plain_choose(s):
    E, groups = s["experts"], s["groups"]
    p = _plain_scores(s)
    c = p if s["bias_v"] is None else p + s["bias_v"].double()[None, :]
    if groups > 1:
        per = E // groups
        left = c.view(-1, per).clone()
        value = torch.zeros_like(left[:, 0])
        for _ in range(min(s["best"], per)):
            value = value + left.amax(dim=1)
            left.scatter_(1, _first_largest(left)[:, None], -math.inf)
        value = value.view(-1, groups)
        kept = torch.zeros_like(value, dtype=torch.bool)
        for _ in range(s["keep"]):
            at = _first_largest(value)[:, None]
            kept.scatter_(1, at, True)
            value.scatter_(1, at, -math.inf)
        c = torch.where(kept.repeat_interleave(per, dim=1), c, -math.inf)
    else:
        c = c.clone()
    ids = []
    for _ in range(s["topk"]):
        at = _first_largest(c)
        ids.append(at)
        c.scatter_(1, at[:, None], -math.inf)
    ids = torch.stack(ids, dim=1)
    w = torch.gather(p, 1, ids)
    if s["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    return ids.int(), (w * s["scale"]).float()


def _plain_choose_grad(s):
    ids = s["ids"].long()
    p = _plain_scores(s).float()
    w = torch.gather(p, 1, ids)
    dw = s["dweights"] * s["scale"]
    if s["renormalize"]:
        total = w.sum(dim=1, keepdim=True)
        dw = (dw - (dw * w).sum(dim=1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter_(1, ids, dw)
    if s["score"] == "sigmoid":
        d = dp * p * (1.0 - p)
    else:
        d = p * (dp - (dp * p).sum(dim=1, keepdim=True))
    return d.to(s["logits"].dtype)


def _run_plain(s):
    op = s["op"]
    if op == "choose":
        ids, w = _plain_choose(s)
        return {"ids": ids, "weights": w}
    if op == "choose_grad":
        return _plain_choose_grad(s)
    block = s["block"]
    b = _plain_values(*s["B"], block)
    if op == "experts":
        v = _act(torch.bmm(_plain_values(*s["A"], block), b.transpose(1, 2)), s["act"])
        used = torch.arange(s["capacity"], device=v.device)[None, :] < s["counts"][:, None]
        s["out"].copy_(torch.where(used[:, :, None], v, s["out"].float()))
        return s["out"]
    if op == "product":
        a = _plain_values(*s["A"], block)
    else:
        codes, scales, rows = _plain_quantize(s["x"], block)
        table = torch.tensor(_VALUES + tuple(-v for v in _VALUES), device=codes.device)
        a = (table[codes.long()] * scales[..., None]).flatten(-2)[:, :s["K"]]
        a = a if rows is None else a * rows[:, None]
    v = a @ b[:, :s["K"]].T
    if s["bias_v"] is not None:
        v = v + s["bias_v"][None, :]
    s["out"].copy_(_act(v, s["act"]))
    return s["out"]


def _run_own(s):
    from tiled_staged_matmul_gb300 import binding as lib
    op = s["op"]
    if op == "choose":
        ids, w = lib.moe_choose(s["logits"], s["topk"], score=s["score"], bias=s["bias_v"], groups=s["groups"],
                                keep_groups=s["keep"], group_best=s["best"], renormalize=s["renormalize"],
                                scale=s["scale"])
        return {"ids": ids, "weights": w}
    if op == "choose_grad":
        return lib.moe_choose_grad(s["dweights"], s["logits"], s["ids"], score=s["score"],
                                   renormalize=s["renormalize"], scale=s["scale"])
    block = s["block"]
    b = lib.Fp4Rows(*s["B"], block)
    if op == "experts":
        return lib.grouped_gemm_fp4(lib.Fp4Rows(*s["A"], block), b, s["counts"], s["out"], activation=s["act"])
    a = lib.Fp4Rows(*s["A"], block) if op == "product" else lib.quantize_fp4(s["x"], block=block)
    return lib.gemm_fp4(a, b, s["out"], bias=s["bias_v"], activation=s["act"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ what a pass needs

def _operand_bytes(rows, K, block):
    return rows * (-(-K // 2) + -(-K // block) + (4 if block == 16 else 0))


def work(case):
    op = case["op"]
    es = _BYTES[case["dtype"]]
    if op in ("choose", "choose_grad"):
        T, E, k = case["tokens"], case["experts"], case["topk"]
        if op == "choose":
            return {"bytes": T * E * es + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 4 * T * E}
        # (only the chosen logits matter to sigmoids and to renormalised weights)
        whole = case["score"] == "softmax" and not case["renormalize"]
        return {"bytes": T * E * es + (T * E if whole else T * k) * es + 8 * T * k,
                "flops": 4 * T * (E if whole else k)}
    N, K, block = case["N"], case["K"], case["block"]
    if op == "experts":
        counts = _counts(case["tokens"], case["topk"], case["groups"], case["capacity"], 0)
        rows, used = int(counts.sum()), int((counts > 0).sum())
        return {"bytes": used * _operand_bytes(N, K, block) + _operand_bytes(rows, K, block) + rows * N * es +
                4 * case["groups"], "flops": 2 * rows * N * K}
    M = case["M"]
    read = _operand_bytes(N, K, block) + (4 * N if case["bias"] else 0)
    read += _operand_bytes(M, K, block) if op == "product" else M * K * es
    return {"bytes": read + M * N * es, "flops": 2 * M * N * K}


# ------------------------------------------------------------------ in 64 bits

def _act64(v, act):
    if act == "gelu":
        return v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
    if act == "silu":
        return v * torch.sigmoid(v)
    if act == "relu":
        return v.clamp(min=0)
    return v


def _nearest64(v, grid):
    """The nearest value of an ascending grid that starts at 0, ties to the even place."""
    g = torch.tensor(grid, device=v.device, dtype=torch.float64)
    a = v.abs().clamp(max=grid[-1]).contiguous()
    hi = torch.searchsorted(g, a).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = g[hi] - a, a - g[lo]
    at = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return torch.copysign(g[at], v)


def _quantized64(x, block):
    """What rows x become, as values."""
    M, K = x.shape
    b = _blocks(x.double(), block)
    top = b.abs().amax(dim=2)
    if block == 32:
        # (an f64 without its fraction is the power of two in it)
        s = (top.clamp(min=2.0 ** -125).view(torch.int64) >> 52 << 52).view(torch.float64) / 4.0
        r = torch.ones(M, device=x.device, dtype=torch.float64)
    else:
        e4m3 = [m * 2.0 ** -9 for m in range(8)]
        e4m3 += [(8 + m) * 2.0 ** (e - 3) for e in range(-6, 9) for m in range(8) if (e, m) != (8, 7)]
        most = top.amax(dim=1).clamp(min=2.0 ** -113)
        r = (most.view(torch.int64) >> 52 << 52).view(torch.float64) / 2048.0
        r = torch.where(r * 1344.0 < most, torch.where(r * 2688.0 < most, 2.0 * r, r), r / 2.0)
        s = _nearest64(top / (6.0 * r[:, None]), e4m3)
    scale = (s * r[:, None])[:, :, None]
    v = _nearest64(torch.where(scale > 0, b / torch.where(scale > 0, scale, 1.0), 0.0), list(_VALUES)) * scale
    return v.reshape(M, -1)[:, :K]


def _values64(codes, tiles, row_scales, block):
    return _plain_values(codes, tiles, None, block).double() * (
        1.0 if row_scales is None else row_scales.double()[..., None])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("choose", "choose_grad"):
        x = s["logits"].double()
        p = torch.softmax(x, dim=1) if case["score"] == "softmax" else torch.sigmoid(x)
        if op == "choose":
            c = p + (0.0 if s["bias_v"] is None else s["bias_v"].double())
            if case["groups"] > 1:
                by = c.view(case["tokens"], case["groups"], -1)
                value = by.sort(dim=2, descending=True).values[:, :, :case["best"]].sum(2)
                order = value.sort(dim=1, descending=True, stable=True).indices[:, :case["keep"]]
                off = torch.full_like(value, -math.inf).scatter(1, order, 0.0)
                c = (by + off[:, :, None]).reshape(c.shape)
            ids = c.sort(dim=1, descending=True, stable=True).indices[:, :case["topk"]]
            w = p.gather(1, ids)
            if case["renormalize"]:
                w = w / w.sum(1, keepdim=True)
            return {"ids": ids.int(), "weights": w * case["scale"]}
        x = x.requires_grad_(True)
        with torch.enable_grad():
            q = torch.softmax(x, dim=1) if case["score"] == "softmax" else torch.sigmoid(x)
            w = q.gather(1, s["ids"].long())
            if case["renormalize"]:
                w = w / w.sum(1, keepdim=True)
            return torch.autograd.grad((w * case["scale"] * s["dweights"].double()).sum(), x)[0]
    b = _values64(*s["B"], case["block"])
    if op == "experts":
        a = _values64(*s["A"], case["block"])
        out = torch.zeros((case["groups"], case["capacity"], case["N"]), device=a.device, dtype=torch.float64)
        for e, n in enumerate(s["counts"].tolist()):
            out[e, :n] = _act64(torch.mm(a[e, :n], b[e].T), case["act"])
        return out
    a = _values64(*s["A"], case["block"]) if op == "product" else _quantized64(s["x"], case["block"])
    out = torch.empty((case["M"], case["N"]), device=a.device, dtype=torch.float64)
    step = 2048
    for i in range(0, case["M"], step):
        v = torch.mm(a[i:i + step, :case["K"]], b[:, :case["K"]].T)
        if s["bias_v"] is not None:
            v = v + s["bias_v"].double()
        out[i:i + step] = _act64(v, case["act"])
    return out
