"""The choice of experts and its gradient on the GPU, against their definition
in 64 bits.

Choices are compared for equality.  Weights: the exponentials of f32 arguments
are off by 2 units in the last place (2^-22 relative) and by the argument's own
rounding, 2^-24 |x - max|; a softmax's total adds up at most 1024 of them in a
tree (at most 37 additions in a row), divisions and products round once each.
For logits within D of each other that is below (50 + 2 D) 2^-24 relative, twice
that for a quotient of two such sums.  Gradients are sums of at most 33 such
terms; each term is off by no more than (150 + 4 D) 2^-24 of its magnitude."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ROUNDOFF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}
INF = float("inf")


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    from tiled_staged_matmul_gb300 import binding
    return binding


def scores_of(x, score):
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1 / (1 + np.exp(-x))
        p = np.exp(x - np.max(x))
        return p / p.sum()


def reference(x, topk, score="softmax", bias=None, groups=1, keep=1, best=2, renormalize=False, scale=1.0):
    """(ids, weights) of an f64 array of logits, token by token."""
    T, E = x.shape
    ids, weights = np.full((T, topk), -1), np.zeros((T, topk))
    for t in range(T):
        there = x[t] > -INF
        if bias is not None:
            there &= bias > -INF
        if not (x[t] > -INF).any():
            continue
        s = scores_of(x[t], score)
        c = s if bias is None else s + bias
        # Without a bias the logits' order is the scores' (which may tie where
        # they round alike).
        order = x[t] if bias is None else c
        if keep < groups:
            per = E // groups
            value = np.full(groups, -INF)
            for g in range(groups):
                inside = [e for e in range(g * per, (g + 1) * per) if there[e]]
                inside.sort(key=lambda e: (-order[e], e))
                if inside:
                    value[g] = order[inside[0]] if best == 1 else sum(c[e] for e in inside[:2])
            kept = sorted(range(groups), key=lambda g: (-value[g], g))[:keep]
            there &= np.isin(np.arange(E) // per, kept)
        chosen = sorted(np.flatnonzero(there), key=lambda e: (-order[e], e))[:topk]
        ids[t, :len(chosen)] = chosen
        w = s[chosen]
        if renormalize and len(chosen):
            m = x[t, chosen] if score == "softmax" else np.minimum(x[t, chosen], 0)
            w = np.exp(m - m.max())
            if score == "sigmoid":
                w = w / (1 + np.exp(-np.abs(x[t, chosen])))
            w = w / w.sum()
        weights[t, :len(chosen)] = w * scale
    return ids, weights


def check(b, x, topk, **kw):
    """x: tokens x experts on the CPU, in the type it has; returns the ids."""
    names = {"keep": "keep_groups", "best": "group_best"}
    bias = kw.get("bias")
    lib = {names.get(k, k): v for k, v in kw.items()}
    if bias is not None:
        lib["bias"] = bias.cuda()
    ids, w = b.moe_choose(x.cuda(), topk, **lib)
    ref = dict(kw, bias=None if bias is None else bias.double().numpy())
    xd = x.double().numpy()
    want, ww = reference(xd, topk, **ref)
    got = ids.cpu().numpy()
    assert np.array_equal(got, want), (np.argwhere(got != want)[:5], got[got != want][:5], want[got != want][:5])
    finite = xd[np.isfinite(xd)]
    D = float(finite.max() - finite.min()) if finite.size else 0.0
    err = 2 * (50 + 2 * D) * 2.0 ** -24 * np.abs(ww) + 2.0 ** -126
    assert (np.abs(w.cpu().double().numpy() - ww) <= err).all()
    return ids


SHAPES = [(1, 1, 1), (3, 2, 2), (32, 64, 6), (33, 60, 8), (5, 8, 8), (100, 100, 7), (65, 128, 4), (40, 160, 6),
          (17, 255, 32), (300, 256, 8), (31, 384, 8), (20, 513, 10), (9, 1000, 31), (8, 1024, 32), (2000, 16, 2)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score,biased,renormalize", [("softmax", False, False), ("softmax", False, True),
                                                      ("softmax", True, False), ("sigmoid", False, False),
                                                      ("sigmoid", True, True)])
def test_choice(b, T, E, k, score, biased, renormalize, dtype):
    g = torch.Generator().manual_seed(T * 7 + E)
    x = (2 * torch.randn((T, E), generator=g)).to(TYPES[dtype])
    bias = 0.1 * torch.randn(E, generator=g) if biased else None
    check(b, x, k, score=score, bias=bias, renormalize=renormalize, scale=2.5 if biased else 1.0)


@pytest.mark.parametrize("T,E,k,groups,keep,best", [
    (40, 256, 8, 8, 4, 2), (33, 160, 6, 8, 3, 1), (20, 64, 6, 4, 1, 2), (17, 16, 3, 16, 5, 2), (12, 96, 5, 3, 2, 2),
    (9, 500, 10, 5, 2, 2), (7, 512, 8, 32, 7, 2), (6, 1024, 8, 16, 4, 2), (25, 34, 4, 17, 6, 1), (8, 40, 20, 8, 2, 2),
    (10, 256, 8, 8, 8, 2), (5, 24, 12, 6, 2, 1)])
@pytest.mark.parametrize("score,biased", [("softmax", False), ("softmax", True), ("sigmoid", False), ("sigmoid", True)])
def test_groups(b, T, E, k, groups, keep, best, score, biased):
    """(40, 20 of 8 groups, 2 kept: only 10 are there to choose from.)"""
    g = torch.Generator().manual_seed(E + groups)
    for dtype in TYPES.values():
        x = torch.randn((T, E), generator=g).to(dtype)
        bias = 0.2 * torch.randn(E, generator=g) if biased else None
        check(b, x, k, score=score, bias=bias, groups=groups, keep=keep, best=best, renormalize=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties_go_to_the_lower_number(b, score):
    g = torch.Generator().manual_seed(3)
    x = torch.randint(0, 4, (200, 64), generator=g).float()
    for bias in (None, torch.zeros(64), torch.randint(0, 2, (64,), generator=g).float()):
        check(b, x, 6, score=score, bias=bias)
        check(b, x, 6, score=score, bias=bias, groups=8, keep=3)
        check(b, x.bfloat16(), 32, score=score, bias=bias, groups=4, keep=3, renormalize=True)
    check(b, torch.zeros((5, 256)), 8, score=score, bias=torch.zeros(256), groups=8, keep=4)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_that_f32_cannot_tell_apart(b, score):
    """Logits a unit in the last place apart, and biases that make up for the
    difference of two scores to within an f32 rounding: the choice is that of
    f64."""
    g = torch.Generator().manual_seed(5)
    T, E = 400, 32
    x = 1 + torch.randint(0, 8, (T, E), generator=g).float() * 2.0 ** -23
    check(b, x, 8, score=score)
    check(b, x, 8, score=score, bias=torch.zeros(E))
    check(b, x, 8, score=score, bias=torch.zeros(E), groups=8, keep=3)
    check(b, x, 8, score=score, groups=8, keep=3)
    # One token's scores and biases that nearly sum to 1.
    x = torch.randn((1, E), generator=g)
    s = scores_of(x[0].double().numpy(), score)
    bias = torch.from_numpy((1 - s).astype(np.float32))
    near = x + torch.randint(-2, 3, (T, E), generator=g) * 2.0 ** -24
    check(b, near, 8, score=score, bias=bias)
    check(b, near, 31, score=score, bias=bias)
    check(b, near, 32, score=score, bias=bias)
    check(b, near, 6, score=score, bias=bias, groups=8, keep=4)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_hidden_experts(b, score, dtype):
    g = torch.Generator().manual_seed(7)
    x = torch.randn((60, 48), generator=g)
    x[torch.rand((60, 48), generator=g) < 0.7] = -INF
    x[5], x[59] = -INF, -INF
    x[6, :], x[6, 40] = -INF, 1.0
    x[7, 0] = torch.finfo(TYPES[dtype]).min
    x = x.to(TYPES[dtype])
    bias = torch.randn(48, generator=g)
    bias[::5] = -INF
    for kw in ({}, {"bias": bias}, {"groups": 6, "keep": 2}, {"bias": bias, "groups": 12, "keep": 5},
               {"groups": 8, "keep": 3, "best": 1}):
        for renormalize in (False, True):
            check(b, x, 10, score=score, renormalize=renormalize, **kw)


def test_far_logits(b):
    """Scores that underflow in f32 still have their order and their shares."""
    x = torch.tensor([[-200.0, -300.0, -201.0, -250.0], [500.0, -500.0, 499.0, 90.0], [-90.0, -88.0, -104.0, -1e38]])
    check(b, x, 3, score="sigmoid", renormalize=True)
    check(b, x, 4, score="softmax", renormalize=True)
    check(b, x, 3, score="sigmoid")


def test_what_is_not_a_number(b):
    x = torch.randn((8, 40), generator=torch.Generator().manual_seed(2))
    x[1, 39], x[4, 0] = float("nan"), INF
    for score, bad in (("softmax", [1, 4]), ("sigmoid", [1])):
        ids, w = b.moe_choose(x.cuda(), 5, score=score, groups=4, keep_groups=2)
        for t in range(8):
            if t in bad:
                assert ids[t].tolist() == [0, 1, 2, 3, 4] and torch.isnan(w[t]).all()
            else:
                assert not torch.isnan(w[t]).any()
    assert b.moe_choose(x.cuda(), 1, score="sigmoid")[1][4, 0] == 1
    bias = torch.zeros(40)
    bias[17] = float("nan")
    ids, w = b.moe_choose(x.cuda(), 5, score="sigmoid", bias=bias.cuda())
    assert torch.isnan(w).all() and (ids.cpu() == torch.arange(5)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,keep", [(256, 8, 1, 1), (256, 8, 8, 2), (1000, 20, 1, 1), (300, 30, 3, 1)])
def test_the_largest_lie_together(b, score, E, k, groups, keep):
    """Experts in order of their scores, up and down, with and without a bias: what is
    chosen is a few lanes'."""
    g = torch.Generator().manual_seed(E)
    x = 0.1 * torch.randn((40, E), generator=g)
    slope = torch.linspace(-3, 3, E)
    for by in (slope, slope.flip(0)):
        check(b, x + by, k, score=score, groups=groups, keep=keep, renormalize=True)
        check(b, x + by, k, score=score, bias=by.clone(), groups=groups, keep=keep, renormalize=True)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_rows_of_any_pitch_and_base(b, dtype):
    for E, pitch, offset in ((64, 64, 0), (64, 72, 0), (64, 65, 0), (64, 64, 1), (60, 61, 3), (2, 3, 1), (128, 136, 4)):
        g = torch.Generator().manual_seed(E + pitch)
        buf = torch.full((offset + 20 * pitch,), float("nan"), dtype=TYPES[dtype])
        x = buf[offset:].view(20, pitch)[:, :E]
        x.copy_(torch.randn((20, E), generator=g).to(TYPES[dtype]))
        dev = buf.cuda()[offset:].view(20, pitch)[:, :E]
        k = min(4, E)
        ids, w = b.moe_choose(dev, k)
        want, ww = reference(x.double().numpy(), k)
        assert np.array_equal(ids.cpu().numpy(), want)
        out = torch.full((offset + 20 * pitch + 8,), 41.0, dtype=TYPES[dtype], device="cuda")
        view = out[offset:offset + 20 * pitch].view(20, pitch)[:, :E]
        dw = torch.randn((20, k), generator=g)
        b.moe_choose_grad(dw.cuda(), dev, ids, view)
        check_grad(view, x, want, dw, dtype, "softmax", False, 1.0)
        view.fill_(41.0)
        assert (out == 41.0).all()


# ------------------------------------------------------------------ gradient

def grad_reference(x, ids, dw, score, renormalize, scale):
    """(dlogits, sum of the terms' magnitudes) in f64."""
    T, E = x.shape
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        on = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        if not on:
            continue
        s = scores_of(x[t], score)
        e = ids[t, on]
        d = dw[t, on] * scale
        if renormalize:
            m = x[t, e] if score == "softmax" else np.minimum(x[t, e], 0)
            p = np.exp(m - m.max()) / (1 if score == "softmax" else 1 + np.exp(-np.abs(x[t, e])))
            p = p / p.sum()
            own = p * (1 if score == "softmax" else 1 / (1 + np.exp(x[t, e])))
            np.add.at(out[t], e, own * (d - (d * p).sum()))
            np.add.at(mag[t], e, own * (np.abs(d) + (np.abs(d) * p).sum()))
        elif score == "sigmoid":
            np.add.at(out[t], e, d * s[e] / (1 + np.exp(x[t, e])))
            np.add.at(mag[t], e, np.abs(d) * s[e] / (1 + np.exp(x[t, e])))
        else:
            np.add.at(out[t], e, d * s[e])
            np.add.at(mag[t], e, np.abs(d) * s[e])
            out[t] -= s * (d * s[e]).sum()
            mag[t] += s * (np.abs(d) * s[e]).sum()
    return out, mag


def check_grad(got, x, ids, dw, dtype, score, renormalize, scale):
    xd = x.double().numpy()
    want, mag = grad_reference(xd, ids, dw.double().numpy(), score, renormalize, float(np.float32(scale)))
    finite = xd[np.isfinite(xd)]
    D = float(finite.max() - finite.min()) if finite.size else 0.0
    err = (150 + 4 * D) * 2.0 ** -24 * mag + 2.0 ** -125
    err = err + ROUNDOFF[dtype] * (np.abs(want) + err) + TINY[dtype]
    bad = ~(np.abs(got.cpu().double().numpy() - want) <= err)
    assert not bad.any(), (np.argwhere(bad)[:5], got.cpu().double().numpy()[bad][:5], want[bad][:5])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient(b, T, E, k, score, renormalize, dtype):
    g = torch.Generator().manual_seed(T + E * 3)
    x = (2 * torch.randn((T, E), generator=g)).to(TYPES[dtype])
    ids, _ = b.moe_choose(x.cuda(), k, score=score)
    dw = torch.randn((T, k), generator=g)
    got = b.moe_choose_grad(dw.cuda(), x.cuda(), ids, score=score, renormalize=renormalize, scale=1.5)
    assert got.dtype == TYPES[dtype]
    check_grad(got, x, ids.cpu().numpy(), dw, dtype, score, renormalize, 1.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_of_ids_that_are_not_there_or_twice(b, score, renormalize):
    g = torch.Generator().manual_seed(9)
    x = torch.randn((30, 20), generator=g)
    x[3, :10], x[4] = -INF, -INF
    ids = torch.randint(-2, 23, (30, 6), generator=g)
    ids[:, 5] = ids[:, 0]
    ids[3] = torch.tensor([12, 13, -1, -1, 19, 12])
    ids[4] = -1
    ids[5] = -1
    ids = ids.int()
    dw = torch.randn((30, 6), generator=g)
    dw[ids < 0] = float("nan")
    dw[ids >= 20] = float("nan")
    got = b.moe_choose_grad(dw.cuda(), x.cuda(), ids.cuda(), score=score, renormalize=renormalize)
    check_grad(got, x, ids.numpy(), torch.nan_to_num(dw), "f32", score, renormalize, 1.0)
    assert (got[4] == 0).all() and (got[5] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_against_differences(b, score, renormalize):
    """Of the loss sum dw . w, w by the definition in f64, ids held fixed: central
    differences with a step of 2^-10 are off by a sixth of its square times the
    third derivative (at most 4 sum |dw|: a weight's derivatives are products of
    numbers below 1)."""
    g = torch.Generator().manual_seed(11)
    T, E, k = 6, 12, 4
    x = torch.randn((T, E), generator=g)
    ids, _ = b.moe_choose(x.cuda(), k, score=score)
    dw = torch.randn((T, k), generator=g)
    got = b.moe_choose_grad(dw.cuda(), x.cuda(), ids, score=score, renormalize=renormalize, scale=1.0).cpu().double()
    at = ids.cpu().long()

    def loss(v):
        p = torch.softmax(v, 1) if score == "softmax" else torch.sigmoid(v)
        w = p.gather(1, at)
        return ((w / w.sum(1, keepdim=True) if renormalize else w) * dw.double()).sum(1)

    h = 2.0 ** -10
    limit = (h * h * dw.double().abs().sum(1) + 2.0 ** -20 * dw.double().abs().sum(1))[:, None]
    for e in range(E):
        step = torch.zeros((T, E), dtype=torch.float64)
        step[:, e] = h
        d = (loss(x.double() + step) - loss(x.double() - step)) / (2 * h)
        assert ((got[:, e] - d).abs() <= limit[:, 0]).all()


def test_streams_and_graphs(b):
    x = torch.randn((3000, 64), generator=torch.Generator().manual_seed(1))
    y = torch.randn((3000, 64), generator=torch.Generator().manual_seed(2))
    dev = x.cuda()
    want, ww = b.moe_choose(dev, 6)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        ids, w = b.moe_choose(dev, 6, stream=side)
        d = b.moe_choose_grad(w, dev, ids, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(ids, want) and torch.equal(w, ww)
    assert torch.equal(d, b.moe_choose_grad(ww, dev, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, w = b.moe_choose(dev, 6)
        d = b.moe_choose_grad(w, dev, ids)
    for v in (x, y, x):
        dev.copy_(v)
        graph.replay()
        i2, w2 = b.moe_choose(v.cuda(), 6)
        assert torch.equal(ids, i2) and torch.equal(w, w2) and torch.equal(d, b.moe_choose_grad(w2, dev, i2))


def test_no_tokens_and_no_choices(b):
    ids, w = b.moe_choose(torch.zeros((0, 8), device="cuda"), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    ids, w = b.moe_choose(torch.zeros((5, 8), device="cuda"), 0)
    d = b.moe_choose_grad(w, torch.ones((5, 8), device="cuda"), ids)
    assert ids.shape == (5, 0) and (d == 0).all()
