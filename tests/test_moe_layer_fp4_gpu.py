"""The example's layer with its router and its 4-bit form: the calls together, as
a program makes them.

A value that rounds the other way changes a 4-bit code by a whole step, so each
stage is checked against 64 bits from the stage's own inputs, and the layer's
result is the stages' one after another, bit for bit.  Sums of products: n / 16
+ 2 additions of 2^-23 of their terms' magnitudes for 4-bit products, (n + 4)
2^-24 for f16 ones; f16 outputs round by 2^-11 (half the smallest subnormal,
2^-25); silu has a slope below 1.1 and is computed within 2^-20 of its value."""
import numpy as np
import pytest
import torch

import fp4_util as fp4
import test_choose_gpu as choice

pytestmark = pytest.mark.gpu

U16, U32, TINY = 2.0 ** -11, 2.0 ** -24, 2.0 ** -25


@pytest.fixture(scope="module")
def tsm():
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    from tiled_staged_matmul_gb300 import binding
    return binding


def make(tokens, groups, width, hidden, capacity, seed):
    from examples.moe_layer import MoELayer
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g)
    # (A router with rows of a multiple of 16 bytes: the f16 product's copy of
    # another cannot be captured into a graph.)
    router = torch.zeros((width, -(-groups // 8) * 8), dtype=torch.float16, device="cuda")[:, :groups]
    layer = MoELayer((rand(groups, width, hidden) * width ** -0.5).half().cuda(),
                     (rand(groups, hidden, width) * hidden ** -0.5).half().cuda(), capacity,
                     router.copy_((rand(width, groups) * width ** -0.5).half()))
    return layer, rand(tokens, width).half().cuda()


def values_of(rows, e, n, K):
    """Expert e's first n rows of a 3-D operand as f64 values."""
    one = fp4.unpacked(type(rows)(rows.codes[e, :n], rows.block_scales[e], None, rows.block), K)
    return fp4.values(one[0][:, :K].astype(np.int64), one[1][:, :-(-K // rows.block)].astype(np.int64),
                      None if rows.scales is None else rows.scales[e, :n].cpu().numpy(), rows.block)


def check_stage(rows, weights, out, counts, K, act):
    for e, n in enumerate(counts):
        a, w = values_of(rows, e, n, K), values_of(weights, e, weights.codes.shape[1], K)
        v, err = a @ w.T, (K / 16 + 2) * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T)
        err = err + 4 * U32 * np.abs(v)
        if act:
            s = v / (1 + np.exp(-v))
            v, err = s, 1.1 * err + 2.0 ** -20 * np.abs(s)
        err = err + U16 * (np.abs(v) + err) + TINY
        got = out[e, :n].cpu().double().numpy()
        assert (np.abs(got - v) <= err).all(), e


def check_rows(rows, x, counts, K):
    """The operand is x's first rows, quantised."""
    for e, n in enumerate(counts):
        if n:
            codes, bytes_, scales = fp4.quantised(x[e, :n].cpu().double().numpy(), rows.block)
            want = fp4.values(codes.astype(np.int64), bytes_.astype(np.int64), scales, rows.block)
            assert np.array_equal(values_of(rows, e, n, K), want), e


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("tokens,topk,groups,capacity,width,hidden", [
    (1, 2, 4, 4, 64, 96), (37, 2, 4, 24, 136, 72), (200, 3, 8, 64, 256, 192), (600, 2, 4, 300, 128, 200)])
def test_router_and_4_bit_serving(tsm, tokens, topk, groups, capacity, width, hidden, block):
    layer, x = make(tokens, groups, width, hidden, capacity, tokens)
    layer.quantise_fp4(block)
    ids, weights, (_, logits, _) = layer.choose(x, topk)
    want, ww = choice.reference(logits.cpu().double().numpy(), topk, renormalize=True)
    assert np.array_equal(ids.cpu().numpy(), want)
    assert np.abs(weights.cpu().double().numpy() - ww).max() <= 2.0 ** -17

    out = layer.serve_fp4(x, ids, weights)

    slots, counts = tsm.moe_route(ids, groups, capacity)
    rows = tsm.moe_dispatch(x, slots, groups, capacity)
    n = counts.tolist()
    q = tsm.quantize_fp4(rows, counts, block=block)
    check_rows(q, rows, n, width)
    check_rows(layer.f1, layer.W1.transpose(1, 2), [hidden] * groups, width)
    check_rows(layer.f2, layer.W2.transpose(1, 2), [width] * groups, hidden)
    a = tsm.grouped_gemm_fp4(q, layer.f1, counts, activation="silu", out_dtype=torch.float16)
    check_stage(q, layer.f1, a, n, width, True)
    qa = tsm.quantize_fp4(a, counts, block=block)
    check_rows(qa, a, n, hidden)
    y = tsm.grouped_gemm_fp4(qa, layer.f2, counts, out_dtype=torch.float16)
    check_stage(qa, layer.f2, y, n, hidden, False)
    tsm.check(tsm.gemm_get_device_status(0))
    assert torch.equal(out, tsm.moe_combine(y, slots, weights))

    # The same in a graph, replayed on other tokens: padded ones among them.
    x2 = torch.randn((tokens, width), generator=torch.Generator().manual_seed(5)).half().cuda()
    still = x.clone()
    layer.serve_fp4(still, ids, weights)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        i, w, _ = layer.choose(still, topk)
        served = layer.serve_fp4(still, i, w)
    for v in (x2, x):
        still.copy_(v)
        graph.replay()
        i2, w2, _ = layer.choose(v, topk)
        assert torch.equal(i, i2) and torch.equal(w, w2)
        assert torch.equal(served, layer.serve_fp4(v, i2, w2))


def test_router_step(tsm):
    """Choice, layer and back: the gradients by way of the weights."""
    tokens, topk, groups, width, hidden, capacity = 60, 3, 8, 96, 72, 40
    layer, x = make(tokens, groups, width, hidden, capacity, 3)
    ids, weights, chosen = layer.choose(x, topk)
    out, saved = layer.forward(x, ids, weights)
    dout = torch.randn((tokens, width), generator=torch.Generator().manual_seed(4)).half().cuda()
    dweights = layer.backward(dout, saved)[1]
    dx, drouter = layer.choose_backward(dweights, chosen)
    logits = chosen[1].cpu().double().numpy()
    d, mag = choice.grad_reference(logits, ids.cpu().numpy(), dweights.cpu().double().numpy(), "softmax", True, 1.0)
    D = float(logits.max() - logits.min())
    e = (150 + 4 * D) * U32 * mag + U32 * np.abs(d)
    e = e + U16 * (np.abs(d) + e) + TINY  # (dlogits as f16, for the products)
    R, X = layer.router.cpu().double().numpy(), x.cpu().double().numpy()
    for got, v, err, n in ((dx, d @ R.T, e @ np.abs(R).T + (groups + 4) * U32 * (np.abs(d) + e) @ np.abs(R).T, groups),
                           (drouter, X.T @ d, np.abs(X).T @ e + (tokens + 4) * U32 * np.abs(X).T @ (np.abs(d) + e), tokens)):
        if got.dtype == torch.float16:
            err = err + U16 * (np.abs(v) + err) + TINY
        assert (np.abs(got.cpu().double().numpy() - v) <= err).all()
    # Differences of the loss dweights . weights in 64 bits, along one direction of
    # x and of the router.
    g = torch.Generator().manual_seed(6)
    sx, sr = (torch.randn(v.shape, generator=g).double().numpy() for v in (x, layer.router))
    at, dw = ids.cpu().long().numpy(), dweights.cpu().double().numpy()

    def loss(s):
        z = (X + s * sx) @ (R + s * sr)
        w = np.exp(np.take_along_axis(z, at, 1))
        return float((w / w.sum(1, keepdims=True) * dw).sum())

    # (The formula, at the logits in 64 bits: those of the library are f32.)
    dz, _ = choice.grad_reference(X @ R, at, dw, "softmax", True, 1.0)
    along = float((dz @ R.T * sx).sum() + (X.T @ dz * sr).sum())
    h = 1e-5
    assert abs((loss(h) - loss(-h)) / (2 * h) - along) <= 1e-6 * float(np.abs(dz @ R.T * sx).sum() + np.abs(X.T @ dz * sr).sum())


def test_the_example_runs(tsm, capsys):
    from examples import moe_layer
    moe_layer.main()
    assert capsys.readouterr().out.count("4 bits") == 2
