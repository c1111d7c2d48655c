"""Microscaled 4-bit rows on the GPU: quantisation and products.

Quantisation is compared code by code with the definition in 64 bits.

Products: codes are multiples of 1/2 and at most 6.  With block scales that
are powers of two between 1/2 and 2 every product is a multiple of 2^-4 and a
sum of K of them at most 144 K, so that for K below 7000 every partial sum is
exact in f32, whatever the order, and results are compared for equality.

With any scales a product of two codes and two e4m3 scales has 14 bits at most
and is exact; the f32 sum of K of them, each addition off by at most 2^-23 of
the magnitudes added up (rounded or cut off), by K 2^-23 of them in the worst
case; sums of 16 products and more are formed at once, which leaves K / 16
additions.  Scaling and bias add 4 roundings of 2^-24, the activations have
slopes of at most 1.13 and add at most 8e-7 + 2^-22 |v|; one rounding to the
output type adds its unit roundoff."""
import math

import numpy as np
import pytest
import torch

import fp4_util as fp4

pytestmark = pytest.mark.gpu

ROUNDOFF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
PRIOR = 41.0  # what C holds before a call


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.fail("the GPU tests need a CUDA device")
    from tiled_staged_matmul_gb300 import binding
    return binding


def up(n, m):
    return max(m, -(-n // m) * m)


# ------------------------------------------------------------------ quantisation

def check_quantised(b, x, block, got):
    """x: the M x K values on the CPU."""
    K = x.shape[1]
    codes, bytes_, scales = fp4.quantised(x.double().numpy(), block)
    c, s = fp4.unpacked(got, K)
    blocks = bytes_.shape[1]
    assert np.array_equal(s[:, :blocks], bytes_), np.argwhere(s[:, :blocks] != bytes_)[:4]
    assert (s[:, blocks:] == 0).all()
    # (A negative value that becomes 0 may keep its sign.)
    same = (c[:, :K] == codes) | ((codes == 0) & (c[:, :K] & 7 == 0))
    assert same.all(), (np.argwhere(~same)[:4], c[:, :K][~same][:4], codes[~same][:4])
    assert (c[:, K:] == 0).all()
    if block == 16:
        assert np.array_equal(got.scales.cpu().double().numpy(), scales, equal_nan=True)
    else:
        assert got.scales is None


QUANT = [(1, 1), (1, 16), (3, 15), (2, 33), (5, 64), (7, 100), (33, 255), (130, 256), (129, 1000), (300, 1030), (1, 4096),
         (17, 4097), (700, 512), (620, 2050), (3, 16384), (2, 16401), (1, 70001), (650, 8192), (640, 9000)]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K", QUANT)
def test_quantisation(b, M, K, dtype, block):
    g = torch.Generator().manual_seed(M * 31 + K)
    x = torch.randn((M, K), generator=g) * torch.exp(torch.randn((M, 1), generator=g))
    x = (x * torch.exp(2 * torch.randn((M, -(-K // 16)), generator=g)).repeat_interleave(16, 1)[:, :K]).to(TORCH[dtype])
    check_quantised(b, x.float(), block, b.quantize_fp4(x.cuda(), block=block))


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("pitch,offset", [(0, 0), (8, 0), (5, 0), (0, 1), (0, 8), (3, 3)])
def test_quantisation_of_views(b, dtype, block, pitch, offset):
    """Rows at any pitch and base: the values past a row's end are NaN."""
    M, K = 37, 200
    g = torch.Generator().manual_seed(pitch * 7 + offset)
    x = torch.randn((M, K), generator=g).to(TORCH[dtype])
    buf = torch.full((offset + M * (K + pitch) + 8,), float("nan"), dtype=TORCH[dtype], device="cuda")
    view = buf[offset:offset + M * (K + pitch)].view(M, K + pitch)[:, :K]
    view.copy_(x)
    check_quantised(b, x.float(), block, b.quantize_fp4(view, block=block))


@pytest.mark.parametrize("block", [16, 32])
def test_quantisation_at_the_borders(b, block):
    """Every middle between two codes and its neighbours in f32, under every scale
    of one exponent; and the scales' own middles."""
    rows = []
    middles = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], dtype=np.float32)
    for m in range(8):  # block maxima that give each mantissa of e4m3
        top = np.float32(6 * (8 + m) * 16)
        v = middles * np.float32((8 + m) * 16)
        near = np.concatenate([[top], v[:-1], np.nextafter(v[:-1], np.float32(0))])
        far = np.concatenate([[top], v[:-1], np.nextafter(v[:-1], np.float32(1e9))])
        pad = np.zeros((2, 32), dtype=np.float32)
        pad[0, :15], pad[1, :15] = near, far
        # a second block whose largest value fixes the row's scale
        rows += [np.concatenate([p, np.full(32, 2688.0, dtype=np.float32)]) for p in pad]
    tops = np.arange(6 * 16, 6 * 33, 3, dtype=np.float32)  # block maxima on the scales' middles
    for t in np.concatenate([tops, np.nextafter(tops, np.float32(0)), np.nextafter(tops, np.float32(1e9))]):
        row = np.zeros(64, dtype=np.float32)
        row[0], row[1], row[32] = t, t / 3, 2688.0
        rows.append(row)
    for scale in (1.0, 2.0 ** 100, 2.0 ** -100, 2.0 ** -126, 2.0 ** 116):
        x = torch.from_numpy(np.stack(rows)) * scale
        x[:, 1::2] *= -1
        check_quantised(b, x, block, b.quantize_fp4(x.cuda(), block=block))


@pytest.mark.parametrize("block", [16, 32])
def test_quantisation_of_extremes(b, block):
    rows = [torch.zeros(80), torch.full((80,), 2.0 ** -149), torch.full((80,), 3.4028234e38),
            torch.full((80,), 2.0 ** -126), torch.full((80,), -2.0 ** -130), -torch.zeros(80)]
    mixed = torch.zeros(80)
    mixed[0], mixed[20], mixed[40], mixed[79] = 3e38, 1e-30, 2.0 ** -140, -1.0
    x = torch.stack(rows + [mixed])
    check_quantised(b, x, block, b.quantize_fp4(x.cuda(), block=block))


def test_what_is_not_finite(b):
    """Blocks of 16: the row's scale is NaN and its codes 0; of 32: the block's."""
    x = torch.randn((6, 100), generator=torch.Generator().manual_seed(4))
    x[1, 50], x[3, 0], x[4, 99] = float("nan"), float("inf"), -float("inf")
    for dtype in TORCH.values():
        got = b.quantize_fp4(x.to(dtype).cuda(), block=16)
        bad = torch.tensor([False, True, False, True, True, False])
        assert torch.equal(torch.isnan(got.scales.cpu()), bad)
        assert not got.codes.cpu()[bad].any() and got.codes.cpu()[~bad].any(1).all()
        got = b.quantize_fp4(x.to(dtype).cuda(), block=32)
        _, s = fp4.unpacked(got, 100)
        want = np.zeros((6, 4), dtype=bool)
        want[1, 1] = want[3, 0] = want[4, 3] = True
        assert np.array_equal(s == 255, want)
        c = got.codes.cpu().numpy()
        assert not c[1, 16:32].any() and c[1, :16].any() and c[1, 32:].any()


@pytest.mark.parametrize("block", [16, 32])
def test_quantisation_of_groups(b, block):
    """Rows past a matrix's count are neither read nor written."""
    G, M, K = 5, 140, 150
    g = torch.Generator().manual_seed(8)
    x = torch.randn((G, M, K), generator=g)
    counts = [0, 140, 1, 77, 129]
    for e, n in enumerate(counts):
        x[e, n:] = float("nan")
    dx, dc = x.cuda(), torch.tensor(counts, dtype=torch.int32, device="cuda")
    width, blocks = 75, -(-K // block)
    tiles = (G, 2, -(-blocks // 4), 512)
    q = torch.full((G, M, 80), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full(tiles, 0x5A, dtype=torch.uint8, device="cuda")
    r = torch.full((G, M), PRIOR, device="cuda")
    b.check(b.fp4_quantize_rows(dx.data_ptr(), "f32", block, q.data_ptr(), s.data_ptr(), r.data_ptr(), dc.data_ptr(), M, K,
                                K, 80, M * K, M * 80, M, G))
    for e, n in enumerate(counts):
        assert (q[e, n:] == 0x5A).all() and (q[e, :, width:] == 0x5A).all()
        assert (r[e, n:] == PRIOR).all() and (block == 16 or (r[e] == PRIOR).all())
        i, k = np.meshgrid(np.arange(n, 256), np.arange(tiles[2] * 4), indexing="ij")
        assert (s[e].reshape(-1).cpu().numpy()[fp4.scale_place(i, k, blocks)] == 0x5A).all()
        if n:
            check_quantised(b, x[e, :n], block,
                            b.Fp4Rows(q[e, :n, :width], s[e], r[e, :n] if block == 16 else None, block))


# ------------------------------------------------------------------ products

def whole_operand(b, rows, K, block, seed, **kw):
    """An operand whose products have exact f32 sums, and its values."""
    g = np.random.default_rng(seed)
    codes = g.integers(0, 16, (rows, K)).astype(np.int64)
    blocks = -(-K // block)
    bytes_ = (np.array([48, 56, 64]) if block == 16 else np.array([126, 127, 128]))[g.integers(0, 3, (rows, blocks))]
    return fp4.on_gpu(b, codes, bytes_, None, block, **kw), fp4.values(codes, bytes_, None, block)


SIZES = [(1, 1, 1), (1, 128, 64), (1, 1000, 4096), (2, 17, 15), (3, 257, 1023), (8, 130, 1024), (16, 1000, 2049),
         (31, 500, 128), (32, 144, 5000), (33, 40, 333), (64, 256, 4100), (65, 300, 64), (97, 333, 4095), (128, 128, 1024),
         (128, 2000, 6000), (129, 127, 1100), (200, 512, 2304), (255, 260, 130), (257, 1030, 513), (300, 700, 1537),
         (513, 65, 4097), (1000, 1000, 1000), (130, 20000, 300), (7, 40000, 257), (2500, 1500, 96)]


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_sums_are_exact(b, M, N, K, block):
    A, va = whole_operand(b, M, K, block, M * 7 + K)
    B, vb = whole_operand(b, N, K, block, N * 5 + K)
    want = (va @ vb.T).astype(np.float32)
    for pc in (1, 8):
        buf = torch.full((M * up(N, pc) + 32,), PRIOR, device="cuda")
        C = buf[3:3 + M * up(N, pc)].view(M, up(N, pc))[:, :N]
        b.gemm_fp4(A, B, C)
        b.check(b.gemm_get_device_status(0))
        got = C.cpu().numpy()
        assert np.array_equal(got, want), np.argwhere(got != want)[:4]
        C.fill_(PRIOR)
        assert (buf == PRIOR).all(), "written past C"


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M", [5, 100, 300])
@pytest.mark.parametrize("pa,oa,pb,ob", [(177, 0, 176, 0), (176, 16, 208, 32), (192, 3, 176, 0), (176, 0, 181, 8),
                                         (179, 1, 171, 5)])
def test_operands_at_any_pitch_and_base(b, M, block, pa, oa, pb, ob):
    N, K = 150, 341
    A, va = whole_operand(b, M, K, block, M, pitch=pa, offset=oa)
    B, vb = whole_operand(b, N, K, block, N, pitch=pb, offset=ob)
    C = b.gemm_fp4(A, B)
    b.check(b.gemm_get_device_status(0))
    assert np.array_equal(C.cpu().numpy(), (va @ vb.T).astype(np.float32))


ACTS = {"none": lambda v: v, "relu": lambda v: np.maximum(v, 0), "leaky_relu": lambda v: np.where(v > 0, v, 0.2 * v),
        "gelu": lambda v: v * 0.5 * np.vectorize(math.erfc)(-v / math.sqrt(2)),
        "gelu_tanh": lambda v: v / 2 * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))),
        "silu": lambda v: v / (1 + np.exp(-v))}


def any_operand(b, rows, K, block, seed):
    """An operand of quantised normal values with row scales (block 16), or none."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, K)) * np.exp(g.standard_normal((rows, 1)))
    codes, bytes_, scales = fp4.quantised(x.astype(np.float32), block)
    if scales is not None:
        scales = (scales * g.uniform(0.7, 1.4, rows)).astype(np.float32)
    return fp4.on_gpu(b, codes, bytes_, scales, block), fp4.values(codes, bytes_, scales, block)


def check_product(got, va, vb, dtype, alpha=1.0, bias=None, act="none"):
    K = va.shape[1]
    s, mag = va @ vb.T * alpha, np.abs(va) @ np.abs(vb).T * abs(alpha)
    v = s + (0 if bias is None else bias[None, :].astype(np.float64))
    err = (K / 16 + 2) * 2.0 ** -23 * mag + 4 * 2.0 ** -24 * (mag + np.abs(v))
    want = ACTS[act](v)
    if act != "none":
        err = 1.13 * err + 8e-7 * np.abs(v) + 2.0 ** -22 * np.abs(v)
    err = err + ROUNDOFF[dtype] * (np.abs(want) + err) + TINY[dtype]
    got = got.cpu().double().numpy()
    bad = ~(np.abs(got - want) <= err)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], err[bad][:4])


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("M,N,K", [(3, 200, 300), (50, 131, 1000), (300, 259, 600)])
def test_epilogue(b, M, N, K, act, dtype, block):
    A, va = any_operand(b, M, K, block, M + K)
    B, vb = any_operand(b, N, K, block, N + K)
    bias = np.random.default_rng(N).standard_normal(N).astype(np.float32)
    alpha = 0.5 / math.sqrt(K)
    out = torch.full((M, N + 5), PRIOR, dtype=TORCH[dtype], device="cuda")
    b.gemm_fp4(A, B, out[:, :N], alpha=alpha, bias=torch.from_numpy(bias).cuda(), activation=act, slope=0.2)
    b.check(b.gemm_get_device_status(0))
    check_product(out[:, :N], va, vb, dtype, np.float32(alpha).astype(np.float64), bias, act)
    assert (out[:, N:] == PRIOR).all()


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (16, 3000, 20000), (128, 256, 30000), (200, 256, 40000), (1, 1, 100000)])
def test_long_sums(b, M, N, K, block):
    A, va = any_operand(b, M, K, block, 1)
    B, vb = any_operand(b, N, K, block, 2)
    out = b.gemm_fp4(A, B)
    b.check(b.gemm_get_device_status(0))
    check_product(out, va, vb, "f32")
    assert torch.equal(out, b.gemm_fp4(A, B)), "not reproducible"


def stacked(b, operands):
    """2-D operands of one shape as one 3-D operand."""
    return b.Fp4Rows(torch.stack([o.codes for o in operands]), torch.stack([o.block_scales for o in operands]),
                     None if operands[0].scales is None else torch.stack([o.scales for o in operands]), operands[0].block)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("batch,M,N,K", [(3, 5, 40, 96), (2, 60, 200, 300), (4, 130, 300, 257), (7, 100, 128, 64)])
def test_batches(b, batch, M, N, K, dtype, block):
    a = [any_operand(b, M, K, block, 10 + i) for i in range(batch)]
    w = [any_operand(b, N, K, block, 20 + i) for i in range(batch)]
    bias = np.random.default_rng(5).standard_normal((batch, N)).astype(np.float32)
    got = b.gemm_fp4(stacked(b, [x[0] for x in a]), stacked(b, [x[0] for x in w]), bias=torch.from_numpy(bias).cuda(),
                     out_dtype=TORCH[dtype])
    b.check(b.gemm_get_device_status(0))
    for i in range(batch):
        check_product(got[i], a[i][1], w[i][1], dtype, 1.0, bias[i])


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("cap,N,K,counts", [
    (16, 130, 300, [0, 16, 1, 7]), (40, 300, 513, [40, 0, 33, 2, 39]), (100, 128, 1030, [99, 100, 0, 1]),
    (300, 260, 257, [300, 0, 129, 256, 1, 257]), (512, 64, 64, [0, 0, 0]), (130, 700, 2000, [130, 3]),
    (20, 40, 100, [i % 21 for i in range(300)])])
def test_groups(b, cap, N, K, counts, block):
    G = len(counts)
    a = [whole_operand(b, cap, K, block, 3 + i) for i in range(min(G, 6))]
    w = [whole_operand(b, N, K, block, 50 + i) for i in range(min(G, 6))]
    A = stacked(b, [a[i % len(a)][0] for i in range(G)])
    B = stacked(b, [w[i % len(w)][0] for i in range(G)])
    # Rows past a count hold anything.
    for e, n in enumerate(counts):
        A.codes[e, n:] = 0x77
    out = torch.full((G, cap, N + 3), PRIOR, dtype=torch.float32, device="cuda")
    b.grouped_gemm_fp4(A, B, torch.tensor(counts, dtype=torch.int32, device="cuda"), out[..., :N])
    b.check(b.gemm_get_device_status(0))
    got = out.cpu().numpy()
    for e, n in enumerate(counts):
        want = a[e % len(a)][1][:n] @ w[e % len(w)][1].T
        assert np.array_equal(got[e, :n, :N], want.astype(np.float32)), e
        assert (got[e, n:] == PRIOR).all() and (got[e, :, N:] == PRIOR).all()


def test_counts_out_of_range_are_clamped_and_reported(b):
    a, w = whole_operand(b, 20, 64, 16, 1), whole_operand(b, 30, 64, 16, 2)
    A, B = stacked(b, [a[0]] * 3), stacked(b, [w[0]] * 3)
    want = torch.from_numpy((a[1] @ w[1].T).astype(np.float32)).cuda()
    for K0 in (False, True):
        out = torch.full((3, 20, 30), PRIOR, device="cuda")
        counts = torch.tensor([25, -3, 4], dtype=torch.int32, device="cuda")
        if K0:
            b.check(b.gemm_fp4_grouped_scaled(0, 0, out.data_ptr(), 0, 0, 0, 0, 16, counts.data_ptr(), 3, 20, 30, 0, 0, 0,
                                              30, 0, 0, 600))
        else:
            b.grouped_gemm_fp4(A, B, counts, out)
        assert b.gemm_get_device_status(0) == b.GEMM_ERR_INVALID_VALUE
        assert b.gemm_get_device_status(0) == b.GEMM_OK
        w0 = torch.zeros_like(want) if K0 else want
        assert torch.equal(out[0], w0) and (out[1] == PRIOR).all()
        assert torch.equal(out[2, :4], w0[:4]) and (out[2, 4:] == PRIOR).all()


def test_nan_scales_reach_their_rows_only(b):
    """A NaN row (of A or B) makes its row (column) of C NaN and nothing else."""
    for block in (16, 32):
        x = torch.randn((40, 100), generator=torch.Generator().manual_seed(1))
        y = torch.randn((150, 100), generator=torch.Generator().manual_seed(2))
        x[7, 50], y[33, 0], y[149, 99] = float("nan"), float("inf"), float("nan")
        out = b.gemm_fp4(b.quantize_fp4(x.cuda(), block=block), b.quantize_fp4(y.cuda(), block=block)).cpu()
        want = torch.zeros((40, 150), dtype=torch.bool)
        want[7], want[:, 33], want[:, 149] = True, True, True
        assert torch.equal(torch.isnan(out), want)


def test_empty_sizes(b):
    for block in (16, 32):
        e = b.quantize_fp4(torch.zeros((0, 64), device="cuda"), block=block)
        w = b.quantize_fp4(torch.ones((8, 64), device="cuda"), block=block)
        assert b.gemm_fp4(e, w).shape == (0, 8) and b.gemm_fp4(w, e).shape == (8, 0)
        k0 = b.quantize_fp4(torch.zeros((5, 0), device="cuda"), block=block)
        assert k0.scales is None or (k0.scales == 0).all()
        bias = torch.tensor([1.0, -2.0, 3.0, 0.0, 5.0], device="cuda")
        assert torch.equal(b.gemm_fp4(k0, k0, bias=bias, activation="relu"), bias.clamp(min=0).expand(5, 5))


def test_streams_graphs_and_calls_without_a_pause(b):
    """On another stream; many calls in a row; captured, with the inputs changed
    between replays.  Sizes whose tiles are cut along K, and whole ones."""
    for M, N, K in ((2, 300, 5000), (100, 700, 3500), (300, 1100, 2100)):
        A, va = whole_operand(b, M, K, 16, 1)
        B, vb = whole_operand(b, N, K, 16, 2)
        A2, va2 = whole_operand(b, M, K, 16, 3)
        want = torch.from_numpy((va @ vb.T).astype(np.float32)).cuda()
        want2 = torch.from_numpy((va2 @ vb.T).astype(np.float32)).cuda()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        outs = [b.gemm_fp4(A, B, stream=side) for _ in range(20)]
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
        outs = [b.gemm_fp4(A if i % 2 else A2, B) for i in range(30)]
        assert all(torch.equal(o, want if i % 2 else want2) for i, o in enumerate(outs))
        out = torch.empty_like(want)
        out_b = torch.empty_like(want)
        graph, graph_b = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.gemm_fp4(A, B, out)
            b.gemm_fp4(A, B, out)
        with torch.cuda.graph(graph_b):
            b.gemm_fp4(A2, B, out_b)
        for i in range(6):
            out.fill_(PRIOR)
            graph.replay()
            graph_b.replay()
            b.gemm_fp4(A2, B)
            assert torch.equal(out, want) and torch.equal(out_b, want2), i
            want, A_new = (want2, A2) if i == 2 else (want, None)
            if A_new is not None:
                A.codes.copy_(A2.codes)
                A.block_scales.copy_(A2.block_scales)
        b.check(b.gemm_get_device_status(0))


@pytest.mark.parametrize("block", [16, 32])
def test_quantise_and_multiply(b, block):
    """A linear layer as a program runs it, against its own quantised operands."""
    for M, N, K in ((1, 500, 1024), (20, 300, 700), (200, 600, 513)):
        g = torch.Generator().manual_seed(M)
        x, w = torch.randn((M, K), generator=g), torch.randn((N, K), generator=g)
        got = b.gemm_fp4(b.quantize_fp4(x.half().cuda(), block=block), b.quantize_fp4(w.half().cuda(), block=block),
                         out_dtype=torch.float16)
        va = fp4.values(*fp4.quantised(x.half().double().numpy(), block), block)
        vb = fp4.values(*fp4.quantised(w.half().double().numpy(), block), block)
        check_product(got, va, vb, "f16")
