"""8-bit integer products and row quantisation on the GPU.

The integer sums are exact, so without scales an f32 result is the sum
rounded once to f32, and is compared for equality.  With scales: the sum's
conversion and each of the products scale_a, scale_b, alpha and the sum with
the bias round once (unit roundoff 2^-24 each), so the value before the
activation errs by at most 5 x 2^-24 times its scaled sum's magnitude plus
2^-24 of its own.  The activations have slopes of at most 1.13; the kernels'
own forms of erf, exp and the division add at most 8e-7 + 2^-22 |v| of |v|.
One rounding to the output type adds its unit roundoff."""
import numpy as np
import pytest
import torch

import oracle

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


def codes(shape, seed, kind="uniform"):
    g = torch.Generator().manual_seed(seed)
    if kind == "low":
        return torch.full(shape, -128, dtype=torch.int8)
    if kind == "high":
        return torch.full(shape, 127, dtype=torch.int8)
    return torch.randint(-128, 128, shape, generator=g, dtype=torch.int32).to(torch.int8)


def padded(x, pitch, offset=0, fill=91):
    """x on the GPU as a view with row pitch `pitch`, `offset` elements into
    its buffer, other bytes `fill`; (view, buffer)."""
    *lead, rows, cols = x.shape
    mats = int(np.prod(lead)) if lead else 1
    buf = torch.full((offset + mats * rows * pitch + 64,), fill, dtype=x.dtype, device="cuda")
    view = buf[offset:offset + mats * rows * pitch].view(*lead, rows, pitch)[..., :cols]
    view.copy_(x)
    return view, buf


def sums(A, B):
    """The exact integer sums in f64 (below 2^53)."""
    return torch.matmul(A.double(), B.double()).numpy()


def up(n, m):
    return max(m, -(-n // m) * m)


SIZES = [(1, 1, 1), (1, 128, 64), (1, 1000, 4096), (2, 17, 15), (3, 257, 1023), (8, 130, 1024), (15, 64, 1025),
         (16, 1000, 2049), (17, 96, 700), (31, 500, 128), (32, 144, 5000), (33, 40, 333), (48, 129, 2048),
         (64, 256, 4100), (65, 300, 64), (97, 333, 4095), (128, 128, 1024), (129, 127, 1100), (200, 512, 2304),
         (255, 260, 130), (257, 1030, 513), (300, 700, 1537), (513, 65, 4097), (1000, 1000, 1000)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_sums_are_exact(b, M, N, K):
    A, B = codes((M, K), M * 7 + K), codes((K, N), N * 5 + K)
    want = sums(A, B).astype(np.float32)
    for pa, pb, pc, oa, ob in ((16, 16, 1, 0, 0), (1, 1, 1, 0, 0), (16, 16, 8, 0, 0), (16, 1, 3, 16, 3),
                               (1, 16, 4, 5, 16)):
        dA, _ = padded(A, up(K, pa), oa)
        dB, _ = padded(B, up(N, pb), ob)
        C, buf = padded(torch.full((M, N), PRIOR), up(N, pc), 3, fill=PRIOR)
        b.gemm_s8(dA, dB, out=C)
        b.check(b.gemm_get_device_status(0))
        got = C.cpu().numpy()
        assert np.array_equal(got, want), np.argwhere(got != want)[:4]
        C.fill_(PRIOR)
        assert bool((buf == PRIOR).all())  # nothing outside C was written


@pytest.mark.parametrize("M", [1, 16, 40, 130, 300])
@pytest.mark.parametrize("ka,kb", [("low", "low"), ("high", "low"), ("high", "high"), ("low", "uniform")])
def test_extreme_codes_stay_exact(b, M, ka, kb):
    """Long sums of the largest products: far past f32's 24 bits."""
    for K, N in ((1024, 70), (1056, 130), (8200, 256), (131071, 33)):
        A, B = codes((M, K), 1, ka), codes((K, N), 2, kb)
        A[:, ::37] += 1 if ka == "low" else -1
        got = b.gemm_s8(A.cuda(), B.cuda()).cpu().numpy()
        assert np.array_equal(got, sums(A, B).astype(np.float32))


def test_empty_and_single(b):
    for M, N in ((1, 1), (5, 130), (140, 9)):
        A = torch.empty((M, 0), dtype=torch.int8, device="cuda")
        B = torch.empty((0, N), dtype=torch.int8, device="cuda")
        bias = torch.arange(N, device="cuda", dtype=torch.float32) - 4
        out = b.gemm_s8(A, B, bias=bias, activation="relu")
        assert torch.equal(out, bias.clamp(min=0).expand(M, N))
    out = torch.full((0, 8), 1.0, device="cuda")
    assert b.gemm_s8(torch.empty((0, 4), dtype=torch.int8, device="cuda"), codes((4, 8), 1).cuda(), out=out) is out


def value_reference(S, sa, sb, alpha, bias, act):
    """(result, bound before the output rounding) in f64."""
    scaled = alpha * sa[..., :, None] * sb[..., None, :] * S
    v = scaled + (bias[..., None, :] if bias is not None else 0.0)
    tol = 5 * 2.0 ** -24 * np.abs(scaled) * (1 + 2.0 ** -20) + 2.0 ** -24 * np.abs(v)
    out = oracle.activation_f64(v, act, 0.01)
    if act != "none":
        tol = 1.13 * tol + np.abs(v) * (8e-7 + 2.0 ** -22 * np.minimum(np.abs(v), 90.0))
    return out, tol


def check_values(got, want, tol, out_type):
    assert np.all(np.abs(got - want) <= tol + ROUNDOFF[out_type] * (np.abs(want) + tol) + TINY[out_type])


@pytest.mark.parametrize("act", ["none", "relu", "leaky_relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("out_type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 300, 500), (16, 256, 2048), (20, 77, 96), (70, 260, 1100), (180, 516, 2100)])
def test_scales_bias_and_activation(b, M, N, K, out_type, act):
    g = torch.Generator().manual_seed(M + N)
    A, B = codes((M, K), 3), codes((K, N), 4)
    sa = torch.rand((M,), generator=g) * 0.03 + 1e-3
    sb = (torch.rand((N,), generator=g) - 0.3) * 0.02
    bias = torch.randn((N,), generator=g)
    dA, _ = padded(A, up(K, 16))
    dB, _ = padded(B, up(N, 16))
    want, tol = value_reference(sums(A, B), sa.double().numpy(), sb.double().numpy(), 0.75,
                                bias.double().numpy(), act)
    for pc in (1, 8, 5):
        C, _ = padded(torch.full((M, N), PRIOR, dtype=TORCH[out_type]), up(N, pc), fill=PRIOR)
        b.gemm_s8(dA, dB, sa.cuda(), sb.cuda(), C, alpha=0.75, bias=bias.cuda(), activation=act)
        check_values(C.double().cpu().numpy(), want, tol, out_type)
    b.check(b.gemm_get_device_status(0))


@pytest.mark.parametrize("M,N,K,batch", [(1, 64, 100, 5), (24, 130, 1030, 3), (150, 200, 260, 4)])
def test_batches(b, M, N, K, batch):
    A, B = codes((batch, M, K), 5), codes((batch, K, N), 6)
    g = torch.Generator().manual_seed(1)
    sa, sb = torch.rand((batch, M), generator=g), torch.rand((N,), generator=g)  # one scale_b for all
    dA, _ = padded(A, up(K, 16))
    dB, _ = padded(B, up(N, 16))
    out = b.gemm_s8(dA, dB, sa.cuda(), sb.cuda())
    want, tol = value_reference(sums(A, B), sa.double().numpy(), np.broadcast_to(sb.double().numpy(), (batch, N)),
                                1.0, None, "none")
    check_values(out.double().cpu().numpy(), want, tol, "f32")


@pytest.mark.parametrize("groups,M,N,K", [(1, 4, 40, 64), (5, 16, 200, 1100), (6, 32, 130, 257), (9, 40, 136, 520),
                                          (4, 200, 300, 1030), (7, 300, 520, 300), (300, 8, 24, 40)])
def test_grouped(b, groups, M, N, K):
    g = torch.Generator().manual_seed(groups)
    rows = torch.randint(0, M + 1, (groups,), generator=g, dtype=torch.int32)
    rows[0] = M
    if groups > 2:
        rows[1], rows[2] = 0, 1
    A, B = codes((groups, M, K), 7), codes((groups, K, N), 8)
    sa, sb = torch.rand((groups, M), generator=g) * 0.02, torch.rand((groups, N), generator=g) * 0.02
    for i, r in enumerate(rows.tolist()):
        sa[i, r:] = float("nan")
    dA, _ = padded(A, up(K, 16))
    dB, _ = padded(B, up(N, 16))
    for pitch in (up(N, 8), N):
        C, buf = padded(torch.full((groups, M, N), PRIOR, dtype=torch.float16), pitch, fill=PRIOR)
        b.grouped_gemm_s8(dA, dB, sa.cuda(), sb.cuda(), rows.cuda(), C, activation="silu")
        b.check(b.gemm_get_device_status(0))
        got = C.double().cpu().numpy()
        for i, r in enumerate(rows.tolist()):
            assert np.all(got[i, r:] == PRIOR)
            want, tol = value_reference(sums(A[i, :r], B[i]), sa[i, :r].double().numpy(), sb[i].double().numpy(),
                                        1.0, None, "silu")
            check_values(got[i, :r], want, tol, "f16")


@pytest.mark.parametrize("M", [8, 150])
def test_grouped_counts_out_of_range_are_clamped_and_reported(b, M):
    A, B = codes((3, M, 64), 9).cuda(), codes((3, 64, 32), 10).cuda()
    rows = torch.tensor([M + 5, -2, 3], dtype=torch.int32, device="cuda")
    out = b.grouped_gemm_s8(A, B, None, None, rows)
    st = b.gemm_get_device_status(0)
    assert st == b.GEMM_ERR_INVALID_VALUE
    assert b.gemm_get_device_status(0) == b.GEMM_OK
    got = out.cpu().numpy()
    assert np.array_equal(got[0], sums(A[0].cpu(), B[0].cpu()).astype(np.float32))
    assert np.all(got[1] == 0) and np.all(got[2, 3:] == 0)
    assert np.array_equal(got[2, :3], sums(A[2, :3].cpu(), B[2].cpu()).astype(np.float32))


def test_nan_scale_reaches_its_row_and_column_only(b):
    for M in (4, 40, 200):
        A, B = codes((M, 256), 11).cuda(), codes((256, 160), 12).cuda()
        sa, sb = torch.ones(M, device="cuda"), torch.ones(160, device="cuda")
        sa[2], sb[7] = float("nan"), float("inf")
        out = b.gemm_s8(A, B, sa, sb).cpu()
        assert bool(torch.isnan(out[2]).all())
        rest = [i for i in range(M) if i != 2]
        assert bool((~torch.isfinite(out[rest][:, 7])).all())
        cols = [j for j in range(160) if j != 7]
        assert bool(torch.isfinite(out[rest][:, cols]).all())


@pytest.mark.parametrize("M,N,K", [(4, 4096, 4096), (64, 1500, 3000), (520, 2100, 1600)])
def test_repeats_and_other_streams(b, M, N, K):
    A, B = codes((M, K), 13).cuda(), codes((K, up(N, 16)), 14).cuda()[:, :N]
    sa, sb = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    first = b.gemm_s8(A, B, sa, sb)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(first) for _ in range(9)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        b.gemm_s8(A, B, sa, sb, o, stream=streams[i % 3])
    torch.cuda.synchronize()
    b.check(b.gemm_get_device_status(0))
    assert all(torch.equal(first, o) for o in outs)


@pytest.mark.parametrize("M", [3, 100, 300])
def test_capture_in_a_graph(b, M):
    A, B = codes((M, 2048), 15).cuda(), codes((2048, 1024), 16).cuda()
    out = b.gemm_s8(A, B)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.gemm_s8(A, B, out=out)
    for seed in (17, 18):
        A.copy_(codes((M, 2048), seed))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.cpu().numpy(), sums(A.cpu(), B.cpu()).astype(np.float32))


# ------------------------------------------------------------------ quantisation

def quantize_reference(x):
    """The definition in f32 (its scale and quotient are f32 values)."""
    x = x.float().numpy()
    top = np.abs(x).max(axis=-1) if x.shape[-1] else np.zeros(x.shape[:-1], np.float32)
    with np.errstate(all="ignore"):
        scale = (top / np.float32(127)).astype(np.float32)
        q = np.rint((x / np.where(scale > 0, scale, 1)[..., None]).astype(np.float32))
    q = np.clip(np.where((scale > 0)[..., None], q, 0), -127, 127)
    bad = ~np.isfinite(top)
    scale[bad] = np.nan
    q[bad] = 0
    return q.astype(np.int8), scale


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (1, 4096), (5, 8192), (4, 8200), (130, 100), (2, 40000), (17, 1023)])
def test_quantize_rows(b, M, K, dtype):
    g = torch.Generator().manual_seed(K)
    x = (torch.randn((M, K), generator=g) * torch.exp(3 * torch.randn((M, 1), generator=g))).to(TORCH[dtype])
    if M > 2:
        x[0] = 0.0
        x[1, K // 2] = float("inf")
        x[2, K // 3] = float("nan")
    if M > 4:
        x[3] = torch.sign(x[3].float()).to(x.dtype) * 5e-8  # subnormal in f16
        x[4, 0] = torch.finfo(x.dtype).max
    want_q, want_s = quantize_reference(x)
    for pitch in (K, up(K, 16), K + 3):
        dx, _ = padded(x, pitch, fill=float("nan"))
        q, s = b.quantize_rows(dx)
        assert np.array_equal(q.cpu().numpy(), want_q)
        assert np.array_equal(s.cpu().numpy(), want_s, equal_nan=True)
        buf = torch.full((M, K + 5), 33, dtype=torch.int8, device="cuda")
        b.quantize_rows(dx, q=buf[:, :K])
        assert np.array_equal(buf[:, :K].cpu().numpy(), want_q) and bool((buf[:, K:] == 33).all())


def test_quantize_rows_grouped(b):
    x = torch.randn((4, 9, 64), device="cuda").bfloat16()
    rows = torch.tensor([0, 9, 4, 30], dtype=torch.int32, device="cuda")
    q = torch.full((4, 9, 64), 55, dtype=torch.int8, device="cuda")
    s = torch.full((4, 9), -1.0, device="cuda")
    b.quantize_rows(x, rows, q, s)
    want_q, want_s = quantize_reference(x.cpu())
    for e, r in enumerate((0, 9, 4, 9)):
        assert np.array_equal(q[e, :r].cpu().numpy(), want_q[e, :r]) and np.array_equal(s[e, :r].cpu().numpy(), want_s[e, :r])
        assert bool((q[e, r:] == 55).all()) and bool((s[e, r:] == -1).all())


def test_quantised_product_is_near_the_product(b):
    """x W with both quantised: each code is within half a step, so a cell is
    within (|x| sw + |w| sx + sx sw / 2) / 2 summed over k."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn((30, 512), generator=g).half()
    W = torch.randn((512, 80), generator=g).half()
    q, sx = b.quantize_rows(x.cuda())
    qw, sw = b.quantize_rows(W.t().contiguous().cuda())
    out = b.gemm_s8(q, qw.t().contiguous(), sx, sw).double().cpu()
    sx, sw = sx.double().cpu(), sw.double().cpu()
    want = x.double() @ W.double()
    bound = (x.double().abs().sum(1)[:, None] * sw / 2 + W.double().abs().sum(0) * sx[:, None] / 2
             + 512 * sx[:, None] * sw / 4) * (1 + 1e-5)
    assert bool(((out - want).abs() <= bound).all())


def test_refusals(b):
    A, B = codes((4, 32), 1).cuda(), codes((32, 8), 2).cuda()
    with pytest.raises(TypeError):
        b.gemm_s8(A.float(), B)
    with pytest.raises(ValueError):
        b.gemm_s8(A, B[:16])
    with pytest.raises(ValueError):
        b.gemm_s8(A, B, torch.ones(5, device="cuda"))
    with pytest.raises(ValueError):
        b.gemm_s8(A.t(), A)
    with pytest.raises(ValueError):
        b.grouped_gemm_s8(A[None], B[None], None, None, torch.tensor([1], device="cuda"))
    with pytest.raises(b.GemmError):  # past the longest exact sum
        b.gemm_s8(torch.empty((1, 131072), dtype=torch.int8, device="cuda"),
                  torch.empty((131072, 1), dtype=torch.int8, device="cuda"))
    host = torch.zeros((4, 32), dtype=torch.int8)
    C = torch.empty((4, 8), device="cuda")
    assert b.gemm_s8_scaled(host.data_ptr(), B.data_ptr(), C.data_ptr(), 0, 0, 4, 8, 32, 32, 8, 8) \
        == b.GEMM_ERR_INVALID_VALUE
    assert b.gemm_s8_scaled(A.data_ptr(), B.data_ptr(), A.data_ptr(), 0, 0, 4, 8, 32, 32, 8, 8) == b.GEMM_ERR_ALIAS
    with pytest.raises(TypeError):
        b.quantize_rows(A)


@pytest.mark.parametrize("groups,M,N,K", [(33, 32, 200, 70), (17, 16, 300, 1030), (300, 9, 40, 33), (70, 300, 130, 130)])
def test_every_count_of_rows(b, groups, M, N, K):
    """Counts 0, 1, 2 ... M in turn, in more groups than one launch takes, too."""
    rows = [(i * (1 if M < groups else 7)) % (M + 1) for i in range(groups)]
    A, B = codes((groups, M, K), groups), codes((groups, K, N), groups + 1)
    C = torch.full((groups, M, N), PRIOR, device="cuda")
    b.grouped_gemm_s8(A.cuda(), B.cuda(), None, None, torch.tensor(rows, dtype=torch.int32, device="cuda"), C)
    b.check(b.gemm_get_device_status(0))
    got = C.cpu().numpy()
    for g, r in enumerate(rows):
        assert np.array_equal(got[g, :r], sums(A[g, :r], B[g]).astype(np.float32)), g
        assert (got[g, r:] == PRIOR).all(), g


@pytest.mark.parametrize("M", [5, 20, 100, 300])
def test_small_and_large_sums_together(b, M):
    """Sums on both sides of 2^22 and 2^24, where the ways to f32 differ."""
    K, N = 3000, 70
    A, B = codes((M, K), M), codes((K, N), M + 1)
    for i, edge in enumerate((255, 256, 257, 1023, 1024, 1025)):
        if 2 * i + 1 < M:
            A[2 * i + 1] = 0
            A[2 * i + 1, :edge] = -128
        B[:, 2 * i] = -128
        B[:, 2 * i + 1] = 127
    C = b.gemm_s8(A.cuda(), B.cuda())
    b.check(b.gemm_get_device_status(0))
    assert np.array_equal(C.cpu().numpy(), sums(A, B).astype(np.float32))


# Sizes that pairs of CTAs multiply (the smaller ones above go to single CTAs).
@pytest.mark.parametrize("M,N,K", [(1500, 2100, 1200), (1537, 2049, 1025), (900, 3000, 2000), (4000, 4100, 130)])
def test_large_sums_are_exact(b, M, N, K):
    A, B = codes((M, K), M + K), codes((K, N), N + K)
    want = sums(A, B).astype(np.float32)
    for pitch in (16, 1):
        dA, _ = padded(A, up(K, 16))
        dB, _ = padded(B, up(N, 16))
        C, buf = padded(torch.full((M, N), PRIOR), up(N, pitch) + (pitch == 16) * 16, 4, fill=PRIOR)
        b.gemm_s8(dA, dB, out=C)
        b.check(b.gemm_get_device_status(0))
        assert np.array_equal(C.cpu().numpy(), want)
        C.fill_(PRIOR)
        assert (buf == PRIOR).all()


@pytest.mark.parametrize("act", ["none", "relu", "leaky_relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("out_type", ["f32", "f16", "bf16"])
def test_large_with_scales_bias_and_activation(b, out_type, act):
    M, N, K = 1300, 2500, 700
    g = torch.Generator().manual_seed(5)
    A, B = codes((M, K), 1), codes((K, N), 2)
    sa = torch.rand((M,), generator=g) * 0.03 + 1e-3
    sb = (torch.rand((N,), generator=g) - 0.3) * 0.02
    bias = torch.randn((N,), generator=g)
    want, tol = value_reference(sums(A, B), sa.double().numpy(), sb.double().numpy(), 0.75, bias.double().numpy(), act)
    for pitch in (16, 1):
        C, _ = padded(torch.full((M, N), PRIOR, dtype=TORCH[out_type]), up(N + pitch, pitch), fill=PRIOR)
        b.gemm_s8(A.cuda(), B.cuda(), sa.cuda(), sb.cuda(), C, alpha=0.75, bias=bias.cuda(), activation=act)
        b.check(b.gemm_get_device_status(0))
        check_values(C.double().cpu().numpy(), want, tol, out_type)


def test_large_groups(b):
    groups, M, N, K = 40, 300, 1024, 520
    rows = [0, 300, 1, 255, 256, 257, 128, 129, 299, 64] * 4
    A, B = codes((groups, M, K), 3), codes((groups, K, N), 4)
    C = torch.full((groups, M, N), PRIOR, device="cuda")
    b.grouped_gemm_s8(A.cuda(), B.cuda(), None, None, torch.tensor(rows, dtype=torch.int32, device="cuda"), C)
    b.check(b.gemm_get_device_status(0))
    got = C.cpu().numpy()
    for g, r in enumerate(rows):
        assert np.array_equal(got[g, :r], sums(A[g, :r], B[g]).astype(np.float32)), g
        assert (got[g, r:] == PRIOR).all(), g


def test_capture_of_a_pair_that_cuts_its_tiles(b):
    M, N, K = 300, 5008, 8192
    A, B = codes((M, K), 8).cuda(), codes((K, N), 9).cuda()
    C = torch.zeros((M, N), device="cuda")
    want = b.gemm_s8(A, B).clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.gemm_s8(A, B, out=C)
    for _ in range(3):
        C.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(C, want)
    b.check(b.gemm_get_device_status(0))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_scales_are_quotients_for_every_mantissa(b, dtype):
    """max / 127 as a division rounds it: a multiplication by the rounded
    reciprocal gives another scale for 6 of the 128 mantissas of bf16 and 46 of
    the 1024 of f16, and then another code where x / scale lies on a tie (the
    halves of the maximum: 63.5)."""
    n = {"f32": 4096, "f16": 1024, "bf16": 128}[dtype]
    top = (1 + torch.arange(n, dtype=torch.float64) / n).to(TORCH[dtype])
    half = top / 2  # (exact)
    x = torch.stack([top, half, -half, top / 4, -top, torch.zeros_like(top)], 1)
    want_q, want_s = quantize_reference(x)
    for rows in (x, x[:100], x.repeat(1, 50)):
        q, s = b.quantize_rows(rows.cuda())
        m = rows.shape[0]
        assert np.array_equal(s.cpu().numpy(), want_s[:m])
        assert np.array_equal(q.cpu().numpy(), np.tile(want_q[:m], rows.shape[1] // 6))


@pytest.mark.parametrize("act", ["none", "relu", "leaky_relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("out_type", ["f32", "f16", "bf16"])
def test_a_row_does_not_depend_on_the_rows_beside_it(b, out_type, act):
    """The same rows in calls of 1 to 1400: every kernel, the same bits."""
    N, K = 2600, 700
    g = torch.Generator().manual_seed(21)
    A, B = codes((1400, K), 21).cuda(), codes((K, up(N, 16)), 22).cuda()[:, :N]
    sa = (torch.rand((1400,), generator=g) * 0.03 + 1e-3).cuda()
    sb = ((torch.rand((N,), generator=g) - 0.3) * 0.02).cuda()
    bias = torch.randn((N,), generator=g).cuda()
    for kw in ({"bias": bias, "alpha": 0.7}, {"alpha": 0.7}, {"bias": bias}):
        for scales in ((sa, sb), (None, sb), (sa, None)):
            def call(m):
                return b.gemm_s8(A[:m], B, *(v[:m] if v is sa else v for v in scales), activation=act,
                                 out_dtype=TORCH[out_type], **kw)
            all_rows = call(1400)
            for m in (1, 16, 17, 32, 33, 128, 300):
                assert torch.equal(call(m), all_rows[:m]), m
    groups = b.grouped_gemm_s8(A[:60].view(2, 30, K), torch.stack([B, B]), sa[:60].view(2, 30), sb,
                               torch.tensor([30, 7], dtype=torch.int32, device="cuda"), alpha=0.7, bias=bias,
                               activation=act, out_dtype=TORCH[out_type])
    rows = b.gemm_s8(A, B, sa, sb, alpha=0.7, bias=bias, activation=act, out_dtype=TORCH[out_type])
    assert torch.equal(groups[0], rows[:30]) and torch.equal(groups[1, :7], rows[30:37])


@pytest.mark.parametrize("K", [0, 48])
def test_counts_out_of_range_are_reported_without_a_sum_too(b, K):
    groups, M, N = 300, 6, 16  # (more groups than one launch takes)
    A, B = codes((groups, M, K), 23).cuda(), codes((groups, K, N), 24).cuda()
    bias = torch.arange(N, device="cuda", dtype=torch.float32)
    rows = torch.full((groups,), M, dtype=torch.int32)
    want = None
    for at, bad in ((None, None), (0, M + 1), (5, -1), (299, 2 ** 31 - 1)):
        counts = rows.clone()
        if at is not None:
            counts[at] = bad
        out = b.grouped_gemm_s8(A, B, None, None, counts.cuda(), torch.full((groups, M, N), PRIOR, device="cuda"),
                                bias=bias)
        assert b.gemm_get_device_status(0) == (b.GEMM_OK if at is None else b.GEMM_ERR_INVALID_VALUE)
        assert b.gemm_get_device_status(0) == b.GEMM_OK
        if at is None:
            want = out
        else:
            expect = want.clone()
            if bad < 0:
                expect[at] = PRIOR
            assert torch.equal(out, expect)


# From 608 rows on 152 SMs a warp takes a row of at most 256 pieces (of 16 or 4
# bytes, or one element), and 128 threads a longer one, past 1024 pieces in a loop.
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,K", [(611, 100), (1003, 1023), (1001, 1), (2000, 64), (700, 8200), (650, 40000), (613, 257)])
def test_quantize_many_rows(b, M, K, dtype):
    g = torch.Generator().manual_seed(M + K)
    x = (torch.randn((M, K), generator=g) * torch.exp(3 * torch.randn((M, 1), generator=g))).to(TORCH[dtype])
    x[7] = 0.0
    x[8, K // 2] = float("inf")
    x[M - 1, K // 3] = float("nan")
    x[M - 2] = torch.sign(x[M - 2].float()).to(x.dtype) * 5e-8
    x[M - 3, 0] = torch.finfo(x.dtype).max
    want_q, want_s = quantize_reference(x)
    for pitch, out_pitch in ((K, K), (up(K, 16), up(K, 16)), (K + 2, K + 5), (K + 1, up(K, 4))):
        dx, _ = padded(x, pitch, fill=float("nan"))
        buf = torch.full((M, out_pitch), 33, dtype=torch.int8, device="cuda")
        q, s = b.quantize_rows(dx, q=buf[:, :K])
        assert np.array_equal(q.cpu().numpy(), want_q)
        assert np.array_equal(s.cpu().numpy(), want_s, equal_nan=True)
        assert bool((buf[:, K:] == 33).all())


@pytest.mark.parametrize("M,K", [(9, 64), (70, 1408), (90, 5000)])
def test_quantize_experts_rows_with_counts(b, M, K):
    """Kernels of each size, with counts of every kind."""
    groups = 70
    g = torch.Generator().manual_seed(M)
    x = torch.randn((groups, M, K), generator=g).half()
    rows = torch.randint(-2, M + 3, (groups,), generator=g, dtype=torch.int32)
    q = torch.full((groups, M, K), 55, dtype=torch.int8, device="cuda")
    s = torch.full((groups, M), -1.0, device="cuda")
    b.quantize_rows(x.cuda(), rows.cuda(), q, s)
    want_q, want_s = quantize_reference(x)
    q, s = q.cpu().numpy(), s.cpu().numpy()
    for e, r in enumerate(rows.clamp(0, M).tolist()):
        assert np.array_equal(q[e, :r], want_q[e, :r]) and np.array_equal(s[e, :r], want_s[e, :r])
        assert (q[e, r:] == 55).all() and (s[e, r:] == -1).all()


def test_large_operands_of_any_pitch(b):
    """Packed copies of more than one grid's bytes, at every byte offset."""
    M, N, K = 1030, 4099, 5003
    A, B = codes((M, K), 25), codes((K, N), 26)
    want = b.gemm_s8(padded(A, up(K, 16))[0], padded(B, up(N, 16))[0])
    for oa, ob in ((0, 0), (1, 2), (2, 3), (3, 1)):
        assert torch.equal(b.gemm_s8(padded(A, K, oa)[0], padded(B, N, ob)[0]), want)
    assert np.array_equal(want[::97].cpu().numpy(), sums(A[::97], B).astype(np.float32))
