// fp4_api.cu -- host side of the choice of experts and of the microscaled 4-bit
// operators (include/tsm_gemm.h): argument checks, launch shapes and launches.
#include "api_checks.h"
#include "fp4_plan.h"

#include <algorithm>
#include <mutex>

namespace tsm {
namespace {

// What both directions of the choice share.
gemm_status_t check_choose(int32_t elem_type, int64_t tokens, int64_t experts, int64_t topk, int64_t ld, int32_t score)
{
    if (!known_elem(elem_type))
        return fail(GEMM_ERR_INVALID_VALUE, "unknown element type %d", elem_type);
    if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)
        return fail(GEMM_ERR_INVALID_VALUE, "unknown score %d", score);
    if (tokens < 0 || tokens > kInt32Max)
        return fail(GEMM_ERR_INVALID_VALUE, "tokens must be in [0, 2^31)");
    if (experts < 1 || experts > kMaxChooseExperts)
        return fail(GEMM_ERR_INVALID_VALUE, "experts must be in [1, %d], not %lld", kMaxChooseExperts, (long long)experts);
    if (topk < 0 || topk > kMaxChooseTopk || topk > experts)
        return fail(GEMM_ERR_INVALID_VALUE, "topk must be in [0, %d] and at most the experts, not %lld", kMaxChooseTopk,
                    (long long)topk);
    if (ld < experts)
        return fail(GEMM_ERR_INVALID_VALUE, "a row pitch is below the experts (%lld)", (long long)experts);
    return GEMM_OK;
}

}  // namespace
}  // namespace tsm

using namespace tsm;

extern "C" {

gemm_status_t choose_experts(const void *logits, int32_t elem_type, const float *bias, int32_t *ids, float *weights,
                             int64_t tokens, int64_t experts, int64_t topk, int64_t ld, int32_t score, int64_t groups,
                             int64_t keep_groups, int32_t group_best, int32_t renormalize, float scale,
                             gemm_stream_t stream)
{
    g_last_error.clear();
    gemm_status_t st = check_choose(elem_type, tokens, experts, topk, ld, score);
    if (st != GEMM_OK)
        return st;
    if (groups < 1 || groups > kMaxChooseGroups || experts % groups != 0)
        return fail(GEMM_ERR_INVALID_VALUE, "groups must be in [1, %d] and divide the experts (%lld), not %lld", kMaxChooseGroups,
                    (long long)experts, (long long)groups);
    if ((groups & (groups - 1)) != 0 && experts > kMaxChooseUneven)
        return fail(GEMM_ERR_INVALID_VALUE, "at most %d experts in %lld groups (no power of two)", kMaxChooseUneven,
                    (long long)groups);
    if (keep_groups < 1 || keep_groups > groups)
        return fail(GEMM_ERR_INVALID_VALUE, "keep_groups must be in [1, groups], not %lld", (long long)keep_groups);
    if (group_best != 1 && group_best != 2)
        return fail(GEMM_ERR_INVALID_VALUE, "group_best must be 1 or 2, not %d", group_best);
    const int64_t eb = elem_bytes(elem_type);
    if (misaligned(logits, eb) || misaligned(bias, 4) || misaligned(ids, 4) || misaligned(weights, 4))
        return fail(GEMM_ERR_MISALIGNED, "every buffer must sit at its elements' natural alignment");
    const Buffer buf[] = {{logits, topk ? span(tokens, experts, ld, eb) : 0, "logits", false},
                          {bias, bias ? experts * 4 : 0, "bias", false},
                          {ids, tokens * topk * 4, "ids", true},
                          {weights, tokens * topk * 4, "weights", true}};
    if ((st = check_buffers(buf, 4)) != GEMM_OK || tokens == 0 || topk == 0)
        return st;
    int dev = 0;
    DeviceState *ds = nullptr;
    if ((st = current(&dev, &ds)) != GEMM_OK || (st = check_on_device(buf, 4, dev)) != GEMM_OK)
        return st;
    ChooseParams p = {};
    p.logits = logits;
    p.bias = bias;
    p.ids = ids;
    p.weights = weights;
    p.tokens = tokens;
    p.ld = tokens > 1 ? ld : experts;
    p.experts = int32_t(experts);
    p.topk = int32_t(topk);
    p.groups = int32_t(groups);
    p.keep = int32_t(keep_groups);
    p.best = group_best;
    p.sigmoid = score == MOE_SCORE_SIGMOID;
    p.renormalize = renormalize != 0;
    p.scale = scale;
    const bool aligned = ((reinterpret_cast<uintptr_t>(logits) | uint64_t(p.ld * eb)) & 15u) == 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = elem_type == GEMM_OUT_F32   ? launch_choose<kOutF32>(p, aligned, ds->sms, s)
                          : elem_type == GEMM_OUT_F16 ? launch_choose<kOutF16>(p, aligned, ds->sms, s)
                                                      : launch_choose<kOutBF16>(p, aligned, ds->sms, s);
    return e == cudaSuccess ? GEMM_OK : fail_cuda(e, "choice launch");
}

gemm_status_t choose_experts_grad(const float *dweights, const void *logits, int32_t elem_type, const int32_t *ids,
                                  void *dlogits, int64_t tokens, int64_t experts, int64_t topk, int64_t ld, int64_t ld_d,
                                  int32_t score, int32_t renormalize, float scale, gemm_stream_t stream)
{
    g_last_error.clear();
    gemm_status_t st = check_choose(elem_type, tokens, experts, topk, std::min(ld, ld_d), score);
    if (st != GEMM_OK)
        return st;
    const int64_t eb = elem_bytes(elem_type);
    if (misaligned(logits, eb) || misaligned(dlogits, eb) || misaligned(ids, 4) || misaligned(dweights, 4))
        return fail(GEMM_ERR_MISALIGNED, "every buffer must sit at its elements' natural alignment");
    const Buffer buf[] = {{dweights, tokens * topk * 4, "dweights", false},
                          {logits, span(tokens, experts, ld, eb), "logits", false},
                          {ids, tokens * topk * 4, "ids", false},
                          {dlogits, span(tokens, experts, ld_d, eb), "dlogits", true}};
    if ((st = check_buffers(buf, 4)) != GEMM_OK || tokens == 0)
        return st;
    int dev = 0;
    DeviceState *ds = nullptr;
    if ((st = current(&dev, &ds)) != GEMM_OK || (st = check_on_device(buf, 4, dev)) != GEMM_OK)
        return st;
    ChooseParams p = {};
    p.logits = logits;
    p.ids = const_cast<int32_t *>(ids);
    p.dweights = dweights;
    p.dlogits = dlogits;
    p.tokens = tokens;
    p.ld = tokens > 1 ? ld : experts;
    p.ld_d = tokens > 1 ? ld_d : experts;
    p.experts = int32_t(experts);
    p.topk = int32_t(topk);
    p.groups = 1;
    p.sigmoid = score == MOE_SCORE_SIGMOID;
    p.renormalize = renormalize != 0;
    p.scale = scale;
    const bool aligned = ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(dlogits) | uint64_t(p.ld * eb) |
                           uint64_t(p.ld_d * eb)) & 15u) == 0;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const cudaError_t e = elem_type == GEMM_OUT_F32   ? launch_choose_grad<kOutF32>(p, aligned, ds->sms, s)
                          : elem_type == GEMM_OUT_F16 ? launch_choose_grad<kOutF16>(p, aligned, ds->sms, s)
                                                      : launch_choose_grad<kOutBF16>(p, aligned, ds->sms, s);
    return e == cudaSuccess ? GEMM_OK : fail_cuda(e, "choice gradient launch");
}

gemm_status_t fp4_quantize_rows(const void *X, int32_t elem_type, int32_t block, uint8_t *q, uint8_t *block_scales,
                                float *scales, const int32_t *group_rows, int64_t M, int64_t K, int64_t ldx, int64_t ldq,
                                int64_t strideX, int64_t strideQ, int64_t scale_stride, int64_t batch, gemm_stream_t stream)
{
    g_last_error.clear();
    if (!known_elem(elem_type))
        return fail(GEMM_ERR_INVALID_VALUE, "unknown element type %d", elem_type);
    if (block != 16 && block != 32)
        return fail(GEMM_ERR_INVALID_VALUE, "blocks have 16 or 32 values, not %d", block);
    if (M < 0 || K < 0 || batch < 0 || M > kInt32Max || K > kInt32Max - 65536 ||
        batch > kInt32Max)
        return fail(GEMM_ERR_INVALID_VALUE, "M and batch must be in [0, 2^31), K in [0, 2^31 - 2^16)");
    if (M > 0 && batch > kInt32Max / M)
        return fail(GEMM_ERR_INVALID_VALUE, "M x batch must be below 2^31");
    const int64_t width = (K + 1) / 2;
    if (ldx < K || ldq < width)
        return fail(GEMM_ERR_INVALID_VALUE, "a row pitch is below the row (%lld values, %lld bytes)", (long long)K, (long long)width);
    if (batch > 1 && M > 0 && (strideX < 0 || strideQ < span(M, width, ldq, 1) || (block == 16 && scale_stride < M)))
        return fail(GEMM_ERR_INVALID_VALUE, "batch strides let matrices of q or of the scales overlap");
    const int64_t eb = elem_bytes(elem_type);
    if (misaligned(X, eb) || misaligned(scales, 4) || misaligned(group_rows, 4))
        return fail(GEMM_ERR_MISALIGNED, "X, scales and group_rows must sit at their natural alignment");
    if (misaligned(block_scales, 16))
        return fail(GEMM_ERR_MISALIGNED, "block_scales must be 16-byte aligned");
    const int64_t tile_rows = scale_tile_rows(M), tile_cols = scale_tile_cols(K, block);
    const Buffer buf[] = {{X, reach(batch, strideX, M, ldx, K, eb), "X", false},
                          {group_rows, group_rows ? batch * 4 : 0, "group_rows", false},
                          {q, reach(batch, strideQ, M, ldq, width, 1), "q", true},
                          {block_scales, reach(batch, tile_rows * tile_cols, tile_rows, tile_cols, tile_cols, kScaleTile),
                           "block_scales", true},
                          {scales, block == 16 ? reach(batch, scale_stride, 1, M, M, 4) : 0, "scales", true}};
    gemm_status_t st = check_buffers(buf, 5);
    if (st != GEMM_OK || M == 0 || batch == 0)
        return st;
    int dev = 0;
    DeviceState *ds = nullptr;
    if ((st = current(&dev, &ds)) != GEMM_OK || (st = check_on_device(buf, 5, dev)) != GEMM_OK)
        return st;
    if (K == 0 && block == 32)
        return GEMM_OK;
    const Fp4QuantParams p = {X, q, block_scales, scales, group_rows, M, K, ldx, ldq, strideX, strideQ, scale_stride, batch,
                              tile_rows, tile_cols};
    const uint64_t x_all = reinterpret_cast<uintptr_t>(X) | uint64_t(M > 1 ? ldx * eb : 0) | uint64_t(batch > 1 ? strideX * eb : 0);
    const uint64_t q_all = reinterpret_cast<uintptr_t>(q) | uint64_t(M > 1 ? ldq : 0) | uint64_t(batch > 1 ? strideQ : 0);
    const cudaError_t e = launch_quantize_fp4(p, elem_type, (x_all & 15u) == 0 && (q_all & 7u) == 0, block,
                                              reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMM_OK : fail_cuda(e, "4-bit row quantisation launch");
}

}  // extern "C"

namespace tsm {
namespace {

std::once_flag g_fp4_once[64];
cudaError_t g_fp4_error[64];
Fp4Capacity g_fp4_capacity[64];

// The operands of a product, beside its Fp4Params.
struct Fp4Operands {
    const uint8_t *A, *B, *scales_a, *scales_b;
    int64_t lda, ldb, sA, sB;  // bytes
    int32_t block;
};

gemm_status_t check_fp4(const Fp4Params &p, const Fp4Operands &o, bool *trivial)
{
    *trivial = p.M == 0 || p.N == 0 || p.batch == 0;
    if (*trivial)
        return GEMM_OK;
    const int64_t width = (int64_t(p.K) + 1) / 2;
    if (p.ldc < p.N)
        return fail(GEMM_ERR_INVALID_VALUE, "ldc (%lld) < N (%d)", (long long)p.ldc, p.N);
    if (o.lda < width || o.ldb < width)
        return fail(GEMM_ERR_INVALID_VALUE, "lda (%lld) or ldb (%lld) < %lld bytes of a row", (long long)o.lda, (long long)o.ldb,
                    (long long)width);
    if (p.batch > 1 && (p.sC <= 0 || (p.K > 0 && (o.sA <= 0 || o.sB <= 0))))
        return fail(GEMM_ERR_INVALID_VALUE, "batch strides must be positive when batch > 1");
    if (p.sa_stride < 0 || p.sb_stride < 0 || p.epi.bias_stride < 0)
        return fail(GEMM_ERR_INVALID_VALUE, "scale and bias strides must be >= 0");
    const int64_t eb = p.epi.out_bytes();
    if (misaligned(p.C, eb))
        return fail(GEMM_ERR_MISALIGNED, "C must be %d-byte aligned (its elements)", int(eb));
    if (misaligned(p.scale_a, 4) || misaligned(p.scale_b, 4) || misaligned(p.epi.bias, 4) || misaligned(p.group_rows, 4))
        return fail(GEMM_ERR_MISALIGNED, "scales, bias and group_rows must be 4-byte aligned");
    if (misaligned(o.scales_a, 16) || misaligned(o.scales_b, 16))
        return fail(GEMM_ERR_MISALIGNED, "block scales must be 16-byte aligned");
    if (p.batch > 1 && p.sC < span(p.M, p.N, p.ldc, 1))
        return fail(GEMM_ERR_ALIAS, "batches of C overlap (strideC too small)");
    return GEMM_OK;
}

// All checks are done and every size is positive (K may be 0).
gemm_status_t launch_product(Fp4Params p, Fp4Operands o, DeviceState *ds, cudaStream_t stream)
{
    cudaError_t e;
    if (p.K == 0) {
        const int64_t total = int64_t(p.M) * p.N * p.batch;
        const int grid = int(std::min<int64_t>((total + 255) / 256, int64_t(ds->sms) * 8));
        e = launch_zero_fill(p.C, p.M, p.N, p.batch, p.ldc, p.sC, p.group_rows, p.epi, grid, stream);
        if (e == cudaSuccess && p.group_rows) {
            S8Params counts = {};
            counts.group_rows = p.group_rows;
            counts.batch = p.batch;
            counts.M = p.M;
            counts.status = p.status;
            e = launch_s8_counts(counts, stream);
        }
        return e == cudaSuccess ? GEMM_OK : fail_cuda(e, "4-bit product of the empty sum");
    }
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess)
        return fail_cuda(e, "cudaGetDevice");
    std::call_once(g_fp4_once[dev], [dev] { g_fp4_error[dev] = set_fp4_attributes(&g_fp4_capacity[dev]); });
    if (g_fp4_error[dev] != cudaSuccess)
        return fail_cuda(g_fp4_error[dev], "setting up the 4-bit product kernels");

    Fp4Plan plan;
    if (!plan.make(p, o.A, o.lda, o.sA, o.B, o.ldb, o.sB, ds->sms, g_fp4_capacity[dev]))
        return fail(GEMM_ERR_INVALID_VALUE, "more than 2^30 output tiles in one call");
    p.tiles_m = plan.tiles_m;
    p.tiles_n = plan.tiles_n;
    p.kb = plan.kb;
    p.workers = plan.workers;
    p.ranks = plan.ranks;
    p.sched = plan.sched;
    p.sched_price = plan.shape.price;
    p.sched_part = plan.shape.part;
    p.timeout_ns = 2000000000ull + uint64_t(p.kb) * 20000ull;
    p.tag = next_launch_epoch() >> 16;
    const int64_t tile_rows_a = scale_tile_rows(p.M), tile_rows_b = scale_tile_rows(p.N);
    const int64_t tile_cols = scale_tile_cols(p.K, o.block);
    p.scale_rows_a = int32_t(tile_rows_a);
    p.scale_rows_b = int32_t(tile_rows_b);
    p.vec_c = !misaligned(p.C, 4) && p.ldc % 2 == 0 && (p.batch == 1 || p.sC % 2 == 0);

    // Workspace: packed copies of operands that cannot be addressed, then the
    // pieces' sums and arrival words.
    char *ws = nullptr;
    const int64_t sums_at = plan.bytes_a + plan.bytes_b, words_at = sums_at + plan.bytes_p;
    if (words_at + plan.bytes_w > 0 &&
        (e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), size_t(words_at + plan.bytes_w), ds->pool, stream)) !=
            cudaSuccess)
        return fail_cuda(e, "4-bit product workspace");
    gemm_status_t st = GEMM_OK;
    const int64_t width = (int64_t(p.K) + 1) / 2;
    const auto pack = [&](const uint8_t *&x, int64_t &ld, int64_t &stride, int64_t at, int64_t ld2, int64_t rows, const char *what) {
        int8_t *to = reinterpret_cast<int8_t *>(ws + at);
        if ((e = launch_pack_s8(reinterpret_cast<const int8_t *>(x), ld, stride, to, ld2, rows * ld2, rows, width, p.batch,
                                ds->sms, stream)) != cudaSuccess)
            st = fail_cuda(e, what);
        x = reinterpret_cast<const uint8_t *>(to);
        ld = ld2;
        stride = rows * ld2;
    };
    if (plan.pack_a)
        pack(o.A, o.lda, o.sA, 0, plan.lda2, p.M, "repacking A");
    if (plan.pack_b && st == GEMM_OK)
        pack(o.B, o.ldb, o.sB, plan.bytes_a, plan.ldb2, p.N, "repacking B");
    if (plan.bytes_w && st == GEMM_OK) {
        // A captured launch is replayed with the tag it was captured with, so
        // its graph clears the words that the replay before it counted up.
        cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
        if ((e = cudaStreamIsCapturing(stream, &capturing)) != cudaSuccess)
            st = fail_cuda(e, "cudaStreamIsCapturing");
        else if (capturing != cudaStreamCaptureStatusNone &&
                 (e = cudaMemsetAsync(ws + words_at, 0, size_t(plan.bytes_w), stream)) != cudaSuccess)
            st = fail_cuda(e, "clearing the arrival words");
    }
    p.partial = reinterpret_cast<float *>(ws + sums_at);
    p.arrivals = reinterpret_cast<unsigned long long *>(ws + words_at);
    alignas(64) Fp4Maps maps;
    // (A single row or matrix may have any pitch: the map wants a multiple of 16.)
    const int64_t lda = p.M > 1 ? o.lda : round_up(o.lda, 16), ldb = p.N > 1 ? o.ldb : round_up(o.ldb, 16);
    const int64_t sA = p.batch > 1 ? o.sA : p.M * lda, sB = p.batch > 1 ? o.sB : p.N * ldb;
    const bool pair = plan.kind == Fp4Kind::kPair;
    const uint32_t box_tiles = uint32_t(kFp4BlockK / (4 * o.block));
    if (st == GEMM_OK)
        st = encode_3d(&maps.a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, o.A, width, p.M, p.batch, lda, sA, 128,
                       uint32_t(pair ? plan.shape.tile_m / 2 : plan.shape.tile_m), CU_TENSOR_MAP_L2_PROMOTION_L2_256B, "A");
    if (st == GEMM_OK)
        st = encode_3d(&maps.b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, o.B, width, p.N, p.batch, ldb, sB, 128, 128,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, "B");
    // Scale tiles: 128 words each, along k, then the rows of tiles of all matrices.
    const auto scales = [&](CUtensorMap *map, const uint8_t *x, int64_t tile_rows, uint32_t box_rows, const char *name) {
        return encode_3d(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, x, kScaleTile / 4, tile_cols, tile_rows * p.batch,
                         kScaleTile / 4, tile_cols * (kScaleTile / 4), kScaleTile / 4, box_tiles,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, name, box_rows, CU_TENSOR_MAP_SWIZZLE_NONE);
    };
    if (st == GEMM_OK)
        st = scales(&maps.scales_a, o.scales_a, tile_rows_a, pair ? 2u : 1u, "block_scales_a");
    if (st == GEMM_OK)
        st = scales(&maps.scales_b, o.scales_b, tile_rows_b, 1u, "block_scales_b");
    if (st == GEMM_OK && (e = launch_fp4(maps, p, plan.kind, o.block, plan.grid, stream)) != cudaSuccess)
        st = fail_cuda(e, "4-bit product launch");
    if (ws)
        cudaFreeAsync(ws, stream);
    return st;
}

gemm_status_t run_fp4(Fp4Params p, const Fp4Operands &o, cudaStream_t stream)
{
    bool trivial = false;
    gemm_status_t st = check_fp4(p, o, &trivial);
    if (st != GEMM_OK || trivial)
        return st;
    const int64_t width = (int64_t(p.K) + 1) / 2, tile_cols = scale_tile_cols(p.K, o.block);
    const auto tiles = [&](int64_t rows) {
        const int64_t n = scale_tile_rows(rows);
        return reach(p.batch, n * tile_cols, n, tile_cols, tile_cols, kScaleTile);
    };
    const Buffer buf[] = {
        {o.A, reach(p.batch, o.sA, p.M, o.lda, width, 1), "A", false},
        {o.B, reach(p.batch, o.sB, p.N, o.ldb, width, 1), "B", false},
        {o.scales_a, tiles(p.M), "block_scales_a", false},
        {o.scales_b, tiles(p.N), "block_scales_b", false},
        {p.scale_a, p.scale_a ? reach(p.batch, p.sa_stride, 1, p.M, p.M, 4) : 0, "scale_a", false},
        {p.scale_b, p.scale_b ? reach(p.batch, p.sb_stride, 1, p.N, p.N, 4) : 0, "scale_b", false},
        {p.epi.bias, p.epi.bias ? reach(p.batch, p.epi.bias_stride, 1, p.N, p.N, 4) : 0, "bias", false},
        {p.group_rows, p.group_rows ? int64_t(p.batch) * 4 : 0, "group_rows", false},
        {p.C, reach(p.batch, p.sC, p.M, p.ldc, p.N, p.epi.out_bytes()), "C", true}};
    if ((st = check_buffers(buf, 9)) != GEMM_OK)
        return st;
    int dev = 0;
    DeviceState *ds = nullptr;
    if ((st = current(&dev, &ds)) != GEMM_OK || (st = check_on_device(buf, 9, dev)) != GEMM_OK)
        return st;
    p.status = ds->status;
    return launch_product(p, o, ds, stream);
}

gemm_status_t fp4_call(const Fp4Operands &o, void *C, const float *scale_a, const float *scale_b, const int32_t *group_rows,
                       bool grouped, int64_t batch, int64_t M, int64_t N, int64_t K, int64_t ldc, int64_t strideC,
                       int64_t scale_a_stride, int64_t scale_b_stride, const gemm_epilogue_t *epi, cudaStream_t stream)
{
    if (M < 0 || N < 0 || K < 0 || batch < 0)
        return fail(GEMM_ERR_INVALID_VALUE, "negative size: M=%lld N=%lld K=%lld batch=%lld", (long long)M, (long long)N,
                    (long long)K, (long long)batch);
    if (o.block != 16 && o.block != 32)
        return fail(GEMM_ERR_INVALID_VALUE, "blocks have 16 or 32 values, not %d", o.block);
    // (Tile coordinates past the edges, and rows of scale tiles of all matrices, stay below 2^31.)
    if (M > kInt32Max - 512 || N > kInt32Max - 512 || batch > kInt32Max ||
        std::max(scale_tile_rows(M), scale_tile_rows(N)) * batch > kInt32Max - 512)
        return fail(GEMM_ERR_INVALID_VALUE, "M, N, batch and batch x max(M, N) / 128 must be below 2^31 - 512");
    // (The schedule counts blocks of two tiles a worker in 32 bits.)
    if (K > int64_t(1) << 23)
        return fail(GEMM_ERR_INVALID_VALUE, "K must be at most 2^23");
    if (grouped && batch > 0 && !group_rows)
        return fail(GEMM_ERR_INVALID_VALUE, "group_rows is NULL");
    Epilogue e;
    gemm_status_t st = epilogue_of(epi, &e);
    if (st != GEMM_OK)
        return st;
    Fp4Params p = {};
    p.C = C;
    p.scale_a = scale_a;
    p.scale_b = scale_b;
    p.sa_stride = scale_a_stride;
    p.sb_stride = scale_b_stride;
    p.M = int32_t(M);
    p.N = int32_t(N);
    p.K = int32_t(K);
    p.batch = int32_t(batch);
    p.ldc = ldc;
    p.sC = batch > 1 ? strideC : 0;
    p.epi = e;
    Fp4Operands x = o;
    if (batch <= 1)
        x.sA = x.sB = 0;
    if (!grouped)
        return run_fp4(p, x, stream);
    // Launches of at most kMaxGroupsPerLaunch groups, in stream order.
    const int64_t tile_cols = scale_tile_cols(K, o.block);
    for (int64_t g0 = 0; g0 < batch; g0 += kMaxGroupsPerLaunch) {
        Fp4Params q = p;
        Fp4Operands y = x;
        q.batch = int32_t(std::min<int64_t>(kMaxGroupsPerLaunch, batch - g0));
        y.A = x.A ? x.A + g0 * x.sA : x.A;
        y.B = x.B ? x.B + g0 * x.sB : x.B;
        y.scales_a = x.scales_a ? x.scales_a + g0 * scale_tile_rows(M) * tile_cols * kScaleTile : x.scales_a;
        y.scales_b = x.scales_b ? x.scales_b + g0 * scale_tile_rows(N) * tile_cols * kScaleTile : x.scales_b;
        q.C = C ? static_cast<char *>(C) + g0 * p.sC * e.out_bytes() : C;
        q.scale_a = scale_a ? scale_a + g0 * scale_a_stride : scale_a;
        q.scale_b = scale_b ? scale_b + g0 * scale_b_stride : scale_b;
        q.epi.bias = e.bias ? e.bias + g0 * e.bias_stride : e.bias;
        q.group_rows = group_rows + g0;
        if ((st = run_fp4(q, y, stream)) != GEMM_OK)
            return st;
    }
    return GEMM_OK;
}

}  // namespace
}  // namespace tsm

extern "C" {

gemm_status_t gemm_fp4_scaled(const uint8_t *A, const uint8_t *B, void *C, const uint8_t *block_scales_a,
                              const uint8_t *block_scales_b, const float *scale_a, const float *scale_b, int32_t block,
                              int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc, int64_t strideA,
                              int64_t strideB, int64_t strideC, int64_t scale_a_stride, int64_t scale_b_stride,
                              int64_t batch, const gemm_epilogue_t *epi, gemm_stream_t stream)
{
    g_last_error.clear();
    return fp4_call({A, B, block_scales_a, block_scales_b, lda, ldb, strideA, strideB, block}, C, scale_a, scale_b, nullptr, false,
                    batch, M, N, K, ldc, strideC, scale_a_stride, scale_b_stride, epi, reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_fp4_grouped_scaled(const uint8_t *A, const uint8_t *B, void *C, const uint8_t *block_scales_a,
                                      const uint8_t *block_scales_b, const float *scale_a, const float *scale_b,
                                      int32_t block, const int32_t *group_rows, int64_t groups, int64_t M, int64_t N,
                                      int64_t K, int64_t lda, int64_t ldb, int64_t ldc, int64_t strideA, int64_t strideB,
                                      int64_t strideC, int64_t scale_a_stride, int64_t scale_b_stride,
                                      const gemm_epilogue_t *epi, gemm_stream_t stream)
{
    g_last_error.clear();
    return fp4_call({A, B, block_scales_a, block_scales_b, lda, ldb, strideA, strideB, block}, C, scale_a, scale_b, group_rows,
                    true, groups, M, N, K, ldc, strideC, scale_a_stride, scale_b_stride, epi,
                    reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
