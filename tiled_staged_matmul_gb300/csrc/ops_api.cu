// ops_api.cu -- host side of the expert token movement and of the 8-bit
// integer products (include/tsm_gemm.h): argument checks, launch shapes and
// launches.
#include "api_internal.h"
#include "ops_internal.h"
#include "s8_plan.h"

#include <algorithm>
#include <mutex>

namespace tsm {
namespace {

constexpr int64_t kInt32Max = 2147483647;
constexpr int64_t kMaxSize = int64_t(1) << 40;

bool misaligned(const void *p, int64_t bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & uintptr_t(bytes - 1)) != 0;
}

int elem_bytes(int32_t t) { return t == GEMM_OUT_F32 ? 4 : 2; }

bool known_elem(int32_t t) { return t == GEMM_OUT_F32 || t == GEMM_OUT_F16 || t == GEMM_OUT_BF16; }

// The current device and its state.
gemm_status_t current(int *dev, DeviceState **ds)
{
    const cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess)
        return fail_cuda(e, "cudaGetDevice");
    return device_state(*dev, ds);
}

// One buffer of a call: checked for its address and, once all are known, on
// the device.
struct Buffer {
    const void *p;
    int64_t bytes;
    const char *name;
    bool written;
};

// Every buffer non-null where it holds something, no written one overlapping
// another.
gemm_status_t check_buffers(const Buffer *b, int n)
{
    for (int i = 0; i < n; ++i)
        if (b[i].bytes > 0 && !b[i].p)
            return fail(GEMM_ERR_INVALID_VALUE, "%s is NULL", b[i].name);
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if ((b[i].written || b[j].written) && overlaps(b[i].p, b[i].bytes, b[j].p, b[j].bytes))
                return fail(GEMM_ERR_ALIAS, "%s overlaps %s", b[i].name, b[j].name);
    return GEMM_OK;
}

gemm_status_t check_on_device(const Buffer *b, int n, int dev)
{
    for (int i = 0; i < n; ++i)
        if (b[i].bytes > 0) {
            const gemm_status_t st = check_device_pointer(b[i].p, b[i].bytes, dev, b[i].name);
            if (st != GEMM_OK)
                return st;
        }
    return GEMM_OK;
}

// Bytes spanned by `batch` matrices `stride` elements apart of `rows` rows `ld`
// apart.  More than 64 bits hold come out as the most that they hold, which
// lies in no allocation.
int64_t reach(int64_t batch, int64_t stride, int64_t rows, int64_t ld, int64_t cols, int64_t elem)
{
    if (batch <= 0 || rows <= 0 || cols <= 0)
        return 0;
    const __int128 bytes = (__int128(batch - 1) * stride + __int128(rows - 1) * ld + cols) * elem;
    return bytes > INT64_MAX ? INT64_MAX : int64_t(bytes);
}

// Bytes of `rows` rows of `width` elements `ld` apart.
int64_t span(int64_t rows, int64_t width, int64_t ld, int64_t elem) { return reach(1, 0, rows, ld, width, elem); }

// Bytes of one access: 16 or 4 where every address, pitch and width in `all`
// (or-ed together, in bytes) is a multiple, else one element.
int access_bytes(uint64_t all, int64_t elem)
{
    return (all & 15u) == 0 ? 16 : (all & 3u) == 0 ? 4 : int(elem);
}

// What the four movement calls share: sizes of both sides and the slots.
gemm_status_t check_move(int64_t tokens, int64_t topk, int64_t rows, int64_t width, int64_t ld_tokens,
                         int64_t ld_rows)
{
    if (tokens < 0 || topk < 0 || rows < 0 || width < 0)
        return fail(GEMM_ERR_INVALID_VALUE, "negative size: tokens=%lld topk=%lld rows=%lld width=%lld",
                    (long long)tokens, (long long)topk, (long long)rows, (long long)width);
    if (tokens > kInt32Max || topk > kInt32Max || rows > kInt32Max || width > kInt32Max ||
        tokens * topk > kMaxSize)
        return fail(GEMM_ERR_INVALID_VALUE, "tokens, topk, rows and width must be below 2^31");
    if (ld_tokens < width || ld_rows < width)
        return fail(GEMM_ERR_INVALID_VALUE, "a row pitch is below the width (%lld)", (long long)width);
    return GEMM_OK;
}

}  // namespace
}  // namespace tsm

using namespace tsm;

extern "C" {

gemm_status_t moe_route_slots(const void *expert_ids, int32_t id_bytes, int32_t *slots, int32_t *counts, int64_t tokens,
                        int64_t topk, int64_t groups, int64_t capacity, gemm_stream_t stream)
{
    g_last_error.clear();
    if (id_bytes != 4 && id_bytes != 8)
        return fail(GEMM_ERR_INVALID_VALUE, "expert ids have 4 or 8 bytes, not %d", id_bytes);
    if (tokens < 0 || topk < 0 || groups < 0 || capacity < 0)
        return fail(GEMM_ERR_INVALID_VALUE, "negative size: tokens=%lld topk=%lld groups=%lld capacity=%lld",
                    (long long)tokens, (long long)topk, (long long)groups, (long long)capacity);
    if (groups > kMaxRouteGroups)
        return fail(GEMM_ERR_INVALID_VALUE, "at most %d groups, not %lld", kMaxRouteGroups, (long long)groups);
    if (tokens > kInt32Max || topk > kInt32Max || tokens * topk > kInt32Max)
        return fail(GEMM_ERR_INVALID_VALUE, "tokens x topk must be below 2^31");
    if (capacity > kInt32Max || groups * capacity > kInt32Max)
        return fail(GEMM_ERR_INVALID_VALUE, "groups x capacity must be below 2^31");
    const int64_t n = tokens * topk;
    if (misaligned(expert_ids, id_bytes) || misaligned(slots, 4) || misaligned(counts, 4))
        return fail(GEMM_ERR_MISALIGNED, "ids, slots and counts must sit at their natural alignment");
    const Buffer buf[] = {{expert_ids, n * id_bytes, "expert_ids", false},
                          {slots, n * 4, "slots", true},
                          {counts, groups * 4, "counts", true}};
    gemm_status_t st = check_buffers(buf, 3);
    if (st != GEMM_OK || (n == 0 && groups == 0))
        return st;
    int dev = 0;
    DeviceState *ds = nullptr;
    if ((st = current(&dev, &ds)) != GEMM_OK || (st = check_on_device(buf, 3, dev)) != GEMM_OK)
        return st;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // One cluster while it holds the chunks.  Else small chunks until they would
    // be many: each rank block adds up the counts of the chunks before its own.
    int rounds = kRouteRoundsSmall;
    while (rounds < kRouteRoundsCluster && n > route_chunk(rounds) * kRouteCluster)
        rounds *= 2;
    const bool cluster = n <= route_chunk(rounds) * kRouteCluster;
    if (!cluster)
        rounds = n > route_chunk(kRouteRoundsSmall) * ds->sms ? kRouteRoundsLarge : kRouteRoundsSmall;
    const int64_t chunks = std::max<int64_t>(1, (n + route_chunk(rounds) - 1) / route_chunk(rounds));
    RouteParams p = {};
    p.ids = expert_ids;
    p.slots = slots;
    p.counts = counts;
    p.n = n;
    p.groups = int32_t(groups);
    p.capacity = int32_t(capacity);
    void *ws = nullptr;
    cudaError_t e;
    if (!cluster) {
        if ((e = cudaMallocFromPoolAsync(&ws, size_t(chunks * std::max<int64_t>(groups, 1) * 4), ds->pool, s)) !=
            cudaSuccess)
            return fail_cuda(e, "routing workspace");
        p.hist = static_cast<int32_t *>(ws);
    }
    if ((e = launch_route(p, id_bytes == 8, rounds, chunks, s)) != cudaSuccess)
        st = fail_cuda(e, "routing launch");
    if (ws)
        cudaFreeAsync(ws, s);
    return st;
}

gemm_status_t moe_dispatch_rows(const void *x, int32_t elem_bytes_, const int32_t *slots, void *rows_out, int64_t tokens,
                           int64_t topk, int64_t rows, int64_t width, int64_t ldx, int64_t ld_rows,
                           gemm_stream_t stream)
{
    g_last_error.clear();
    const int64_t eb = elem_bytes_;
    if (eb != 1 && eb != 2 && eb != 4)
        return fail(GEMM_ERR_INVALID_VALUE, "elements have 1, 2 or 4 bytes, not %d", elem_bytes_);
    gemm_status_t st = check_move(tokens, topk, rows, width, ldx, ld_rows);
    if (st != GEMM_OK)
        return st;
    if (misaligned(x, eb) || misaligned(rows_out, eb) || misaligned(slots, 4))
        return fail(GEMM_ERR_MISALIGNED, "x, rows and slots must sit at their natural alignment");
    const Buffer buf[] = {{x, span(tokens, width, ldx, eb), "x", false},
                          {slots, width ? tokens * topk * 4 : 0, "slots", false},
                          {rows_out, span(rows, width, ld_rows, eb), "rows", true}};
    if ((st = check_buffers(buf, 3)) != GEMM_OK || tokens == 0 || topk == 0 || width == 0 || rows == 0)
        return st;
    int dev = 0;
    DeviceState *ds = nullptr;
    if ((st = current(&dev, &ds)) != GEMM_OK || (st = check_on_device(buf, 3, dev)) != GEMM_OK)
        return st;
    // The widest unit that divides both bases, both pitches and the width.
    int64_t vec = 16;
    const uint64_t all = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(rows_out) |
                         uint64_t(width * eb) | uint64_t(tokens > 1 ? ldx * eb : 0) | uint64_t(ld_rows * eb);
    while (all & uint64_t(vec - 1))
        vec /= 2;
    MoveParams p = {};
    p.src = x;
    p.dst = rows_out;
    p.slots = slots;
    p.tokens = tokens;
    p.topk = topk;
    p.rows = rows;
    p.width = width * eb / vec;
    p.ld_src = tokens > 1 ? ldx * eb / vec : p.width;
    p.ld_dst = ld_rows * eb / vec;
    const cudaError_t e = launch_dispatch(p, int(vec), ds->sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMM_OK : fail_cuda(e, "dispatch launch");
}

}  // extern "C"

namespace tsm {
namespace {

gemm_status_t combine(const void *rows_in, int32_t elem_type, const int32_t *slots, const float *weights, void *out,
                      int64_t tokens, int64_t topk, int64_t rows, int64_t width, int64_t ld_rows, int64_t ld_out,
                      cudaStream_t stream)
{
    if (!known_elem(elem_type))
        return fail(GEMM_ERR_INVALID_VALUE, "unknown element type %d", elem_type);
    gemm_status_t st = check_move(tokens, topk, rows, width, ld_out, ld_rows);
    if (st != GEMM_OK)
        return st;
    const int64_t eb = elem_bytes(elem_type);
    if (misaligned(rows_in, eb) || misaligned(out, eb) || misaligned(slots, 4) || misaligned(weights, 4))
        return fail(GEMM_ERR_MISALIGNED, "every buffer must sit at its elements' natural alignment");
    const Buffer buf[] = {{rows_in, span(rows, width, ld_rows, eb), "rows", false},
                          {slots, width ? tokens * topk * 4 : 0, "slots", false},
                          {weights, weights && width ? tokens * topk * 4 : 0, "weights", false},
                          {out, span(tokens, width, ld_out, eb), "out", true}};
    if ((st = check_buffers(buf, 4)) != GEMM_OK || tokens == 0 || width == 0)
        return st;
    int dev = 0;
    DeviceState *ds = nullptr;
    if ((st = current(&dev, &ds)) != GEMM_OK || (st = check_on_device(buf, 4, dev)) != GEMM_OK)
        return st;
    const uint64_t all = reinterpret_cast<uintptr_t>(rows_in) | reinterpret_cast<uintptr_t>(out) |
                         uint64_t(width * eb) | uint64_t(tokens > 1 ? ld_out * eb : 0) | uint64_t(ld_rows * eb);
    MoveParams p = {};
    p.src = rows_in;
    p.dst = out;
    p.slots = slots;
    p.weights = weights;
    p.tokens = tokens;
    p.topk = topk;
    p.rows = rows;
    p.width = width;
    p.ld_src = ld_rows;
    p.ld_dst = ld_out;
    const cudaError_t e = launch_combine(p, elem_type, access_bytes(all, eb), ds->sms, stream);
    return e == cudaSuccess ? GEMM_OK : fail_cuda(e, "combine launch");
}

}  // namespace
}  // namespace tsm

extern "C" {

gemm_status_t moe_dispatch_rows_grad(const void *drows, int32_t elem_type, const int32_t *slots, void *dx, int64_t tokens,
                                int64_t topk, int64_t rows, int64_t width, int64_t ld_rows, int64_t ldx,
                                gemm_stream_t stream)
{
    g_last_error.clear();
    return combine(drows, elem_type, slots, nullptr, dx, tokens, topk, rows, width, ld_rows, ldx,
                   reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t moe_combine_rows(const void *rows_in, int32_t elem_type, const int32_t *slots, const float *weights,
                          void *out, int64_t tokens, int64_t topk, int64_t rows, int64_t width, int64_t ld_rows,
                          int64_t ld_out, gemm_stream_t stream)
{
    g_last_error.clear();
    return combine(rows_in, elem_type, slots, weights, out, tokens, topk, rows, width, ld_rows, ld_out,
                   reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t moe_combine_rows_grad(const void *dout, const void *rows_in, int32_t elem_type, const int32_t *slots,
                               const float *weights, void *drows, float *dweights, int64_t tokens, int64_t topk,
                               int64_t rows, int64_t width, int64_t ld_dout, int64_t ld_rows, int64_t ld_drows,
                               gemm_stream_t stream)
{
    g_last_error.clear();
    if (!known_elem(elem_type))
        return fail(GEMM_ERR_INVALID_VALUE, "unknown element type %d", elem_type);
    gemm_status_t st = check_move(tokens, topk, rows, width, ld_dout, std::min(ld_rows, ld_drows));
    if (st != GEMM_OK)
        return st;
    const int64_t eb = elem_bytes(elem_type);
    if (misaligned(dout, eb) || misaligned(rows_in, eb) || misaligned(drows, eb) || misaligned(slots, 4) ||
        misaligned(weights, 4) || misaligned(dweights, 4))
        return fail(GEMM_ERR_MISALIGNED, "every buffer must sit at its elements' natural alignment");
    const int64_t n4 = tokens * topk * 4;
    const Buffer buf[] = {{dout, span(tokens, width, ld_dout, eb), "dout", false},
                          {rows_in, span(rows, width, ld_rows, eb), "rows", false},
                          {slots, n4, "slots", false},
                          {weights, weights ? n4 : 0, "weights", false},
                          {drows, span(rows, width, ld_drows, eb), "drows", true},
                          {dweights, dweights ? n4 : 0, "dweights", true}};
    if ((st = check_buffers(buf, 6)) != GEMM_OK || tokens == 0 || topk == 0)
        return st;
    int dev = 0;
    DeviceState *ds = nullptr;
    if ((st = current(&dev, &ds)) != GEMM_OK || (st = check_on_device(buf, 6, dev)) != GEMM_OK)
        return st;
    const uint64_t all = reinterpret_cast<uintptr_t>(rows_in) | reinterpret_cast<uintptr_t>(drows) |
                         reinterpret_cast<uintptr_t>(dout) | uint64_t(width * eb) |
                         uint64_t(tokens > 1 ? ld_dout * eb : 0) | uint64_t(ld_rows * eb) | uint64_t(ld_drows * eb);
    MoveParams p = {};
    p.src = rows_in;
    p.dst = drows;
    p.dout = dout;
    p.slots = slots;
    p.weights = weights;
    p.dweights = dweights;
    p.tokens = tokens;
    p.topk = topk;
    p.rows = width ? rows : 0;
    p.width = width;
    p.ld_src = ld_rows;
    p.ld_dst = ld_drows;
    p.ld_dout = ld_dout;
    const cudaError_t e = launch_combine_grad(p, elem_type, access_bytes(all, eb), ds->sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMM_OK : fail_cuda(e, "combine gradient launch");
}

gemm_status_t quantize_rows_s8(const void *X, int32_t elem_type, int8_t *q, float *scales, const int32_t *group_rows,
                               int64_t M, int64_t K, int64_t ldx, int64_t ldq, int64_t strideX, int64_t strideQ,
                               int64_t scale_stride, int64_t batch, gemm_stream_t stream)
{
    g_last_error.clear();
    if (!known_elem(elem_type))
        return fail(GEMM_ERR_INVALID_VALUE, "unknown element type %d", elem_type);
    if (M < 0 || K < 0 || batch < 0 || M > kInt32Max || K > kInt32Max || batch > kInt32Max)
        return fail(GEMM_ERR_INVALID_VALUE, "M, K and batch must be in [0, 2^31)");
    if (M > 0 && batch > kInt32Max / M)
        return fail(GEMM_ERR_INVALID_VALUE, "M x batch must be below 2^31");
    if (ldx < K || ldq < K)
        return fail(GEMM_ERR_INVALID_VALUE, "a row pitch is below K (%lld)", (long long)K);
    if (batch > 1 && M > 0 && (strideX < 0 || strideQ < span(M, K, ldq, 1) || scale_stride < M))
        return fail(GEMM_ERR_INVALID_VALUE, "batch strides let matrices of q or of the scales overlap");
    const int64_t eb = elem_bytes(elem_type);
    if (misaligned(X, eb) || misaligned(scales, 4) || misaligned(group_rows, 4))
        return fail(GEMM_ERR_MISALIGNED, "X, scales and group_rows must sit at their natural alignment");
    const Buffer buf[] = {{X, reach(batch, strideX, M, ldx, K, eb), "X", false},
                          {group_rows, group_rows ? batch * 4 : 0, "group_rows", false},
                          {q, reach(batch, strideQ, M, ldq, K, 1), "q", true},
                          {scales, reach(batch, scale_stride, 1, M, M, 4), "scales", true}};
    gemm_status_t st = check_buffers(buf, 4);
    if (st != GEMM_OK || M == 0 || batch == 0)
        return st;
    int dev = 0;
    DeviceState *ds = nullptr;
    if ((st = current(&dev, &ds)) != GEMM_OK || (st = check_on_device(buf, 4, dev)) != GEMM_OK)
        return st;
    QuantParams p = {X, q, scales, group_rows, M, K, ldx, ldq, strideX, strideQ, scale_stride, batch};
    // (A piece's codes are as many bytes as it has elements.)
    const uint64_t x_all = reinterpret_cast<uintptr_t>(X) | uint64_t(K * eb) | uint64_t(M > 1 ? ldx * eb : 0) |
                           uint64_t(batch > 1 ? strideX * eb : 0);
    const uint64_t q_all = reinterpret_cast<uintptr_t>(q) | uint64_t(M > 1 ? ldq : 0) | uint64_t(batch > 1 ? strideQ : 0);
    const int bytes = access_bytes(x_all | q_all * uint64_t(eb), eb);
    const cudaError_t e = launch_quantize_rows(p, elem_type, bytes, ds->sms, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? GEMM_OK : fail_cuda(e, "row quantisation launch");
}

}  // extern "C"

namespace tsm {
namespace {

gemm_status_t check_s8(const S8Params &p, bool *trivial)
{
    *trivial = p.M == 0 || p.N == 0 || p.batch == 0;
    if (*trivial)
        return GEMM_OK;
    if (p.ldc < p.N)
        return fail(GEMM_ERR_INVALID_VALUE, "ldc (%lld) < N (%d)", (long long)p.ldc, p.N);
    if (p.K > 0 && p.lda < p.K)
        return fail(GEMM_ERR_INVALID_VALUE, "lda (%lld) < K (%d)", (long long)p.lda, p.K);
    if (p.K > 0 && p.ldb < p.N)
        return fail(GEMM_ERR_INVALID_VALUE, "ldb (%lld) < N (%d)", (long long)p.ldb, p.N);
    if (p.batch > 1 && (p.sC <= 0 || (p.K > 0 && (p.sA <= 0 || p.sB <= 0))))
        return fail(GEMM_ERR_INVALID_VALUE, "batch strides must be positive when batch > 1");
    if (p.sa_stride < 0 || p.sb_stride < 0 || p.epi.bias_stride < 0)
        return fail(GEMM_ERR_INVALID_VALUE, "scale and bias strides must be >= 0");
    const int64_t eb = p.epi.out_bytes();
    if (misaligned(p.C, eb))
        return fail(GEMM_ERR_MISALIGNED, "C must be %d-byte aligned (its elements)", int(eb));
    if (misaligned(p.scale_a, 4) || misaligned(p.scale_b, 4) || misaligned(p.epi.bias, 4) ||
        misaligned(p.group_rows, 4))
        return fail(GEMM_ERR_MISALIGNED, "scales, bias and group_rows must be 4-byte aligned");
    if (p.batch > 1 && p.sC < span(p.M, p.N, p.ldc, 1))
        return fail(GEMM_ERR_ALIAS, "batches of C overlap (strideC too small)");
    return GEMM_OK;
}

std::once_flag g_s8_once[64];
cudaError_t g_s8_error[64];
S8Capacity g_s8_capacity[64];

// All checks are done and every size is positive (K may be 0).
gemm_status_t launch_product(S8Params p, DeviceState *ds, cudaStream_t stream)
{
    cudaError_t e;
    if (p.K == 0) {
        const int64_t total = int64_t(p.M) * p.N * p.batch;
        const int grid = int(std::min<int64_t>((total + 255) / 256, int64_t(ds->sms) * 8));
        e = launch_zero_fill(p.C, p.M, p.N, p.batch, p.ldc, p.sC, p.group_rows, p.epi, grid, stream);
        if (e == cudaSuccess && p.group_rows)
            e = launch_s8_counts(p, stream);
        return e == cudaSuccess ? GEMM_OK : fail_cuda(e, "int8 product of the empty sum");
    }
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess)
        return fail_cuda(e, "cudaGetDevice");
    std::call_once(g_s8_once[dev], [dev] { g_s8_error[dev] = set_s8_attributes(&g_s8_capacity[dev]); });
    if (g_s8_error[dev] != cudaSuccess)
        return fail_cuda(g_s8_error[dev], "setting up the int8 product kernels");

    S8Plan plan;
    if (!plan.make(p, ds->sms, g_s8_capacity[dev]))
        return fail(GEMM_ERR_INVALID_VALUE, "more than 2^30 output tiles in one call");
    const S8Shape shape = plan.shape;
    const bool few = plan.few();
    p.tiles_m = plan.tiles_m;
    p.tiles_n = plan.tiles_n;
    p.kb = plan.kb;
    p.workers = plan.workers;
    p.ranks = plan.ranks;
    p.kb_each = plan.kb / plan.ranks;
    p.kb_more = plan.kb % plan.ranks;
    p.sched = plan.sched;
    p.timeout_ns = 2000000000ull + uint64_t(p.kb) * 20000ull;
    p.tag = next_launch_epoch() >> 16;
    const int64_t per16 = 16 / p.epi.out_bytes();
    p.vec_c = !misaligned(p.C, 16) && p.ldc % per16 == 0 && (p.batch == 1 || p.sC % per16 == 0);

    // Workspace: packed copies of operands that cannot be addressed, then the
    // pieces' sums and arrival words.
    const int64_t bytes_a = plan.bytes_a, bytes_b = plan.bytes_b, bytes_p = plan.bytes_p, bytes_w = plan.bytes_w;
    const int64_t lda2 = plan.lda2, ldb2 = plan.ldb2;
    char *ws = nullptr;
    if (bytes_a + bytes_b + bytes_p + bytes_w > 0 &&
        (e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), size_t(bytes_a + bytes_b + bytes_p + bytes_w),
                                     ds->pool, stream)) != cudaSuccess)
        return fail_cuda(e, "int8 product workspace");
    gemm_status_t st = GEMM_OK;
    if (plan.pack_a) {
        int8_t *to = reinterpret_cast<int8_t *>(ws);
        if ((e = launch_pack_s8(p.A, p.lda, p.sA, to, lda2, p.M * lda2, p.M, p.K, p.batch, ds->sms, stream)) !=
            cudaSuccess)
            st = fail_cuda(e, "repacking A");
        p.A = to;
        p.lda = lda2;
        p.sA = p.M * lda2;
    }
    if (plan.pack_b && st == GEMM_OK) {
        int8_t *to = reinterpret_cast<int8_t *>(ws + bytes_a);
        if ((e = launch_pack_s8(p.B, p.ldb, p.sB, to, ldb2, p.K * ldb2, p.K, p.N, p.batch, ds->sms, stream)) !=
            cudaSuccess)
            st = fail_cuda(e, "repacking B");
        p.B = to;
        p.ldb = ldb2;
        p.sB = p.K * ldb2;
    }
    if (bytes_w && st == GEMM_OK) {
        // A captured launch is replayed with the tag it was captured with, so
        // its graph clears the words that the replay before it counted up.
        cudaStreamCaptureStatus capturing = cudaStreamCaptureStatusNone;
        if ((e = cudaStreamIsCapturing(stream, &capturing)) != cudaSuccess)
            st = fail_cuda(e, "cudaStreamIsCapturing");
        else if (capturing != cudaStreamCaptureStatusNone &&
                 (e = cudaMemsetAsync(ws + bytes_a + bytes_b + bytes_p, 0, size_t(bytes_w), stream)) != cudaSuccess)
            st = fail_cuda(e, "clearing the arrival words");
    }
    p.partial = reinterpret_cast<int32_t *>(ws + bytes_a + bytes_b);
    p.arrivals = reinterpret_cast<unsigned long long *>(ws + bytes_a + bytes_b + bytes_p);
    alignas(64) CUtensorMap map_a, map_b;
    // (A single row or matrix may have any pitch: the map wants a multiple of 16.)
    const int64_t lda = p.M > 1 ? p.lda : round_up(p.lda, 16), ldb = p.K > 1 ? p.ldb : round_up(p.ldb, 16);
    const int64_t sA = p.batch > 1 ? p.sA : p.M * lda, sB = p.batch > 1 ? p.sB : p.K * ldb;
    if (st == GEMM_OK)
        st = encode_3d(&map_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.A, p.K, p.M, p.batch, lda, sA,
                       uint32_t(shape.block_k), few ? uint32_t(shape.tile_m) : 128u,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, "A", 1,
                       few ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B);
    if (st == GEMM_OK)
        st = encode_3d(&map_b, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p.B, p.N, p.K, p.batch, ldb, sB, 128, uint32_t(shape.block_k),
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, "B");
    if (st == GEMM_OK) {
        e = launch_s8(map_a, map_b, p, plan.kind, plan.grid, stream);
        if (e != cudaSuccess)
            st = fail_cuda(e, "int8 product launch");
    }
    if (ws)
        cudaFreeAsync(ws, stream);
    return st;
}

gemm_status_t run_s8(S8Params p, cudaStream_t stream)
{
    bool trivial = false;
    gemm_status_t st = check_s8(p, &trivial);
    if (st != GEMM_OK || trivial)
        return st;
    const Buffer buf[] = {
        {p.A, p.K ? reach(p.batch, p.sA, p.M, p.lda, p.K, 1) : 0, "A", false},
        {p.B, p.K ? reach(p.batch, p.sB, p.K, p.ldb, p.N, 1) : 0, "B", false},
        {p.scale_a, p.scale_a ? reach(p.batch, p.sa_stride, 1, p.M, p.M, 4) : 0, "scale_a", false},
        {p.scale_b, p.scale_b ? reach(p.batch, p.sb_stride, 1, p.N, p.N, 4) : 0, "scale_b", false},
        {p.epi.bias, p.epi.bias ? reach(p.batch, p.epi.bias_stride, 1, p.N, p.N, 4) : 0, "bias", false},
        {p.group_rows, p.group_rows ? int64_t(p.batch) * 4 : 0, "group_rows", false},
        {p.C, reach(p.batch, p.sC, p.M, p.ldc, p.N, p.epi.out_bytes()), "C", true}};
    if ((st = check_buffers(buf, 7)) != GEMM_OK)
        return st;
    int dev = 0;
    DeviceState *ds = nullptr;
    if ((st = current(&dev, &ds)) != GEMM_OK || (st = check_on_device(buf, 7, dev)) != GEMM_OK)
        return st;
    p.status = ds->status;
    return launch_product(p, ds, stream);
}

gemm_status_t s8_call(const int8_t *A, const int8_t *B, void *C, const float *scale_a, const float *scale_b,
                      const int32_t *group_rows, bool grouped, int64_t batch, int64_t M, int64_t N, int64_t K,
                      int64_t lda, int64_t ldb, int64_t ldc, int64_t strideA, int64_t strideB, int64_t strideC,
                      int64_t scale_a_stride, int64_t scale_b_stride, const gemm_epilogue_t *epi,
                      cudaStream_t stream)
{
    if (M < 0 || N < 0 || K < 0 || batch < 0)
        return fail(GEMM_ERR_INVALID_VALUE, "negative size: M=%lld N=%lld K=%lld batch=%lld", (long long)M,
                    (long long)N, (long long)K, (long long)batch);
    // (Tile coordinates past the edges stay below 2^31.)
    if (M > kInt32Max - 512 || N > kInt32Max - 512 || batch > kInt32Max)
        return fail(GEMM_ERR_INVALID_VALUE, "M and N must be below 2^31 - 512, batch below 2^31");
    // |S| <= 128 * 128 * K has to fit 32 bits.
    if (K > 131071)
        return fail(GEMM_ERR_INVALID_VALUE, "K must be below 131072: longer sums can pass 32 bits");
    if (grouped && batch > 0 && !group_rows)
        return fail(GEMM_ERR_INVALID_VALUE, "group_rows is NULL");
    Epilogue e;
    gemm_status_t st = epilogue_of(epi, &e);
    if (st != GEMM_OK)
        return st;
    S8Params p = {};
    p.A = A;
    p.B = B;
    p.C = C;
    p.scale_a = scale_a;
    p.scale_b = scale_b;
    p.sa_stride = scale_a_stride;
    p.sb_stride = scale_b_stride;
    p.M = int32_t(M);
    p.N = int32_t(N);
    p.K = int32_t(K);
    p.batch = int32_t(batch);
    p.lda = lda;
    p.ldb = ldb;
    p.ldc = ldc;
    p.sA = batch > 1 ? strideA : 0;
    p.sB = batch > 1 ? strideB : 0;
    p.sC = batch > 1 ? strideC : 0;
    p.epi = e;
    if (!grouped)
        return run_s8(p, stream);
    // Launches of at most kMaxGroupsPerLaunch groups, in stream order.
    for (int64_t g0 = 0; g0 < batch; g0 += kMaxGroupsPerLaunch) {
        S8Params q = p;
        q.batch = int32_t(std::min<int64_t>(kMaxGroupsPerLaunch, batch - g0));
        q.A = A ? A + g0 * p.sA : A;
        q.B = B ? B + g0 * p.sB : B;
        q.C = C ? static_cast<char *>(C) + g0 * p.sC * e.out_bytes() : C;
        q.scale_a = scale_a ? scale_a + g0 * scale_a_stride : scale_a;
        q.scale_b = scale_b ? scale_b + g0 * scale_b_stride : scale_b;
        q.epi.bias = e.bias ? e.bias + g0 * e.bias_stride : e.bias;
        q.group_rows = group_rows + g0;
        if ((st = run_s8(q, stream)) != GEMM_OK)
            return st;
    }
    return GEMM_OK;
}

}  // namespace
}  // namespace tsm

extern "C" {

gemm_status_t gemm_s8_scaled(const int8_t *A, const int8_t *B, void *C, const float *scale_a, const float *scale_b,
                             int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc, int64_t strideA,
                             int64_t strideB, int64_t strideC, int64_t scale_a_stride, int64_t scale_b_stride,
                             int64_t batch, const gemm_epilogue_t *epi, gemm_stream_t stream)
{
    g_last_error.clear();
    return s8_call(A, B, C, scale_a, scale_b, nullptr, false, batch, M, N, K, lda, ldb, ldc, strideA, strideB,
                   strideC, scale_a_stride, scale_b_stride, epi, reinterpret_cast<cudaStream_t>(stream));
}

gemm_status_t gemm_s8_grouped_scaled(const int8_t *A, const int8_t *B, void *C, const float *scale_a,
                                     const float *scale_b, const int32_t *group_rows, int64_t groups, int64_t M,
                                     int64_t N, int64_t K, int64_t lda, int64_t ldb, int64_t ldc, int64_t strideA,
                                     int64_t strideB, int64_t strideC, int64_t scale_a_stride,
                                     int64_t scale_b_stride, const gemm_epilogue_t *epi, gemm_stream_t stream)
{
    g_last_error.clear();
    return s8_call(A, B, C, scale_a, scale_b, group_rows, true, groups, M, N, K, lda, ldb, ldc, strideA, strideB,
                   strideC, scale_a_stride, scale_b_stride, epi, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
