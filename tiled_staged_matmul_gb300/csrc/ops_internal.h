// ops_internal.h -- what ops_api.cu and the kernels of the expert token
// movement (moe_kernels.cu) and of the 8-bit integer products
// (s8_kernels.cu) share.  Not part of the public ABI.
#pragma once

#include "gemm_internal.h"

namespace tsm {

// ------------------------------------------------------------- token movement

constexpr int kMaxRouteGroups = 1024;  // experts of one routing call (shared-memory counters)

struct RouteParams {
    const void *ids;      // n expert numbers, int32 or int64
    int32_t *slots;       // n
    int32_t *counts;      // groups
    int32_t *hist;        // chunks x groups counts per chunk (more than one chunk), else null
    int64_t n;            // tokens x choices
    int32_t groups;
    int32_t capacity;
};
// One CTA ranks kRouteChunk(rounds) assignments.
constexpr int kRouteWarps = 16;
constexpr int kRouteRoundsSmall = 2, kRouteRoundsLarge = 16;
__host__ __device__ constexpr int64_t route_chunk(int rounds) { return int64_t(kRouteWarps) * 32 * rounds; }
cudaError_t launch_route(const RouteParams &p, bool wide_ids, int rounds, int64_t chunks, cudaStream_t stream);

// Token rows <-> expert rows.  Row r of the experts' side is base + r * ld;
// slots[t * topk + j] names the row of token t's j-th choice, -1 for none.
struct MoveParams {
    const void *src;        // dispatch: tokens; combine: experts' rows; combine_grad: experts' rows
    void *dst;              // dispatch: experts' rows; combine: tokens; combine_grad: experts' row gradients
    const void *dout;       // combine_grad: the tokens' gradient
    const int32_t *slots;
    const float *weights;   // null: all ones
    float *dweights;        // combine_grad
    int64_t tokens;
    int64_t topk;
    int64_t rows;           // rows on the experts' side (a slot at or past it is skipped)
    int64_t width;          // elements (dispatch: units of the vector width)
    int64_t ld_src, ld_dst, ld_dout;  // row pitches, elements (dispatch: vector units)
};
// dispatch moves whole rows as units of `vec` bytes (16, 8, 4, 2 or 1).
cudaError_t launch_dispatch(const MoveParams &p, int vec, int sms, cudaStream_t stream);
// `vec`: 16-byte accesses (every row 16-byte aligned), else element by element.
cudaError_t launch_combine(const MoveParams &p, int elem, bool vec, int sms, cudaStream_t stream);
cudaError_t launch_combine_grad(const MoveParams &p, int elem, bool vec, cudaStream_t stream);

// ------------------------------------------------------------- row quantisation

struct QuantParams {
    const void *X;           // batch x M rows of K, ldx / strideX apart
    int8_t *q;               // ldq / strideQ apart
    float *scales;           // batch x M, stride_s apart
    const int32_t *group_rows;  // null, or the rows of each batch that are computed
    int64_t M, K, ldx, ldq, sX, sQ, sS, batch;
};
cudaError_t launch_quantize_rows(const QuantParams &p, int elem, bool vec, cudaStream_t stream);

// ------------------------------------------------------------- int8 products

struct S8Params {
    const int8_t *A, *B;
    void *C;                  // epi.out_type elements
    const float *scale_a;     // M per matrix, sa_stride apart; null: ones
    const float *scale_b;     // N per matrix, sb_stride apart; null: ones
    int64_t sa_stride, sb_stride;
    int32_t M, N, K, batch;
    int64_t lda, ldb, ldc, sA, sB, sC;
    const int32_t *group_rows;  // grouped: the rows of each matrix, clamped to [0, M]; else null
    Epilogue epi;
    uint32_t *status;
};
cudaError_t launch_s8_simple(const S8Params &p, cudaStream_t stream);

}  // namespace tsm
