// moe_kernels.cu -- moving token rows to their experts and back.
//
//   route         slots[t][j] = e * capacity + rank, e = ids[t][j], rank = the
//                 number of earlier (t', j') < (t, j) with the same expert; -1
//                 when rank >= capacity or e is no expert.
//                 counts[e] = min(capacity, choices of e).
//   dispatch      rows[slots[t][j]] = x[t]
//   dispatch_grad dx[t] = sum_j drows[slots[t][j]]           (combine without weights)
//   combine       out[t] = sum_j w[t][j] rows[slots[t][j]]
//   combine_grad  drows[slots[t][j]] = w[t][j] dout[t],  dw[t][j] = <dout[t], rows[slots[t][j]]>
//
// All of it is bound by memory (one multiply-add for two to four bytes), or,
// for a decode step's few tokens, by launch and load latency.  Every kernel
// is built around the token: its row is read once for all its choices
// (dispatch, combine_grad) or written once (combine), so each byte crosses
// HBM once and no inverse map of the slots is needed.  Sums run in f32 over j
// in ascending order, rounded once to the rows' type; there are no atomics on
// floating-point data, so a call is bitwise reproducible.
#include "launch.cuh"
#include "ops_internal.h"
#include "piece.cuh"
#include "s8_ptx.cuh"

#include <type_traits>

namespace tsm {

namespace {

// ------------------------------------------------------------- route

// The expert of assignment i, or -1.
template <bool WIDE>
__device__ __forceinline__ int32_t expert_of(const RouteParams &p, int64_t i)
{
    if (i >= p.n)
        return -1;
    const int64_t e = WIDE ? static_cast<const long long *>(p.ids)[i]
                           : int64_t(static_cast<const int32_t *>(p.ids)[i]);
    return e >= 0 && e < p.groups ? int32_t(e) : -1;
}

// Counts per expert of one chunk (several chunks only).
template <bool WIDE, int ROUNDS>
__global__ void __launch_bounds__(32 * kRouteWarps) tsm_moe_count_kernel(RouteParams p)
{
    extern __shared__ uint32_t count[];
    chain_next();
    chain_wait();
    for (int e = int(threadIdx.x); e < p.groups; e += int(blockDim.x))
        count[e] = 0;
    __syncthreads();
    const int64_t first = int64_t(blockIdx.x) * route_chunk(ROUNDS);
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int32_t e = expert_of<WIDE>(p, first + int64_t(r) * blockDim.x + threadIdx.x);
        if (e >= 0)
            atomicAdd(count + e, 1u);
    }
    __syncthreads();
    for (int e = int(threadIdx.x); e < p.groups; e += int(blockDim.x))
        p.hist[int64_t(blockIdx.x) * p.groups + e] = int32_t(count[e]);
}

// Ranks of one chunk.  Warp w holds ROUNDS x 32 consecutive assignments; a
// lane's rank is what the warp counted in earlier rounds, plus the lower lanes
// of the same expert (a warp match), plus the earlier warps' counts, plus the
// earlier chunks'.  Those come from the count kernel's table or, where one
// cluster holds all chunks (CLUSTER), from the other CTAs' shared memory, with
// one launch and no table: 16384 choices of 8 experts 4.3 us, not 6.0; 32768 of
// 64 7.9 and 8.0; a decode step's 32, one chunk, 2.3.
template <bool WIDE, int ROUNDS, bool CLUSTER>
__global__ void __launch_bounds__(32 * kRouteWarps) tsm_moe_rank_kernel(RouteParams p)
{
    extern __shared__ uint32_t smem[];
    uint32_t *const base = smem;                                        // [groups]
    uint32_t *const total = smem + p.groups;                            // [groups], of this chunk (CLUSTER)
    uint16_t *const seen = reinterpret_cast<uint16_t *>(smem + (CLUSTER ? 2 : 1) * p.groups);  // [warps][groups]
    const int warp = int(threadIdx.x >> 5), lane = int(threadIdx.x & 31);
    const int G = p.groups;
    chain_next();
    chain_wait();
    const int64_t first = int64_t(blockIdx.x) * route_chunk(ROUNDS) + int64_t(warp) * 32 * ROUNDS;
    int32_t id[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r)
        id[r] = expert_of<WIDE>(p, first + 32 * r + lane);
    for (int i = lane; i < G; i += 32)
        seen[warp * G + i] = 0;
    // The earlier chunks' counts, while the ids are on their way.
    for (int e = int(threadIdx.x); !CLUSTER && e < G; e += int(blockDim.x)) {
        uint32_t before = 0;
        for (int64_t c = 0; c < int64_t(blockIdx.x); ++c)
            before += uint32_t(p.hist[c * G + e]);
        base[e] = before;
    }
    __syncwarp();
    uint32_t at[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const uint32_t same = __match_any_sync(0xffffffffu, id[r]);
        const uint32_t lower = __popc(same & ((1u << lane) - 1u));
        uint32_t earlier = 0;
        if (id[r] >= 0)
            earlier = seen[warp * G + id[r]];
        __syncwarp();
        if (id[r] >= 0 && lower == 0)
            seen[warp * G + id[r]] = uint16_t(earlier + __popc(same));
        __syncwarp();
        at[r] = earlier + lower;
    }
    __syncthreads();
    // Exclusive sums over the warps, in place; the chunk's total.
    const bool last = blockIdx.x == gridDim.x - 1;
    for (int e = int(threadIdx.x); e < G; e += int(blockDim.x)) {
        uint32_t sum = 0;
        for (int w = 0; w < kRouteWarps; ++w) {
            const uint32_t c = seen[w * G + e];
            seen[w * G + e] = uint16_t(sum);
            sum += c;
        }
        if (CLUSTER)
            total[e] = sum;
        else if (last)
            p.counts[e] = int32_t(min(base[e] + sum, uint32_t(p.capacity)));
    }
    if (CLUSTER) {
        ptx::cluster_sync();
        for (int e = int(threadIdx.x); e < G; e += int(blockDim.x)) {
            uint32_t x[kRouteCluster - 1], before = 0;
#pragma unroll
            for (uint32_t c = 0; c < kRouteCluster - 1; ++c)
                x[c] = c < blockIdx.x ? ptx::ld_cluster_u32(ptx::mapa_shared(ptx::smem_addr(total + e), c)) : 0u;
#pragma unroll
            for (uint32_t c = 0; c < kRouteCluster - 1; ++c)
                before += x[c];
            base[e] = before;
            if (last)
                p.counts[e] = int32_t(min(before + total[e], uint32_t(p.capacity)));
        }
        ptx::cluster_arrive_relaxed();
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int64_t i = first + 32 * r + lane;
        if (i < p.n) {
            int32_t slot = -1;
            if (id[r] >= 0) {
                const uint32_t rank = base[id[r]] + seen[warp * G + id[r]] + at[r];
                if (rank < uint32_t(p.capacity))
                    slot = id[r] * p.capacity + int32_t(rank);
            }
            p.slots[i] = slot;
        }
    }
    if (CLUSTER)
        ptx::cluster_wait();  // no CTA leaves while another may still read its totals
}

// ------------------------------------------------------------- row types

// Row `slot` of the experts' side exists.
__device__ __forceinline__ bool has_row(const MoveParams &p, int32_t slot)
{
    return slot >= 0 && int64_t(slot) < p.rows;
}

// ------------------------------------------------------------- dispatch

// A warp copies kCopyUnroll x 32 units of one token's row to all its slots.
// 8192 tokens to 2 of 8 experts, 4096 bf16: 31 us, 0.97 of the copy rate.
constexpr int kCopyUnroll = 4;

template <typename U>
__global__ void __launch_bounds__(256) tsm_moe_dispatch_kernel(MoveParams p)
{
    chain_next();
    chain_wait();
    const int lane = int(threadIdx.x & 31);
    const int64_t per = 32 * kCopyUnroll;
    const int64_t segs = (p.width + per - 1) / per;
    const int64_t warps = int64_t(gridDim.x) * (blockDim.x / 32);
    for (int64_t i = int64_t(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5); i < p.tokens * segs;
         i += warps) {
        const int64_t t = i / segs;
        const int64_t c0 = (i - t * segs) * per + lane;
        const U *src = static_cast<const U *>(p.src) + t * p.ld_src;
        U v[kCopyUnroll];
#pragma unroll
        for (int k = 0; k < kCopyUnroll; ++k)
            if (c0 + 32 * k < p.width)
                v[k] = src[c0 + 32 * k];
        // The slots a warp's load at a time, ahead of the stores.
        for (int64_t j0 = 0; j0 < p.topk; j0 += 32) {
            const int32_t mine = j0 + lane < p.topk ? p.slots[t * p.topk + j0 + lane] : -1;
            const int n = int(p.topk - j0 < 32 ? p.topk - j0 : 32);
            for (int j = 0; j < n; ++j) {
                const int32_t slot = __shfl_sync(0xffffffffu, mine, j);
                if (!has_row(p, slot))
                    continue;
                U *dst = static_cast<U *>(p.dst) + int64_t(slot) * p.ld_dst;
#pragma unroll
                for (int k = 0; k < kCopyUnroll; ++k)
                    if (c0 + 32 * k < p.width)
                        dst[c0 + 32 * k] = v[k];
            }
        }
    }
}

// ------------------------------------------------------------- combine

// A warp sums U x 32 pieces of a token's row over its choices, K rows at a
// time: U x K loads of a lane in flight.  Many tokens: U = 2, K = 2 (8192
// tokens, 2 choices, 4096 bf16: 33 us, 0.92 of the copy rate; U = 3 39 us, with
// fewer warps on an SM; K = 4 47 us, half its loads without a row.  4096 tokens, 6
// choices, 2048 bf16: 21, 22 and 25); few tokens (a decode step): U = 1, K = 8,
// every warp there is at work and a token's rows loaded in one go.
template <int ET, int BYTES, int U, int K>
__global__ void __launch_bounds__(256) tsm_moe_combine_kernel(MoveParams p)
{
    using P = Piece<ET, BYTES>;
    chain_next();
    chain_wait();
    const int lane = int(threadIdx.x & 31);
    const int64_t pieces = p.width / P::V;
    const int64_t segs = (pieces + 32 * U - 1) / (32 * U);
    const int64_t warps = int64_t(gridDim.x) * (blockDim.x / 32);
    for (int64_t i = int64_t(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5); i < p.tokens * segs; i += warps) {
        const int64_t t = i / segs;
        const int64_t c0 = (i - t * segs) * (32 * U) + lane;
        float acc[U][P::V];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < P::V; ++k)
                acc[u][k] = 0.f;
        for (int64_t j0 = 0; j0 < p.topk; j0 += K) {
            typename P::Raw raw[K][U];
            float w[K];
            // (A choice without a row: zeros, and a weight of zero whatever its own.)
#pragma unroll
            for (int j = 0; j < K; ++j) {
                const bool in = j0 + j < p.topk;
                const int32_t slot = in ? p.slots[t * p.topk + j0 + j] : -1;
                const bool on = has_row(p, slot);
                w[j] = !on ? 0.f : p.weights ? p.weights[t * p.topk + j0 + j] : 1.f;
                const char *row = static_cast<const char *>(p.src) + int64_t(slot) * p.ld_src * P::EB;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    raw[j][u] = {};
                    if (on && c0 + 32 * u < pieces)
                        raw[j][u] = P::get(row, c0 + 32 * u);
                }
            }
#pragma unroll
            for (int j = 0; j < K; ++j)
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float v[P::V];
                    P::widen(raw[j][u], v);
#pragma unroll
                    for (int k = 0; k < P::V; ++k)
                        acc[u][k] = fmaf(w[j], v[k], acc[u][k]);
                }
        }
        char *out = static_cast<char *>(p.dst) + t * p.ld_dst * P::EB;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + 32 * u < pieces)
                P::store(out, c0 + 32 * u, acc[u]);
    }
}

// ------------------------------------------------------------- combine's gradient

// A warp per choice: it walks the token's dout and the choice's row together,
// kGradUnroll pieces of each in flight per lane, writes w dout and keeps the
// dot product, which a butterfly adds up in a fixed order.  The warps of a
// token's choices are neighbours, so dout comes from HBM once and from the L1
// or L2 for the others; nothing waits for another warp.  4095 tokens, 6
// choices, 2048 f16: 35 us, 0.91 of the copy rate (a warp per token, its choices
// one after the other: 51).
constexpr int kGradUnroll = 4;

template <int ET, int BYTES>
__global__ void __launch_bounds__(256) tsm_moe_combine_grad_kernel(MoveParams p)
{
    using P = Piece<ET, BYTES>;
    chain_next();
    chain_wait();
    const int lane = int(threadIdx.x & 31);
    const int64_t pieces = p.width / P::V;
    const int64_t warps = int64_t(gridDim.x) * (blockDim.x / 32);
    for (int64_t i = int64_t(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5); i < p.tokens * p.topk; i += warps) {
        const int32_t slot = p.slots[i];
        float dot = 0.f;
        if (has_row(p, slot)) {
            const float w = p.weights ? p.weights[i] : 1.f;
            const char *dout = static_cast<const char *>(p.dout) + i / p.topk * p.ld_dout * P::EB;
            const char *row = static_cast<const char *>(p.src) + int64_t(slot) * p.ld_src * P::EB;
            char *drow = static_cast<char *>(p.dst) + int64_t(slot) * p.ld_dst * P::EB;
            for (int64_t c0 = lane; c0 < pieces; c0 += 32 * kGradUnroll) {
                typename P::Raw d[kGradUnroll], y[kGradUnroll];
#pragma unroll
                for (int u = 0; u < kGradUnroll; ++u)
                    if (c0 + 32 * u < pieces) {
                        d[u] = P::get(dout, c0 + 32 * u);
                        y[u] = P::get(row, c0 + 32 * u);
                    }
#pragma unroll
                for (int u = 0; u < kGradUnroll; ++u)
                    if (c0 + 32 * u < pieces) {
                        float dv[P::V], yv[P::V], s = 0.f;
                        P::widen(d[u], dv);
                        P::widen(y[u], yv);
#pragma unroll
                        for (int k = 0; k < P::V; ++k) {
                            s = fmaf(dv[k], yv[k], s);
                            dv[k] *= w;
                        }
                        dot += s;
                        P::store(drow, c0 + 32 * u, dv);
                    }
            }
#pragma unroll
            for (int m = 16; m; m >>= 1)
                dot += __shfl_xor_sync(0xffffffffu, dot, m);
        }
        if (lane == 0 && p.dweights)
            p.dweights[i] = dot;
    }
}

// ------------------------------------------------------------- row quantisation

//   scale = max_k |x_k| / 127,  q_k = rint(x_k / scale)   (a row of zeros: scale 0, q 0;
//   a row with an infinity or a NaN: scale NaN, q 0, so that its products are NaN)
//
// One CTA per row; a row of up to kQuantKeep pieces per thread stays in
// registers between the maximum and the rounding, so it is read once.
//
// The codes are those of the IEEE quotient in f32, but few divisions are made:
// x times the rounded reciprocal of the scale is within 127 x 2^-22 of it, and
// where that is further than 1e-4 from the middle between two integers both
// round alike; only the others (one in 5000) are divided.  Adding 1.5 x 2^23
// rounds to the nearest integer, ties to even, and leaves it in the low bits:
// no conversion either.  (8191 x 8192 bf16: 66 us with a division and a
// conversion for each code, 40 us so; at the copy rate it would be 30.)
//
// TPR threads take a row: a warp (eight rows a block, nothing to wait for)
// where that gives a lane no more than kQuantKeep pieces, else 128; 256 where
// there are too few rows to fill the GPU.
constexpr int kQuantKeep = 8;

template <int ET, int BYTES, int TPR>
__global__ void __launch_bounds__(TPR < 256 && TPR > 32 ? TPR : 256) tsm_quantize_rows_kernel(QuantParams p)
{
    using P = Piece<ET, BYTES>;
    constexpr int ROWS = TPR == 32 ? 8 : 1;  // per block
    __shared__ uint32_t part[TPR / 32];
    chain_next();
    chain_wait();
    const int64_t at = int64_t(blockIdx.x) * ROWS + (ROWS > 1 ? threadIdx.x >> 5 : 0);
    if (at >= p.M * p.batch)
        return;
    const int tid = int(threadIdx.x) % TPR;
    const int64_t g = at / p.M;
    const int64_t r = at - g * p.M;
    if (p.group_rows && r >= int64_t(p.group_rows[g]))
        return;
    const char *x = static_cast<const char *>(p.X) + (g * p.sX + r * p.ldx) * P::EB;
    int8_t *q = p.q + g * p.sQ + r * p.ldq;
    const int64_t pieces = p.K / P::V;
    typename P::Raw keep[kQuantKeep];
    uint32_t top = 0;
    auto see = [&](const typename P::Raw &raw) {
        float v[P::V];
        P::widen(raw, v);
#pragma unroll
        for (int k = 0; k < P::V; ++k)
            top = max(top, __float_as_uint(v[k]) & 0x7fffffffu);
    };
#pragma unroll
    for (int i = 0; i < kQuantKeep; ++i) {
        const int64_t c = tid + int64_t(i) * TPR;
        if (c < pieces)
            keep[i] = P::get(x, c);
    }
#pragma unroll
    for (int i = 0; i < kQuantKeep; ++i)
        if (tid + int64_t(i) * TPR < pieces)
            see(keep[i]);
    for (int64_t c = tid + int64_t(kQuantKeep) * TPR; c < pieces; c += TPR)
        see(P::get(x, c));
    top = __reduce_max_sync(0xffffffffu, top);
    if constexpr (TPR > 32) {
        if ((tid & 31) == 0)
            part[tid >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < TPR / 32; ++k)
            top = max(top, part[k]);
    }
    // As bits of non-negative floats the maximum orders infinities and NaNs last.
    const bool finite = top < 0x7f800000u;
    const float scale = finite ? __fdiv_rn(__uint_as_float(top), 127.f) : __uint_as_float(0x7fffffffu);
    const bool zero = !finite || scale == 0.f;
    if (tid == 0)
        p.scales[g * p.sS + r] = scale;
    const float inverse = __frcp_rn(scale);
    const bool divide = !(inverse < __uint_as_float(0x7f800000u));  // (a subnormal scale)
    auto exactly = [&](float v) {
        // |v / scale| can pass 127 by more than a rounding where the scale is subnormal.
        return fminf(fmaxf(rintf(__fdiv_rn(v, scale)), -127.f), 127.f);
    };
    constexpr float kMagic = 12582912.f;  // 1.5 x 2^23
    // Codes of a piece's values, in the low bytes of the results.
    auto codes = [&](const float (&v)[P::V], uint32_t (&out)[P::V]) {
        float near = 0.f;
#pragma unroll
        for (int k = 0; k < P::V; ++k) {
            const float y = v[k] * inverse;
            const float t = y + kMagic;
            near = fmaxf(near, fabsf(y - (t - kMagic)));
            out[k] = __float_as_uint(t);
        }
        if (near > 0.4999f || divide) {
#pragma unroll
            for (int k = 0; k < P::V; ++k)
                out[k] = __float_as_uint(exactly(v[k]) + kMagic);
        }
        if (zero) {
#pragma unroll
            for (int k = 0; k < P::V; ++k)
                out[k] = 0u;
        }
    };
    auto put = [&](int64_t c, const typename P::Raw &raw) {
        float v[P::V];
        uint32_t o[P::V];
        P::widen(raw, v);
        codes(v, o);
        if constexpr (P::V == 1) {
            q[c] = int8_t(o[0]);
        } else if constexpr (P::V == 2) {
            reinterpret_cast<unsigned short *>(q)[c] = uint16_t(__byte_perm(o[0], o[1], 0x0040));
        } else {
            uint32_t w[P::V / 4];
#pragma unroll
            for (int k = 0; k < P::V / 4; ++k)
                w[k] = __byte_perm(__byte_perm(o[4 * k], o[4 * k + 1], 0x0040),
                                   __byte_perm(o[4 * k + 2], o[4 * k + 3], 0x0040), 0x5410);
            if constexpr (P::V == 8)
                reinterpret_cast<uint2 *>(q)[c] = make_uint2(w[0], w[1]);
            else
                reinterpret_cast<uint32_t *>(q)[c] = w[0];
        }
    };
#pragma unroll
    for (int i = 0; i < kQuantKeep; ++i) {
        const int64_t c = tid + int64_t(i) * TPR;
        if (c < pieces)
            put(c, keep[i]);
    }
    for (int64_t c = tid + int64_t(kQuantKeep) * TPR; c < pieces; c += TPR)
        put(c, P::get(x, c));
}

template <bool WIDE, int ROUNDS>
cudaError_t route_in_cluster(const RouteParams &p, int64_t chunks, cudaStream_t stream)
{
    return launch_chained(tsm_moe_rank_kernel<WIDE, ROUNDS, true>, dim3(unsigned(chunks)), 32 * kRouteWarps,
                          size_t(p.groups) * (8 + 2 * kRouteWarps), unsigned(chunks), stream, p);
}

template <bool WIDE, int ROUNDS>
cudaError_t route_as(const RouteParams &p, int64_t chunks, cudaStream_t stream)
{
    constexpr int threads = 32 * kRouteWarps;
    cudaError_t e = cudaSuccess;
    if (chunks > 1)
        e = launch_chained(tsm_moe_count_kernel<WIDE, ROUNDS>, dim3(unsigned(chunks)), threads, size_t(p.groups) * 4, 0,
                           stream, p);
    if (e == cudaSuccess)
        e = launch_chained(tsm_moe_rank_kernel<WIDE, ROUNDS, false>, dim3(unsigned(chunks)), threads,
                           size_t(p.groups) * (4 + 2 * kRouteWarps), 0, stream, p);
    return e;
}

template <typename U>
cudaError_t dispatch_as(const MoveParams &p, int sms, cudaStream_t stream)
{
    const int64_t segs = (p.width + 32 * kCopyUnroll - 1) / (32 * kCopyUnroll);
    const int64_t blocks = (p.tokens * segs + 7) / 8;
    return launch_chained(tsm_moe_dispatch_kernel<U>, dim3(unsigned(min(blocks, int64_t(sms) * 64))), 256, 0, 0, stream, p);
}

}  // namespace

cudaError_t launch_route(const RouteParams &p, bool wide_ids, int rounds, int64_t chunks, cudaStream_t stream)
{
    const auto run = [&](auto wide) {
        constexpr bool W = decltype(wide)::value;
        if (chunks > 1 && !p.hist)
            switch (rounds) {
            case kRouteRoundsSmall: return route_in_cluster<W, kRouteRoundsSmall>(p, chunks, stream);
            case 2 * kRouteRoundsSmall: return route_in_cluster<W, 2 * kRouteRoundsSmall>(p, chunks, stream);
            default: return route_in_cluster<W, kRouteRoundsCluster>(p, chunks, stream);
            }
        return rounds == kRouteRoundsSmall ? route_as<W, kRouteRoundsSmall>(p, chunks, stream)
                                           : route_as<W, kRouteRoundsLarge>(p, chunks, stream);
    };
    return wide_ids ? run(std::true_type{}) : run(std::false_type{});
}

cudaError_t launch_dispatch(const MoveParams &p, int vec, int sms, cudaStream_t stream)
{
    switch (vec) {
    case 16: return dispatch_as<uint4>(p, sms, stream);
    case 8: return dispatch_as<uint2>(p, sms, stream);
    case 4: return dispatch_as<uint32_t>(p, sms, stream);
    case 2: return dispatch_as<unsigned short>(p, sms, stream);
    default: return dispatch_as<unsigned char>(p, sms, stream);
    }
}

namespace {

template <int ET, int BYTES>
cudaError_t combine_as(const MoveParams &p, int sms, cudaStream_t stream)
{
    const int64_t pieces = p.width / Piece<ET, BYTES>::V;
    const auto grid = [&](int u) {
        const int64_t blocks = (p.tokens * ((pieces + 32 * u - 1) / (32 * u)) + 7) / 8;
        return dim3(unsigned(min(blocks, int64_t(sms) * 64)));
    };
    if (p.tokens * pieces < int64_t(sms) * 1024)
        return launch_chained(tsm_moe_combine_kernel<ET, BYTES, 1, 8>, grid(1), 256, 0, 0, stream, p);
    return launch_chained(tsm_moe_combine_kernel<ET, BYTES, 2, 2>, grid(2), 256, 0, 0, stream, p);
}

template <int ET, int BYTES>
cudaError_t combine_grad_as(const MoveParams &p, int sms, cudaStream_t stream)
{
    const int64_t blocks = (p.tokens * p.topk + 7) / 8;
    return launch_chained(tsm_moe_combine_grad_kernel<ET, BYTES>, dim3(unsigned(min(blocks, int64_t(sms) * 64))), 256, 0,
                          0, stream, p);
}

}  // namespace

namespace {

// fn with a type and a piece size fixed at compile time.
template <typename F>
cudaError_t with_piece(int elem, int bytes, F &&fn)
{
    switch (elem) {
    case kOutF32: return bytes == 16 ? fn(Piece<kOutF32, 16>{}) : fn(Piece<kOutF32, 4>{});
    case kOutF16:
        return bytes == 16 ? fn(Piece<kOutF16, 16>{}) : bytes == 4 ? fn(Piece<kOutF16, 4>{}) : fn(Piece<kOutF16, 2>{});
    default:
        return bytes == 16 ? fn(Piece<kOutBF16, 16>{}) : bytes == 4 ? fn(Piece<kOutBF16, 4>{}) : fn(Piece<kOutBF16, 2>{});
    }
}

template <int ET, int BYTES>
cudaError_t quantize_as(const QuantParams &p, int sms, cudaStream_t stream)
{
    const int64_t rows = p.M * p.batch, pieces = p.K / Piece<ET, BYTES>::V;
    if (rows < int64_t(sms) * 4)
        return launch_chained(tsm_quantize_rows_kernel<ET, BYTES, 256>, dim3(unsigned(rows)), 256, 0, 0, stream, p);
    if (pieces <= 32 * kQuantKeep)
        return launch_chained(tsm_quantize_rows_kernel<ET, BYTES, 32>, dim3(unsigned((rows + 7) / 8)), 256, 0, 0, stream, p);
    return launch_chained(tsm_quantize_rows_kernel<ET, BYTES, 128>, dim3(unsigned(rows)), 128, 0, 0, stream, p);
}

// The type and piece size of a Piece as template arguments of fn.
template <int ET, int BYTES>
constexpr int type_of(Piece<ET, BYTES>) { return ET; }
template <int ET, int BYTES>
constexpr int bytes_of(Piece<ET, BYTES>) { return BYTES; }

}  // namespace

cudaError_t launch_combine(const MoveParams &p, int elem, int bytes, int sms, cudaStream_t stream)
{
    return with_piece(elem, bytes, [&](auto x) { return combine_as<type_of(decltype(x){}), bytes_of(decltype(x){})>(p, sms, stream); });
}

cudaError_t launch_combine_grad(const MoveParams &p, int elem, int bytes, int sms, cudaStream_t stream)
{
    return with_piece(elem, bytes, [&](auto x) { return combine_grad_as<type_of(decltype(x){}), bytes_of(decltype(x){})>(p, sms, stream); });
}

cudaError_t launch_quantize_rows(const QuantParams &p, int elem, int bytes, int sms, cudaStream_t stream)
{
    return with_piece(elem, bytes, [&](auto x) { return quantize_as<type_of(decltype(x){}), bytes_of(decltype(x){})>(p, sms, stream); });
}

}  // namespace tsm
