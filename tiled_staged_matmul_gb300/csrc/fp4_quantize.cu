// fp4_quantize.cu -- rows to microscaled 4-bit floating point (e2m1).
//
// Blocks of 16, two levels of scales, for each row:
//   r = 2^e, the smallest (e >= -126) with max_k |x_k| <= 6 * 448 r   (zeros: r = 0)
//   s = max |x| of the block / (6 r), rounded to e4m3;  q_k = x_k / (s r), rounded to e2m1
// Blocks of 32, one level:
//   s = 2^e, e = max(floor(log2(max |x| of the block)) - 2, -127);  q_k = x_k / s, rounded to e2m1
// All roundings to nearest, ties to even; q saturates at 6.
//
// r is a power of two, so x / r is exact and a code is the exact quotient
// rounded once.  The quotient by s is formed in f32 as a correctly rounded
// division (a product with the reciprocal and one correction by the exact
// remainder): f32 rounding never moves a quotient of a 24-bit by a 4-bit number
// onto a middle between two codes that it was not on, since a quotient off a
// middle t is off by at least |t| 2^-24 times the ratio of their mantissas, more
// than half a step of f32 there.  The same holds for max / 6 and e4m3.
//
// Bound by memory: one read of a row, its 16-element units (one block of 16, half
// of one of 32) staying in registers between the maximum and the rounding.  What
// is read and written over the time, of the copy rate of 6.8 TB/s: 8191 x 8192 bf16
// blocks of 16 28.8 us, 0.88 (instructions come next: the corrected division),
// blocks of 32 25.1 us, 1.0; f32 45.1 us, 1.0; 8191 x 2048 bf16 9.1 us, 0.70.
#include "fp4_internal.h"
#include "fp4_ptx.cuh"
#include "launch.cuh"
#include "piece.cuh"

namespace tsm {

namespace {

constexpr int kUnit = 16;    // elements a thread takes at a time
constexpr int kUnitsKept = 2;  // units of a thread that stay in registers

// A unit as it lies in memory; what lies past the row's end as zeros.
template <int ET, bool WIDE>
struct Unit16 {
    using P = Piece<ET, WIDE ? 16 : (ET == kOutF32 ? 4 : 2)>;
    static constexpr int PIECES = kUnit / P::V;
    // (Narrow pieces are held widened.)
    typename Piece<ET, 16>::Raw raw[WIDE ? PIECES : 1];
    float val[WIDE ? 1 : kUnit];

    __device__ __forceinline__ void load(const char *x, int32_t unit, int32_t K)
    {
        using E = Piece<ET, ET == kOutF32 ? 4 : 2>;
        const int32_t k0 = unit * kUnit;
        if constexpr (WIDE) {
            if (k0 + kUnit <= K) {
#pragma unroll
                for (int i = 0; i < PIECES; ++i)
                    raw[i] = P::get(x, unit * PIECES + i);
                return;
            }
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    raw[i].w[w] = 0u;
            if (k0 >= K)
                return;
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    constexpr int PER = 4 / E::EB;  // elements a word
                    const int32_t k = k0 + (i * 4 + w) * PER;
                    uint32_t v = k < K ? E::get(x, k).w[0] : 0u;
                    if (PER == 2 && k + 1 < K)
                        v |= E::get(x, k + 1).w[0] << 16;
                    raw[i].w[w] = v;
                }
        } else {
#pragma unroll
            for (int j = 0; j < kUnit; ++j) {
                float v[1] = {0.f};
                if (k0 + j < K)
                    E::widen(E::get(x, k0 + j), v);
                val[j] = v[0];
            }
        }
    }
    __device__ __forceinline__ void widen(float (&v)[kUnit]) const
    {
        if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                float f[P::V];
                P::widen(raw[i], f);
#pragma unroll
                for (int j = 0; j < P::V; ++j)
                    v[P::V * i + j] = f[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < kUnit; ++j)
                v[j] = val[j];
        }
    }
    // The largest magnitude; NaN where there is one.
    __device__ __forceinline__ float top() const
    {
        if constexpr (WIDE && ET != kOutF32) {
            // (Magnitudes in order are their bits in order, NaNs last.  With maxima of
            // widened values 8191 x 8192 took 33.0 us.)
            static_assert(PIECES == 2, "two pieces");
            uint32_t m = 0u;
#pragma unroll
            for (int w = 0; w < 4; ++w)
                m = __vimax3_u16x2(m, raw[0].w[w] & 0x7fff7fffu, raw[1].w[w] & 0x7fff7fffu);
            const uint32_t most = max(m & 0xffffu, m >> 16);
            return ET == kOutBF16 ? __uint_as_float(most << 16) : __half2float(__ushort_as_half(uint16_t(most)));
        }
        float v[kUnit];
        widen(v);
        float m = 0.f;
#pragma unroll
        for (int j = 0; j < kUnit; j += 2)
            m = ptx::max_abs3_nan(m, v[j], v[j + 1]);
        return m;
    }
};

// x / d as f32 rounds it: c is 1 / d rounded, and one correction by the exact
// remainder makes up for what x c is off (P. Markstein, IA-64 and Elementary
// Functions, 2000).
__device__ __forceinline__ float divide(float x, float d, float c)
{
    const float q = x * c;
    return fmaf(fmaf(-q, d, x), c, q);
}
// Two at a time.
__device__ __forceinline__ void divide2(float &x, float &y, float d, float c)
{
    asm("{\n\t.reg .b64 v, q, r, dd, cc;\n\t"
        "mov.b64 v, {%0, %1};\n\tmov.b64 dd, {%2, %2};\n\tmov.b64 cc, {%3, %3};\n\t"
        "mul.rn.f32x2 q, v, cc;\n\t"
        "fma.rn.f32x2 r, q, dd, v;\n\t"
        "fma.rn.f32x2 q, r, cc, q;\n\t"
        "mov.b64 {%0, %1}, q;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(-d), "f"(c));
}

// ALIGNED: rows of X are 16-byte and rows of q 8-byte aligned.
template <int ET, int BLOCK, bool ALIGNED, int TPR>
__global__ void __launch_bounds__(TPR < 256 && TPR > 32 ? TPR : 256) tsm_quantize_fp4_kernel(Fp4QuantParams p)
{
    constexpr int ROWS = TPR == 32 ? 8 : 1;  // per CTA
    __shared__ uint32_t part[TPR / 32];
    chain_next();
    chain_wait();
    const int64_t at = int64_t(blockIdx.x) * ROWS + (ROWS > 1 ? threadIdx.x >> 5 : 0);
    if (at >= p.M * p.batch)
        return;
    const int tid = int(threadIdx.x) % TPR;
    // (Fewer than 2^31 rows.)
    const int64_t g = p.batch == 1 ? 0 : uint32_t(at) / uint32_t(p.M), r = at - g * p.M;
    if (p.group_rows && r >= int64_t(p.group_rows[g]))
        return;
    const char *x = static_cast<const char *>(p.X) + (g * p.sX + r * p.ldx) * (ET == kOutF32 ? 4 : 2);
    uint8_t *q = p.q + g * p.sQ + r * p.ldq;
    uint8_t *s = p.block_scales + (g * p.tile_rows + r / 128) * p.tile_cols * kScaleTile + (r % 32) * 16 + (r % 128) / 32 * 4;
    const int32_t K = int32_t(p.K);  // (below 2^31 - 2^16: the last units' ends are counted, too)
    const int32_t units = (K + kUnit - 1) / kUnit;
    const int32_t all = int32_t(p.tile_cols) * 4 * (BLOCK / kUnit);  // and those of zeros that fill the last scale tile
    constexpr int KEEP = kUnitsKept;
    Unit16<ET, ALIGNED> keep[KEEP];
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
        keep[i].load(x, tid + i * TPR, K);

    float inverse = 1.f;  // 1 / r
    float r_ = 1.f;       // r
    bool none = false;    // the row's codes are zeros
    bool tiny = false;    // the row's values are worked on 2^60 times as large (r and 1 / r say so)
    float tops[KEEP];
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
        tops[i] = keep[i].top();
    if constexpr (BLOCK == 16) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            top = ptx::max_abs3_nan(top, tops[i], 0.f);
        for (int32_t u = tid + KEEP * TPR; u < units; u += TPR) {
            Unit16<ET, ALIGNED> one;
            one.load(x, u, K);
            top = ptx::max_abs3_nan(top, one.top(), 0.f);
        }
        // As bits of non-negative floats the maximum orders infinities and NaNs last.
        uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
        if constexpr (TPR > 32) {
            if ((tid & 31) == 0)
                part[tid >> 5] = bits;
            __syncthreads();
#pragma unroll
            for (int k = 0; k < TPR / 32; ++k)
                bits = max(bits, part[k]);
        }
        const bool finite = bits < 0x7f800000u;
        // 2688 = 1.3125 x 2^11: with max = m 2^n, 1 <= m < 2, r is 2^(n-11), or twice
        // that where m is larger than 1.3125 (0x280000 of 2^23).
        int e = int(bits >> 23) - 127 - 11 + ((bits & 0x7fffffu) > 0x280000u);
        e = max(e, -126);
        none = !finite || bits == 0;
        if (tid == 0)
            p.scales[g * p.sS + r] = !finite ? __uint_as_float(0x7fffffffu) : bits == 0 ? 0.f : __uint_as_float(uint32_t(127 + e) << 23);
        // (1 / (s r) and the remainders below would leave f32's range.)
        tiny = e < -60;
        if (tiny)
            e += 60;
        inverse = __uint_as_float(uint32_t(127 - e) << 23);
        r_ = __uint_as_float(uint32_t(127 + e) << 23);
    }

    auto put = [&](int32_t u, const Unit16<ET, ALIGNED> &unit, float top) {
        float v[kUnit];
        uint32_t scale;  // as stored
        unit.widen(v);
        if constexpr (BLOCK == 16) {
            if (tiny) {
                top *= 0x1p60f;
#pragma unroll
                for (int j = 0; j < kUnit; ++j)
                    v[j] *= 0x1p60f;
            }
            scale = none ? 0u : ptx::to_e4m3(divide(top * inverse, 6.f, 1.f / 6.f));
            const float sf = ptx::from_e4m3(scale);
            const float d = sf * r_, c = __frcp_rn(sf) * inverse;  // (powers of two: both exact)
#pragma unroll
            for (int j = 0; j < kUnit; j += 2)
                divide2(v[j], v[j + 1], d, c);
        } else {
            // The neighbour lane holds the block's other half.
            const float other = __shfl_xor_sync(0xffffffffu, top, 1);
            const uint32_t bits = max(__float_as_uint(top), __float_as_uint(other));
            scale = bits >= 0x7f800000u ? 255u : uint32_t(max(int(bits >> 23) - 2, 0));
            const float m = __uint_as_float((254u - min(scale, 254u)) << 23);
#pragma unroll
            for (int j = 0; j < kUnit; ++j)
                v[j] *= m;
        }
        // (What a scale of 0 or NaN makes of the values is not kept.)
        const uint32_t kept = (BLOCK == 16 ? scale == 0 : scale == 255u) ? 0u : 0xffffffffu;
        const uint32_t lo = ptx::to_e2m1x8(v) & kept, hi = ptx::to_e2m1x8(v + 8) & kept;
        if (u < units) {
            const int32_t bytes = (K + 1) / 2 - u * 8;  // left in the row
            uint8_t *const to = q + u * 8;
            if (ALIGNED && bytes >= 8) {
                *reinterpret_cast<uint2 *>(to) = make_uint2(lo, hi);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (j < bytes)
                        to[j] = uint8_t((j < 4 ? lo : hi) >> (8 * (j & 3)));
            }
        }
        if (u < all && (BLOCK == 16 || (u & 1) == 0)) {
            const uint32_t b = uint32_t(BLOCK == 16 ? u : u >> 1);
            s[int64_t(b / 4) * kScaleTile + b % 4] = uint8_t(scale);
        }
    };
    // (Whole warps go round: a block of 32 is two lanes'.)
#pragma unroll
    for (int i = 0; i < KEEP; ++i)
        if (i * TPR < all)
            put(tid + i * TPR, keep[i], tops[i]);
    for (int32_t u = tid + KEEP * TPR; u - tid < all; u += TPR) {
        Unit16<ET, ALIGNED> one;
        one.load(x, u, K);
        put(u, one, one.top());
    }
}

template <int ET, int BLOCK, bool ALIGNED>
cudaError_t quantize_as(const Fp4QuantParams &p, cudaStream_t stream)
{
    const int64_t rows = p.M * p.batch, units = (p.K + kUnit - 1) / kUnit;
    // As few threads to a row as keep it (a warp: eight rows a CTA, nothing to wait
    // for), 256 where none do.  So and with 256 throughout, blocks of 16, bf16, us (both
    // while maxima were taken of widened values: now 9.1 and 14.9 of 2048 and 4096): 8191
    // rows of 512 3.8 and 22.0, of 2048 10.1 and 23.6, of 4096 16.3 and 25.5; 512 of
    // 1024 2.0 and 2.5; 16 of 4096 1.7 and 1.6.
    if (units <= 32 * kUnitsKept)
        return launch_chained(tsm_quantize_fp4_kernel<ET, BLOCK, ALIGNED, 32>, dim3(unsigned((rows + 7) / 8)), 256, 0, 0, stream, p);
    if (units <= 64 * kUnitsKept)
        return launch_chained(tsm_quantize_fp4_kernel<ET, BLOCK, ALIGNED, 64>, dim3(unsigned(rows)), 64, 0, 0, stream, p);
    if (units <= 128 * kUnitsKept)
        return launch_chained(tsm_quantize_fp4_kernel<ET, BLOCK, ALIGNED, 128>, dim3(unsigned(rows)), 128, 0, 0, stream, p);
    return launch_chained(tsm_quantize_fp4_kernel<ET, BLOCK, ALIGNED, 256>, dim3(unsigned(rows)), 256, 0, 0, stream, p);
}

template <int ET>
cudaError_t quantize_type(const Fp4QuantParams &p, bool aligned, int block, cudaStream_t stream)
{
    if (block == 16)
        return aligned ? quantize_as<ET, 16, true>(p, stream) : quantize_as<ET, 16, false>(p, stream);
    return aligned ? quantize_as<ET, 32, true>(p, stream) : quantize_as<ET, 32, false>(p, stream);
}

}  // namespace

cudaError_t launch_quantize_fp4(const Fp4QuantParams &p, int elem, bool aligned, int block, cudaStream_t stream)
{
    switch (elem) {
    case kOutF32: return quantize_type<kOutF32>(p, aligned, block, stream);
    case kOutF16: return quantize_type<kOutF16>(p, aligned, block, stream);
    default: return quantize_type<kOutBF16>(p, aligned, block, stream);
    }
}

}  // namespace tsm
