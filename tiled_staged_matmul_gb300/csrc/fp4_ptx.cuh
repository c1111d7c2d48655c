// fp4_ptx.cuh -- inline-PTX wrappers that only the 4-bit operators use.
#pragma once

#include "s8_ptx.cuh"

#include <cuda_fp16.h>

namespace tsm {
namespace ptx {

// The three below are for code that a whole warp runs in step, of which one lane
// (`on`) issues: their operands are then the warp's, in the registers that the
// tensor core's instructions take.  (From a branch of one lane each operand is
// moved there first: three copies and an MMA took 270 cycles to issue.)

// D[tmem] (+)= A[smem desc] x B[smem desc] of e2m1 codes, 64 k, each block of BLK
// scaled by its rows' scales in TMEM (16: e4m3, four a row; 32: e8m0, two a
// row); f32 accumulator.  With PAIR each CTA supplies half of A's rows with their
// scales and half of B's rows; the scales of all of B's rows lie in both.
template <bool PAIR, int BLK>
__device__ __forceinline__ void mma_fp4(bool on, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t a_scales,
                                        uint32_t b_scales, uint32_t accumulate)
{
#define TSM_MMA_FP4(GROUP, VEC)                                                                                            \
    asm volatile("{\n\t.reg .pred p, q;\n\t"                                                                               \
                 "setp.ne.b32 p, %4, 0;\n\t"                                                                               \
                 "setp.ne.b32 q, %7, 0;\n\t"                                                                               \
                 "@q tcgen05.mma.cta_group::" GROUP ".kind::mxf4nvf4.block_scale.scale_vec::" VEC " [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"( \
                     d_tmem),                                                                                              \
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(a_scales), "r"(b_scales), "r"(uint32_t(on))      \
                 : "memory")
    if constexpr (PAIR && BLK == 16)
        TSM_MMA_FP4("2", "4X");
    else if constexpr (PAIR)
        TSM_MMA_FP4("2", "2X");
    else if constexpr (BLK == 16)
        TSM_MMA_FP4("1", "4X");
    else
        TSM_MMA_FP4("1", "2X");
#undef TSM_MMA_FP4
}

// A scale tile (32 rows of 16 bytes of shared memory) to four columns of TMEM,
// the same in each of the four lane quarters.  With PAIR in both CTAs, each from
// its own shared memory.  Ordered before this thread's later MMAs.
template <bool PAIR>
__device__ __forceinline__ void tmem_cp_scales(bool on, uint32_t taddr, uint64_t desc)
{
#define TSM_CP(GROUP)                                                                                                      \
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"                                                        \
                 "@q tcgen05.cp.cta_group::" GROUP ".32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr), "l"(desc), "r"(uint32_t(on)) \
                 : "memory")
    if constexpr (PAIR)
        TSM_CP("2");
    else
        TSM_CP("1");
#undef TSM_CP
}

// As mma_commit.
template <bool PAIR>
__device__ __forceinline__ void mma_commit_if(bool on, uint32_t bar, uint16_t cta_mask = 1)
{
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
            "h"(cta_mask), "r"(uint32_t(on))
            : "memory");
    else
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
                     "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
                     "r"(uint32_t(on))
                     : "memory");
}

// Warp-wide: lane l reads 16 consecutive 32-bit columns of TMEM lane
// (taddr.lane + l).
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t *r)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

// N consecutive columns (8, or a multiple of 16) of the lane, complete on return.
// (Naming the registers after the wait keeps their uses behind it.)
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[N])
{
    static_assert(N == 8 || N % 16 == 0, "columns");
    uint32_t r[N];
    if constexpr (N == 8) {
        tmem_ld_32x32b_x8(taddr, r);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 16)
            tmem_ld_32x32b_x16(taddr + uint32_t(i), r + i);
    }
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) {
        asm volatile("" : "+r"(r[i])::"memory");
        v[i] = __uint_as_float(r[i]);
    }
}

// The largest of |a|, |b| and |c|, NaN where one is.
__device__ __forceinline__ float max_abs3_nan(float a, float b, float c)
{
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// The nearest e4m3 number (ties to even, at most 448), and a code's value.
__device__ __forceinline__ uint32_t to_e4m3(float v)
{
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(0.f), "f"(v));
    return d;
}
__device__ __forceinline__ float from_e4m3(uint32_t code)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(code)));
    return __half2float(__ushort_as_half(uint16_t(h)));
}

// Eight values as e2m1 codes (to nearest, ties to even, at most 6), the first in
// the lowest four bits.
__device__ __forceinline__ uint32_t to_e2m1x8(const float *v)
{
    uint32_t d;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}

// Two values at a time (each as the scalar instructions round it):  x = m (x sx) + b.
__device__ __forceinline__ void mul_fma2(float &x, float &y, float sx, float sy, float m, float b)
{
    asm("{\n\t.reg .b64 v, s, mm, bb;\n\t"
        "mov.b64 v, {%0, %1};\n\tmov.b64 s, {%2, %3};\n\tmov.b64 mm, {%4, %4};\n\tmov.b64 bb, {%5, %5};\n\t"
        "mul.rn.f32x2 v, v, s;\n\t"
        "fma.rn.f32x2 v, v, mm, bb;\n\t"
        "mov.b64 {%0, %1}, v;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(sx), "f"(sy), "f"(m), "f"(b));
}
// x / (1 + 2^(-x log2 e)), to within a few units of f32 where 1 + ... is below 2^126,
// else 0.
__device__ __forceinline__ void silu2(float &x, float &y)
{
    asm("{\n\t.reg .b64 v, t, one;\n\t.reg .f32 a, b;\n\t"
        "mov.b64 v, {%0, %1};\n\tmov.b64 t, {%2, %2};\n\tmov.b64 one, {%3, %3};\n\t"
        "mul.rn.f32x2 t, v, t;\n\t"
        "mov.b64 {a, b}, t;\n\t"
        "ex2.approx.ftz.f32 a, a;\n\tex2.approx.ftz.f32 b, b;\n\t"
        "mov.b64 t, {a, b};\n\t"
        "add.rn.f32x2 t, t, one;\n\t"
        "mov.b64 {a, b}, t;\n\t"
        "rcp.approx.ftz.f32 a, a;\n\trcp.approx.ftz.f32 b, b;\n\t"
        "mov.b64 t, {a, b};\n\t"
        "mul.rn.f32x2 v, v, t;\n\t"
        "mov.b64 {%0, %1}, v;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(-1.4426950408889634f), "f"(1.f));
}

}  // namespace ptx
}  // namespace tsm
