// piece.cuh -- rows of f32, f16 or bf16 read and written a piece at a time.
#pragma once

#include "gemm_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace tsm {

// One access of BYTES bytes (16, 4 or one element) of type ET.
template <int ET, int BYTES>
struct Piece {
    static constexpr int EB = ET == kOutF32 ? 4 : 2;
    static constexpr int V = BYTES / EB;
    static_assert(BYTES == 16 || BYTES == 4 || BYTES == EB, "piece");

    // A piece as it lies in memory (kept so while it waits: half the registers).
    struct Raw {
        uint32_t w[BYTES == 16 ? 4 : 1];
    };
    static __device__ __forceinline__ Raw get(const void *row, int64_t i)
    {
        Raw r;
        if constexpr (BYTES == 16) {
            const uint4 u = static_cast<const uint4 *>(row)[i];
            r.w[0] = u.x;
            r.w[1] = u.y;
            r.w[2] = u.z;
            r.w[3] = u.w;
        } else if constexpr (BYTES == 4) {
            r.w[0] = static_cast<const uint32_t *>(row)[i];
        } else {
            r.w[0] = static_cast<const unsigned short *>(row)[i];
        }
        return r;
    }
    static __device__ __forceinline__ void widen(const Raw &raw, float (&v)[V])
    {
        if constexpr (ET == kOutF32) {
#pragma unroll
            for (int k = 0; k < V; ++k)
                v[k] = __uint_as_float(raw.w[k]);
        } else if constexpr (V == 1) {
            v[0] = ET == kOutF16 ? __half2float(__ushort_as_half(uint16_t(raw.w[0]))) : __uint_as_float(raw.w[0] << 16);
        } else {
#pragma unroll
            for (int k = 0; k < V / 2; ++k) {
                if constexpr (ET == kOutF16) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(raw.w + k));
                    v[2 * k] = f.x;
                    v[2 * k + 1] = f.y;
                } else {
                    v[2 * k] = __uint_as_float(raw.w[k] << 16);
                    v[2 * k + 1] = __uint_as_float(raw.w[k] & 0xffff0000u);
                }
            }
        }
    }
    static __device__ __forceinline__ void store(void *row, int64_t i, const float (&v)[V])
    {
        if constexpr (V == 1) {
            if constexpr (ET == kOutF32)
                static_cast<float *>(row)[i] = v[0];
            else if constexpr (ET == kOutF16)
                static_cast<__half *>(row)[i] = __float2half_rn(v[0]);
            else
                static_cast<__nv_bfloat16 *>(row)[i] = __float2bfloat16_rn(v[0]);
        } else {
            uint32_t w[BYTES / 4];
#pragma unroll
            for (int k = 0; k < BYTES / 4; ++k) {
                if constexpr (ET == kOutF32) {
                    w[k] = __float_as_uint(v[k]);
                } else if constexpr (ET == kOutF16) {
                    const __half2 h = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
                    w[k] = *reinterpret_cast<const uint32_t *>(&h);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
                    w[k] = *reinterpret_cast<const uint32_t *>(&h);
                }
            }
            if constexpr (BYTES == 16)
                static_cast<uint4 *>(row)[i] = make_uint4(w[0], w[1], w[2], w[3]);
            else
                static_cast<uint32_t *>(row)[i] = w[0];
        }
    }
};

}  // namespace tsm
