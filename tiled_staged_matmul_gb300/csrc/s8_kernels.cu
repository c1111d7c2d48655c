// s8_kernels.cu -- products of 8-bit integers with a scale per row and per
// column:
//
//   C[i][j] = act(alpha * scale_a[i] * scale_b[j] * S[i][j] + bias[j]),
//   S[i][j] = sum_k A[i][k] B[k][j]   (a 32-bit integer sum, exact)
//
// One 64 x 64 tile per block, K in steps of 32: both operands are staged in
// shared memory as words of four consecutive k (B's bytes transposed on the
// way in), each thread adds four-way byte products into a 4 x 4 block.
#include "gemm_kernel.cuh"
#include "ops_internal.h"

namespace tsm {

namespace {

constexpr int kSimpleTile = 64, kSimpleK = 32;

__global__ void __launch_bounds__(256) tsm_s8_simple_kernel(S8Params p)
{
    __shared__ int32_t as[kSimpleK / 4][kSimpleTile + 1];
    __shared__ int32_t bs[kSimpleK / 4][kSimpleTile + 1];
    const int64_t z = blockIdx.z;
    const int rows = p.group_rows ? min(max(p.group_rows[z], 0), p.M) : p.M;
    if (p.group_rows && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0 &&
        (p.group_rows[z] < 0 || p.group_rows[z] > p.M))
        atomicOr(p.status, kStatusGroupRows);
    const int64_t m0 = int64_t(blockIdx.y) * kSimpleTile;
    const int64_t n0 = int64_t(blockIdx.x) * kSimpleTile;
    if (m0 >= rows)
        return;
    const int8_t *A = p.A + z * p.sA, *B = p.B + z * p.sB;
    const int tx = int(threadIdx.x & 15), ty = int(threadIdx.x >> 4);
    int32_t acc[4][4] = {};
    for (int32_t k0 = 0; k0 < p.K; k0 += kSimpleK) {
        for (int i = int(threadIdx.x); i < kSimpleTile * (kSimpleK / 4); i += 256) {
            const int64_t m = m0 + i / (kSimpleK / 4);
            const int kq = i % (kSimpleK / 4);
            uint32_t w = 0;
            for (int b = 0; b < 4; ++b) {
                const int64_t k = int64_t(k0) + 4 * kq + b;
                if (m < rows && k < p.K)
                    w |= uint32_t(uint8_t(A[m * p.lda + k])) << (8 * b);
            }
            as[kq][i / (kSimpleK / 4)] = int32_t(w);
        }
        for (int i = int(threadIdx.x); i < kSimpleTile * (kSimpleK / 4); i += 256) {
            const int64_t n = n0 + i % kSimpleTile;
            const int kq = i / kSimpleTile;
            uint32_t w = 0;
            for (int b = 0; b < 4; ++b) {
                const int64_t k = int64_t(k0) + 4 * kq + b;
                if (n < p.N && k < p.K)
                    w |= uint32_t(uint8_t(B[k * p.ldb + n])) << (8 * b);
            }
            bs[kq][i % kSimpleTile] = int32_t(w);
        }
        __syncthreads();
#pragma unroll
        for (int kq = 0; kq < kSimpleK / 4; ++kq)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __dp4a(as[kq][ty * 4 + i], bs[kq][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        for (int j = 0; j < 4; ++j) {
            const int64_t n = n0 + tx + 16 * j;
            if (m >= rows || n >= p.N)
                continue;
            float v = float(acc[i][j]);
            if (p.scale_a)
                v *= p.scale_a[z * p.sa_stride + m];
            if (p.scale_b)
                v *= p.scale_b[z * p.sb_stride + n];
            const float bias = p.epi.bias ? p.epi.bias[z * p.epi.bias_stride + n] : 0.f;
            epi_store(p.C, z * p.sC + m * p.ldc + n, epi_value(v, bias, p.epi), p.epi.out_type);
        }
    }
}

}  // namespace

cudaError_t launch_s8_simple(const S8Params &p, cudaStream_t stream)
{
    const dim3 grid(unsigned((p.N + kSimpleTile - 1) / kSimpleTile),
                    unsigned((p.M + kSimpleTile - 1) / kSimpleTile), unsigned(p.batch));
    tsm_s8_simple_kernel<<<grid, 256, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace tsm
