// fp4_internal.h -- what the host side (fp4_api.cu) and the kernels
// (fp4_quantize.cu, fp4_product.cu) of the microscaled 4-bit operators share.
// Not part of the public ABI.
#pragma once

#include "ops_internal.h"

namespace tsm {

// Block scales are kept in tiles of 512 bytes: 128 rows by 4 blocks, the byte of
// row r and block b at 16 (r % 32) + 4 (r / 32) + b -- the order in which the
// tensor cores take them from TMEM, so that a product's loads are plain copies.
// A matrix has ceil(rows / 128) rows of ceil(blocks / 4) tiles.
constexpr int kScaleTile = 512;
constexpr int64_t scale_tile_rows(int64_t rows) { return (rows + 127) / 128; }
constexpr int64_t scale_tile_cols(int64_t K, int block) { return ((K + block - 1) / block + 3) / 4; }

struct Fp4QuantParams {
    const void *X;              // batch x M rows of K, ldx / strideX apart
    uint8_t *q;                 // two codes a byte, ldq / strideQ bytes apart
    uint8_t *block_scales;      // tiles, matrices one after another
    float *scales;              // blocks of 16: batch x M, sS apart
    const int32_t *group_rows;  // null, or the rows of each batch that are computed
    int64_t M, K, ldx, ldq, sX, sQ, sS, batch;
    int64_t tile_rows, tile_cols;
};
// aligned: rows of X are 16-byte and rows of q 8-byte aligned.
cudaError_t launch_quantize_fp4(const Fp4QuantParams &p, int elem, bool aligned, int block, cudaStream_t stream);

// Arguments of a product (device pointers).  What the kernels call rows are the
// rows of C (tokens), columns are those of C (rows of B).
struct Fp4Params {
    void *C;                    // epi.out_type elements
    const float *scale_a;       // M per matrix, sa_stride apart; null: ones
    const float *scale_b;       // N per matrix, sb_stride apart; null: ones
    int64_t sa_stride, sb_stride;
    int32_t M, N, K, batch;
    int64_t ldc, sC;
    const int32_t *group_rows;  // grouped: the rows of each matrix, clamped to [0, M]; else null
    Epilogue epi;
    // What the launch adds.
    uint32_t *status;
    uint64_t timeout_ns;
    int32_t tiles_m, tiles_n, kb;
    S8Schedule sched;           // unless grouped (then it is made on the device)
    int32_t workers;
    int32_t ranks;              // CTAs (a cluster) that cut a tile's K; 1: the schedule's pieces
    int32_t sched_price, sched_part;
    int32_t scale_rows_a, scale_rows_b;  // rows of scale tiles in a matrix
    int32_t vec_c;              // C's rows are 4-byte aligned (16-bit types: stored in pairs)
    float *partial;             // sums of pieces: two slots per worker
    unsigned long long *arrivals;
    unsigned long long tag;
};

// The kernels: one CTA per tile of 128 columns by 32, 64 or 128 rows, or a CTA
// pair per 256 by 256.
enum class Fp4Kind { kRows32, kRows64, kRows128, kPair };
struct Fp4Shape {
    int tile_m, tile_n;         // rows and columns of C
    int64_t slot_bytes;         // of one worker's partial sums of one tile
    int parts;                  // arrival words per tile
    int32_t price, part;        // S8Schedule::plan's
};
// The prices of a cut, in blocks of 256 k.  Cut where the schedule says so and never,
// us: 16 x 20000 x 16384 37.3 and 47.0, 128 x 20000 x 16384 45.2 and 51.1, 1024 x 5000 x
// 28672 67.0 and 86.1, 2048 x 2560 x 65536 138 and 183, one of 8 experts 3 x 4096 x
// 14336 16.9 and 22.6.  Cut wherever it balances (prices of 0) and as the schedule
// says: 16 x 14336 x 4096 18.6 and 9.7, 97 x 14333 x 4010 22.7 and 11.2, 4096^3 41.1 and
// 31.0.  Parts of 1, 2, 4 and 8 cut a tile further, which few calls notice: one of 8
// experts 512 x 512 x 16384 30.3 us, 27.1 with these.
constexpr Fp4Shape kFp4Shapes[] = {{32, 128, 16384, 4, 20, 8},
                                   {64, 128, 32768, 4, 22, 12},
                                   {128, 128, 65536, 4, 25, 20},
                                   {256, 256, 262144, 8, 30, 32}};
constexpr Fp4Shape fp4_shape(Fp4Kind kind) { return kFp4Shapes[int(kind)]; }
constexpr int kFp4BlockK = 256;  // k of one stage: 128 bytes of a row

struct Fp4Maps {
    CUtensorMap a, b, scales_a, scales_b;
};
// Clusters of 1 to 8 CTAs of the kernels of one CTA that fit on the device at once.
struct Fp4Capacity {
    static constexpr int RANKS = 8;
    int clusters[3][RANKS];
};
cudaError_t set_fp4_attributes(Fp4Capacity *cap);
cudaError_t launch_fp4(const Fp4Maps &maps, const Fp4Params &p, Fp4Kind kind, int block, int grid, cudaStream_t stream);

// ------------------------------------------------------------- choice of experts

struct ChooseParams {
    const void *logits;         // tokens x experts, ld apart
    const float *bias;          // experts, or null
    int32_t *ids;               // tokens x topk
    float *weights;             // tokens x topk
    const float *dweights;      // gradient: tokens x topk
    void *dlogits;              // gradient: tokens x experts, ld_d apart
    int64_t tokens, ld, ld_d;
    int32_t experts, topk, groups, keep, best;
    int32_t sigmoid, renormalize;
    float scale;
    // What the launch adds: experts of a group, and its lanes' logarithm.
    int32_t per, lanes_log;
};
constexpr int kMaxChooseExperts = 1024, kMaxChooseTopk = 32, kMaxChooseGroups = 32;
// Experts where the groups are not a power of two: they leave lanes of the warp idle.
constexpr int kMaxChooseUneven = 512;
// By the logits' type (choose_kernels.cu, one unit each).  aligned: rows are
// 16-byte aligned.
template <int ET>
cudaError_t launch_choose(const ChooseParams &p, bool aligned, int sms, cudaStream_t stream);
template <int ET>
cudaError_t launch_choose_grad(const ChooseParams &p, bool aligned, int sms, cudaStream_t stream);
#define TSM_CHOOSE_OF(ET)                                                                \
    template <>                                                                          \
    cudaError_t launch_choose<ET>(const ChooseParams &, bool, int, cudaStream_t);        \
    template <>                                                                          \
    cudaError_t launch_choose_grad<ET>(const ChooseParams &, bool, int, cudaStream_t)
TSM_CHOOSE_OF(kOutF32);
TSM_CHOOSE_OF(kOutF16);
TSM_CHOOSE_OF(kOutBF16);
#undef TSM_CHOOSE_OF

}  // namespace tsm
