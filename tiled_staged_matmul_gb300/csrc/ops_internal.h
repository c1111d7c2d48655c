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
    int32_t *hist;        // chunks x groups counts per chunk; null: one chunk, or one cluster of them
    int64_t n;            // tokens x choices
    int32_t groups;
    int32_t capacity;
};
// One CTA ranks kRouteChunk(rounds) assignments.
constexpr int kRouteWarps = 16;
constexpr int kRouteRoundsSmall = 2, kRouteRoundsCluster = 8, kRouteRoundsLarge = 16;
constexpr int kRouteCluster = 8;  // chunks that one cluster holds
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
// `bytes` of one access: 16, 4 or an element's; every row is aligned to it and a
// multiple of it long.
cudaError_t launch_combine(const MoveParams &p, int elem, int bytes, int sms, cudaStream_t stream);
cudaError_t launch_combine_grad(const MoveParams &p, int elem, int bytes, int sms, cudaStream_t stream);

// ------------------------------------------------------------- row quantisation

struct QuantParams {
    const void *X;           // batch x M rows of K, ldx / strideX apart
    int8_t *q;               // ldq / strideQ apart
    float *scales;           // batch x M, stride_s apart
    const int32_t *group_rows;  // null, or the rows of each batch that are computed
    int64_t M, K, ldx, ldq, sX, sQ, sS, batch;
};
cudaError_t launch_quantize_rows(const QuantParams &p, int elem, int bytes, int sms, cudaStream_t stream);

// ------------------------------------------------------------- int8 products

// The work of one tiled launch: `tiles` output tiles of `kb` k-blocks each, spread
// over `workers` CTAs (or CTA pairs).  Where that pays, as many whole waves of
// tiles as leave between one and two waves over run tile by tile, and the tiles
// left over (the first `shared` ones) are cut as one long row of shared * kb
// blocks into equal pieces, one per worker, which starts with its piece.  A tile that
// several workers hold pieces of is summed by the one that arrives last, in
// integers, so the order does not matter.
struct S8Schedule {
    int32_t tiles;
    int32_t shared;         // tiles cut into pieces: 0 .. shared - 1 (fewer than two per worker)
    int32_t kb;
    int32_t workers;        // of the whole tiles
    int32_t cutters;        // workers that get a piece
    static constexpr int32_t kMaxTiles = 1 << 30;
    // What a cut costs, in blocks' time.  Whole against cut, us: 300 x 5000 x 8192
    // 74.6 and 65.6, 128 x 4096 x 4096 26.6 and 19.8, 4096^3 106.1 and 104.3; 512 x
    // 14336 x 4096 56.9 and 58.7, 64 x 14336 x 4096 27.0 and 29.4.  16 decides all
    // of these right (6 and 24 do not).
    static constexpr int32_t kCutBlocks = 16;

    int32_t price;          // of a cut

    // `part`: the last contributor's time for one of the others' sums, in quarters
    // of a block's time.
    __host__ __device__ void plan(int32_t tiles_, int32_t kb_, int32_t workers_, int32_t price_ = kCutBlocks, int32_t part = 8)
    {
        tiles = tiles_;
        kb = kb_;
        workers = workers_;
        price = price_;
        const int32_t over = tiles % workers;
        shared = over == 0 ? 0 : tiles < workers ? tiles : over + workers;
        // A tile's contributors: as many as balance the blocks each multiplies
        // with the sums the last one adds up.
        int32_t each = 1;
        while (part * each * each < 4 * kb)
            ++each;
        const int32_t pieces = shared * each;
        cutters = pieces < 1 ? 1 : pieces < workers ? pieces : workers;
        // Cutting has its price: pieces' sums written, arrivals, sums read
        // back.  Whole tiles all the way where the last wave costs no more.
        if (shared && int64_t((tiles + workers - 1) / workers) * kb <= blocks()) {
            shared = 0;
            cutters = 1;
        }
    }
    // The time of the busiest worker, in blocks.
    __host__ __device__ int64_t blocks() const
    {
        return shared ? int64_t((tiles - shared) / workers) * kb + (shared * kb + cutters - 1) / cutters + price
                      : int64_t((tiles + workers - 1) / workers) * kb;
    }
    // First block of worker w's piece (w <= cutters).
    __host__ __device__ int32_t piece_begin(int32_t w) const { return shared * kb * w / cutters; }
    // The worker whose piece holds block x.
    __host__ __device__ int32_t owner(int32_t x) const { return ((x + 1) * cutters - 1) / (shared * kb); }
};

// Arguments of a product (device pointers; strides in elements).
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
    // What the launch adds.
    uint32_t *status;
    uint64_t timeout_ns;
    int32_t tiles_m, tiles_n, kb;
    S8Schedule sched;           // tiled kernels, unless grouped (then it is made on the device)
    int32_t workers;
    int32_t ranks;              // few rows: CTAs (a cluster) that cut a tile's K,
    int32_t kb_each, kb_more;   // blocks for each, and how many take one more
    int32_t vec_c;              // C's rows are 16-byte aligned
    int32_t *partial;           // sums of pieces: two slots per worker
    unsigned long long *arrivals;  // one word per part of a shared tile: launch tag, count
    unsigned long long tag;     // 48 bits of a hash of the launch's number (a word's old contents have them by
                                // chance once in 2^48)
};

// The kernels: few rows (up to 16 or 32, 256 columns a tile); tiled, one CTA per
// 128 x 128 tile or a CTA pair per 256 x 256.
enum class S8Kind { kFew16, kFew32, kOne, kPair };
struct S8Shape {
    int tile_m, tile_n, block_k;
    int64_t slot_bytes;         // of one worker's partial sums of one tile
    int parts;                  // arrival words per tile
};
constexpr S8Shape kS8Shapes[] = {
    {16, 256, 32, 0, 0}, {32, 256, 32, 0, 0}, {128, 128, 128, 65536, 4}, {256, 256, 128, 262144, 8}};
constexpr S8Shape s8_shape(S8Kind kind) { return kS8Shapes[int(kind)]; }
// Clusters of 1 to 8 CTAs of the few-rows kernels that fit on the device at once.
struct S8Capacity {
    static constexpr int KINDS = 8;
    int clusters[KINDS];
};
cudaError_t set_s8_attributes(S8Capacity *cap);
// The tiled kernels for activation ACT (s8_tiled.cu, one unit per activation).
template <int ACT>
cudaError_t set_s8_tiled();
template <int ACT>
cudaError_t launch_s8_tiled(const CUtensorMap &map_a, const CUtensorMap &map_b, const S8Params &p, bool pair, int grid,
                            cudaStream_t stream);
cudaError_t launch_s8(const CUtensorMap &map_a, const CUtensorMap &map_b, const S8Params &p, S8Kind kind, int grid,
                      cudaStream_t stream);
// Raises kStatusGroupRows where a count is outside [0, M] (the products above do so themselves).
cudaError_t launch_s8_counts(const S8Params &p, cudaStream_t stream);
// Rows of `cols` bytes into rows 16-byte aligned and `d_ld` apart.
cudaError_t launch_pack_s8(const int8_t *src, int64_t s_ld, int64_t s_stride, int8_t *dst, int64_t d_ld,
                           int64_t d_stride, int64_t rows, int64_t cols, int64_t batch, int sms,
                           cudaStream_t stream);

}  // namespace tsm
