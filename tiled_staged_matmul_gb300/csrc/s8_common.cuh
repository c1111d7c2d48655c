// s8_common.cuh -- products of 8-bit integers with a scale per row and per
// column:
//
//   C[i][j] = act(alpha * scale_a[i] * scale_b[j] * S[i][j] + bias[j]),
//   S[i][j] = sum_k A[i][k] B[k][j]   (the exact 32-bit integer)
//
// The tensor cores' rate for 8-bit integers on this part is a small fraction
// of their f16 rate, but f16 holds every integer up to 2048 exactly, so the
// f16 pipe can do the work: a product of two codes is at most 2^14, exact in
// the f32 accumulator, and so is the sum of 1024 of them (2^24).  The kernels
// therefore feed the codes as f16 and take the accumulator out into 32-bit
// integers every 1024 of K: S is exact, whatever the order of the pieces.
//
// A code becomes f16 without a conversion instruction: byte c of a word, sign
// bit flipped (c + 128), placed below the byte 0x64 is the f16 number
// 1024 + (c + 128); subtracting 1152 leaves c, exactly.  Five instructions
// turn four codes into two f16 pairs.
#pragma once

#include "gemm_kernel.cuh"
#include "launch.cuh"
#include "ops_internal.h"
#include "s8_ptx.cuh"

namespace tsm {

// Four codes (k, k+1, k+2, k+3 of a word) as two f16 pairs.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t l = __byte_perm(u, 0x64646464u, 0x4140);
    const uint32_t h = __byte_perm(u, 0x64646464u, 0x4342);
    const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&l), off);
    const __half2 b = __hsub2(*reinterpret_cast<const __half2 *>(&h), off);
    lo = *reinterpret_cast<const uint32_t *>(&a);
    hi = *reinterpret_cast<const uint32_t *>(&b);
}

// The tiled kernel's shape (s8_tiled.cu).  PAIR: a CTA pair per 256 x 256 tile,
// else one CTA per 128 x 128.
template <bool PAIR>
struct S8Cfg {
    static constexpr int ROWS = 128;
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int TILE_M = ROWS * CTAS;
    static constexpr int B_COLS = 128;          // columns of B staged by one CTA
    static constexpr int TILE_N = B_COLS * CTAS;  // the MMA's width
    static constexpr int GROUPS = 4;            // groups of four epilogue warps, one per warp of TMEM lanes
    static constexpr int HC = TILE_N / GROUPS;  // columns of one group
    static constexpr int BK = 128;
    static constexpr int A_CODES = ROWS * BK;   // bytes
    static constexpr int B_CODES = B_COLS * BK;
    static constexpr int CODE_STAGE = A_CODES + B_CODES;
    static constexpr int F_BOX = 64 * BK * 2;   // 64 columns of f16
    static constexpr int F_STAGE = 2 * F_BOX;
    static constexpr int S1 = 3, S2 = 3;        // ring depths
    static constexpr int STAGING = 4 * GROUPS * 32 * 32;  // per epilogue warp: 32 rows of 32 bytes
    static constexpr uint32_t GROUP_TERMS = (2 * HC + ROWS) * 4;  // a group's columns' scales and biases, rows' scales
    static constexpr uint32_t TERMS = GROUPS * GROUP_TERMS;
    static constexpr int GROUP_TABLE_OFF = 1024, GROUP_ROWS_OFF = 2048, TERMS_OFF = GROUP_ROWS_OFF + 1024;
    static constexpr int CTRL = TERMS_OFF + 2 * TERMS;
    static constexpr int SMEM_BYTES = 1024 + S1 * CODE_STAGE + S2 * F_STAGE + STAGING + CTRL;
    static_assert(SMEM_BYTES <= 232448, "227 KiB per block");
    static constexpr uint32_t A_COL = 256;      // TMEM: the accumulator, then the f16 A ring
    static_assert(A_COL + S2 * (BK / 2) <= 512 && TILE_N <= 256, "TMEM columns");
    static constexpr int PARTS = GROUPS * CTAS; // (CTA, group) parts of a tile
    static constexpr int32_t SLOT_INTS = PARTS * ROWS * HC;
    static constexpr S8Shape SHAPE = s8_shape(PAIR ? S8Kind::kPair : S8Kind::kOne);
    static_assert(SHAPE.tile_m == TILE_M && SHAPE.tile_n == TILE_N && SHAPE.block_k == BK &&
                  SHAPE.slot_bytes == 4 * SLOT_INTS && SHAPE.parts == PARTS, "the host's idea of a tile");
};

// Where a tile lies.
struct S8Tile {
    int32_t m0, n0, z, rows;
};

// A grouped launch's tables in shared memory, built by one warp: gtab[g], the
// tiles of groups 0 ... g, and grows[g], group g's rows, clamped to [0, M] (a
// count outside raises kStatusGroupRows).  Eight groups a lane, all their loads
// at once: one after another they took 4 us, a third of a decode step's start.
template <int TILE_M>
static __device__ __noinline__ void build_s8_groups(const S8Params &p, uint32_t gtab, uint32_t grows)
{
    constexpr int PER = kMaxGroupsPerLaunch / 32;
    const int lane = int(threadIdx.x & 31);
    int32_t rows[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        rows[i] = __ldcg(p.group_rows + min(lane * PER + i, p.batch - 1));
    uint32_t sum = 0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int32_t r = min(max(rows[i], 0), p.M);
        bad |= r != rows[i];
        rows[i] = r;
        if (lane * PER + i < p.batch)
            sum += uint32_t(r + TILE_M - 1) / TILE_M * uint32_t(p.tiles_n);
    }
    uint32_t scan = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, scan, d);
        if (lane >= d)
            scan += v;
    }
    uint32_t before = scan - sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int g = lane * PER + i;
        if (g < p.batch) {
            before += uint32_t(rows[i] + TILE_M - 1) / TILE_M * uint32_t(p.tiles_n);
            ptx::st_shared_u32(gtab + 4u * g, before);
            ptx::st_shared_u32(grows + 4u * g, uint32_t(rows[i]));
        }
    }
    if (bad)
        atomicOr(p.status, kStatusGroupRows);
    __syncwarp();
}

// The group of a grouped launch's tile; the tile's place in it goes to `tile`.
__device__ __forceinline__ int32_t group_of(int32_t &tile, int32_t groups, uint32_t gtab)
{
    int32_t lo = 0, hi = groups - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi) >> 1;
        if (int32_t(ptx::ld_shared_u32(gtab + 4u * mid)) > tile)
            hi = mid;
        else
            lo = mid + 1;
    }
    if (lo)
        tile -= int32_t(ptx::ld_shared_u32(gtab + 4u * (lo - 1)));
    return lo;
}

// Where the tiled kernel's tiles lie: kRasterRows rows of tiles are walked
// together, column by column.  (Few divisions: each is 0.1 us before the first
// load.)
constexpr int kRasterRows = 8;

__device__ __forceinline__ S8Tile tile_at(int32_t t, const S8Params &p, uint32_t gtab, uint32_t grows, int tile_m, int tile_n)
{
    S8Tile w = {0, 0, 0, p.M};
    int32_t tiles_m = p.tiles_m;
    if (p.group_rows) {
        w.z = group_of(t, p.batch, gtab);
        w.rows = int32_t(ptx::ld_shared_u32(grows + 4u * w.z));
        tiles_m = (w.rows + tile_m - 1) / tile_m;
    } else if (p.batch > 1) {
        const int32_t per = p.tiles_m * p.tiles_n;
        w.z = t / per;
        t -= w.z * per;
    }
    int32_t first_m = 0;
    if (tiles_m > kRasterRows) {
        const int32_t group = kRasterRows * p.tiles_n;
        const int32_t g = t / group;
        first_m = g * kRasterRows;
        t -= g * group;
    }
    const int32_t in_group = min(tiles_m - first_m, kRasterRows);
    int32_t n;
    if (in_group == kRasterRows)
        n = t / kRasterRows;
    else if (in_group == 1)
        n = t;
    else
        n = t / in_group;
    w.m0 = (first_m + t - n * in_group) * tile_m;
    w.n0 = n * tile_n;
    return w;
}

// Bounded mbarrier wait, as wait_bounded, with nothing kept in registers
// between waits: the CTA's abort flag is the word at `flag` in shared memory
// (in a pair, at the same place in the peer), the limit and the status word
// are the launch's.  ACQ_CLUSTER: the phase counts another CTA's arrivals.
template <bool PAIR, bool ACQ_CLUSTER = false>
__device__ __forceinline__ bool s8_wait(uint32_t bar, uint32_t parity, uint32_t flag, const S8Params &p, uint32_t who,
                                        bool honor_abort = true)
{
    auto try_wait = [&]() {
        return ACQ_CLUSTER ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity);
    };
    if (try_wait())
        return true;
    const uint64_t t0 = ptx::globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (try_wait())
            return true;
        if ((it & 31u) == 0) {
            if (honor_abort && ptx::ld_shared_u32(flag))
                return false;
            if (ptx::globaltimer_ns() - t0 > p.timeout_ns) {
                ptx::st_shared_u32(flag, 1u);
                if (PAIR)
                    ptx::st_cluster_u32(ptx::mapa_shared(flag, ptx::cluster_ctarank() ^ 1u), 1u);
                atomicOr(p.status, who);
                return false;
            }
        }
    }
}

}  // namespace tsm
