// s8_kernels.cu -- the 8-bit products' kernel for few rows, the repacking of
// operands that TMA cannot address, and the launches (s8_common.cuh says what
// is computed; s8_tiled.cu holds the tiled kernels).
#include "s8_common.cuh"

namespace tsm {

namespace {

// ------------------------------------------------------------- few rows
//
// Up to 32 rows of A (a decode step): the product reads every code of B once
// and is bound by that.  A tile is 256 columns; its K is cut over the CTAs of a
// cluster (up to 8 of them, by a time model on the host).  In a CTA,
// independent warps in pairs take 32 k of the tile at a time, one warp for each
// 128 columns, so that a row of B is read 256 bytes at a time (reading 128
// bytes of it ran at 4.6 TB/s, 256 at 6.0, 512 no faster).  Each warp has a TMA
// ring of its own and never waits for another.  Measured: 16 x 57344 x 8192
// 80.5 us, 5.9 TB/s (0.88 of the copy rate); 16 x 14336 x 4096 18.4 us and 1 x
// 4096 x 4096 9.3, where a kernel that does nothing but read B takes 13.0 and
// 6.4.
//
// Warp-wide f16 MMAs (16 x 8 x 16 k) run far below the tcgen05 rate, but so few
// rows need no more: one SM's share of the memory rate is 23 codes a cycle, 23
// multiply-adds a row, and the warps' MMAs do about 500.  C^T = B^T A^T is what
// they compute: the wide side of an MMA is 16 of B's columns, the narrow one 8
// rows, so that 8 rows or fewer (one token, most experts of a decode step) take
// half the MMAs that 16 take (64 experts of 1 to 16 rows: 49 -> 44 us).
//
// B's codes go from shared memory to the MMA's operand layout in registers:
// lane 4g + t takes 16 columns (chunk g) of rows 4t ... 4t + 3, and a byte of
// two rows each makes the f16 pair that it has to hold for one column.  Which
// columns and which k a lane's registers stand for is free as long as A's lanes
// agree, so no transpose is needed: rows g and g + 8 of MMA j of 8 are columns
// 16 g + 2j and 16 g + 2j + 1, and k index 2t, 2t + 1, 2t + 8, 2t + 9 is row 4t,
// 4t + 1, 4t + 2, 4t + 3.
//
// A warp's f32 sums go into the CTA's 32-bit ones in shared memory (integer
// atomics: any order gives the same sum) after at most 1024 k.  There are two
// sets of those: four more warps take a finished tile on while the others go on
// with the next.  Each CTA of the cluster finishes its share of the tile: it
// adds up that share of every CTA's sums through distributed shared memory, so
// nothing passes through the workspace (which, with its fences and arrivals,
// cost a tile's end three to five microseconds, this about one).
template <int MT>
struct S8FewCfg {
    static constexpr int ROWS = 16 * MT, COLS = 256, BK = 32;
    static constexpr int WARPS = MT == 1 ? 16 : 8, FINISHERS = 4, STAGES = MT == 1 ? 2 : 3;
    static constexpr int THREADS = 32 * (WARPS + FINISHERS);
    static constexpr int KWARPS = WARPS / 2;  // warps along k
    static constexpr int B_BYTES = BK * 128, A_BYTES = ROWS * BK;
    static constexpr int HALF_SUMS = ROWS * 128;  // of 128 columns (few_rows_sum)
    static constexpr int SUMS = 2 * HALF_SUMS;
    static constexpr int CTRL = 6144, GROUP_TABLE_OFF = 1024, TERMS_OFF = 2048, GROUP_ROWS_OFF = 4608;
    static_assert(TERMS_OFF + 4 * (2 * COLS + ROWS) <= GROUP_ROWS_OFF && kMaxGroupsPerLaunch <= 256, "control block");
    static constexpr int SMEM_BYTES = 1024 + WARPS * STAGES * (B_BYTES + A_BYTES) + 2 * SUMS * 4 + CTRL;
    static_assert(SMEM_BYTES <= 232448 && SMEM_BYTES > 232448 / 2, "227 KiB per block, one block per SM");
    static constexpr S8Shape SHAPE = s8_shape(MT == 1 ? S8Kind::kFew16 : S8Kind::kFew32);
    static_assert(SHAPE.tile_m == ROWS && SHAPE.tile_n == COLS && SHAPE.block_k == BK, "the host's idea of a tile");
    static constexpr int FLUSH = 1024 / BK;   // blocks whose sums f32 holds exactly
    // Registers by role: the MMA warps' accumulators need more than an even share.
    static constexpr int LAUNCH_REGS = MT == 1 ? 96 : 168;
    static constexpr int MMA_REGS = MT == 1 ? 104 : 208, FINISH_REGS = MT == 1 ? 64 : 88;
    static_assert(32 * (WARPS * MMA_REGS + FINISHERS * FINISH_REGS) <= THREADS * LAUNCH_REGS, "register split");
};

// Column pair of a byte column: f16(lo.byte b), f16(hi.byte b).
template <int B>
__device__ __forceinline__ uint32_t code_pair(uint32_t lo, uint32_t hi)
{
    const uint32_t v = (__byte_perm(lo, hi, 0x0400 + 0x0101 * B) & 0x00ff00ffu) ^ 0x64806480u;
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&v), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t *>(&x);
}

// Where a half's sums are kept: rows in groups of eight, then column bit 4, the
// row, and chunks of the four columns 32 apart, column j's chunk at j ^ row ^
// bit 4 -- so that the lanes of an accumulator value (four rows of eight
// columns 16 apart) add to different banks, and sixteen threads read sixteen
// neighbouring columns' chunks.
__device__ __forceinline__ constexpr int few_rows_sum(int octet, int d1, int row, int j, int t)
{
    return ((octet * 2 + d1) * 8 + row) * 64 + 4 * (j ^ row ^ d1) + t;
}

// A CTA's addresses and place in the launch.
struct FewPlace {
    uint32_t sums0, terms0;                       // shared memory: [2][SUMS] ints; scales and biases
    uint32_t sums_full0, sums_free0, ready0, taken0;  // barriers, [2] each
    uint32_t flag, gtab, grows;                   // ...; the groups' tiles, summed, and their rows
    int32_t tiles, cluster, clusters, rank, ranks;
    int32_t last, last_set;                       // the CTA's last tile, and the sums it is in
};

// Where a tile lies; `rows` is its own number of them.  (Short of divisions:
// the first block waits for this.  A matrix has one tile along M, a group at
// most two.)
template <int MT>
__device__ __forceinline__ S8Tile few_rows_tile(const S8Params &p, const FewPlace &f, int32_t tile)
{
    using Cfg = S8FewCfg<MT>;
    S8Tile t = {0, tile, 0, p.M};
    if (p.group_rows) {
        int32_t i = tile;
        t.z = group_of(i, p.batch, f.gtab);
        t.rows = int32_t(ptx::ld_shared_u32(f.grows + 4u * t.z));
        const int two = t.rows > Cfg::ROWS;
        t.m0 = (i & two) * Cfg::ROWS;
        t.n0 = i >> two;
    } else if (p.batch > 1) {
        t.z = tile / p.tiles_n;
        t.n0 = tile - t.z * p.tiles_n;
    }
    t.n0 *= Cfg::COLS;
    t.rows = min(t.rows - t.m0, Cfg::ROWS);
    return t;
}

// Before the first tile: the sums are clear, and the CTA's barriers exist.
template <int MT>
__device__ __forceinline__ void few_rows_start(const FewPlace &f)
{
    using Cfg = S8FewCfg<MT>;
    for (int i = int(threadIdx.x); i < 2 * Cfg::SUMS / 4; i += Cfg::THREADS)
        ptx::st_shared_v4(f.sums0 + 16u * i, 0u, 0u, 0u, 0u);
    ptx::cta_sync();
}

// The first thing of a tile's end: the terms of its epilogue, while the sums
// are on their way (the finishing warps').
template <int MT>
__device__ __forceinline__ S8Tile few_rows_terms(const S8Params &p, const FewPlace &f, int32_t tile, int ft)
{
    using Cfg = S8FewCfg<MT>;
    constexpr int FT = 32 * Cfg::FINISHERS;
    const S8Tile t = few_rows_tile<MT>(p, f, tile);
    for (int c = ft; c < Cfg::COLS; c += FT) {
        const int32_t col = t.n0 + c;
        float sb = 1.f, bias = 0.f;
        if (p.scale_b && col < p.N)
            sb = p.scale_b[t.z * p.sb_stride + col];
        if (p.epi.bias && col < p.N)
            bias = p.epi.bias[t.z * p.epi.bias_stride + col];
        ptx::st_shared_u32(f.terms0 + 4u * c, __float_as_uint(sb));
        ptx::st_shared_u32(f.terms0 + 4u * (Cfg::COLS + c), __float_as_uint(bias));
    }
    // (alpha goes into the row's factor, as in the tiled kernels: a row's bits are
    // the same whichever kernel its call takes.)
    if (ft < Cfg::ROWS)
        ptx::st_shared_u32(f.terms0 + 4u * (2 * Cfg::COLS + ft),
                           __float_as_uint(p.epi.alpha * (p.scale_a && ft < t.rows
                                                              ? p.scale_a[t.z * p.sa_stride + t.m0 + ft] : 1.f)));
    return t;
}

// This CTA's share of a tile: the cluster's sums through the epilogue into C,
// by `threads` threads.  In chunks of four columns 32 apart, two rows' sixteen
// a warp; rows past the last are left out in eights.
template <int MT>
__device__ __forceinline__ void few_rows_share(const S8Params &p, const FewPlace &f, const S8Tile &t, uint32_t sums,
                                               int thread, int threads)
{
    using Cfg = S8FewCfg<MT>;
    const uint32_t sb0 = f.terms0, bias0 = f.terms0 + 4u * Cfg::COLS, sa0 = f.terms0 + 8u * Cfg::COLS;
    const int octets = (t.rows + 7) / 8, lane = thread & 31;
    for (int u = f.rank + f.ranks * (thread >> 5); u < 16 * octets; u += f.ranks * (threads >> 5)) {
        const int i = 32 * u + lane;
        const int j = i & 15, r8 = (i >> 4) & 7, d1 = (i >> 7) & 1, ho = i >> 8;
        const int h = ho >= octets, octet = ho - h * octets;
        const int row = 8 * octet + r8;
        if (row >= t.rows)
            continue;
        const uint32_t at = sums + 4u * uint32_t(h * Cfg::HALF_SUMS + few_rows_sum(octet, d1, r8, j, 0));
        // Every CTA's chunk on its way at once.
        uint4 x[8];
        int32_t v[4] = {};
#pragma unroll
        for (int r = 0; r < 8; ++r)
            x[r] = r < f.ranks ? ptx::ld_cluster_v4(ptx::mapa_shared(at, uint32_t(r))) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            v[0] += int32_t(x[r].x);
            v[1] += int32_t(x[r].y);
            v[2] += int32_t(x[r].z);
            v[3] += int32_t(x[r].w);
        }
        const float sa = __uint_as_float(ptx::ld_shared_u32(sa0 + 4u * row));
        const int c = 128 * h + 16 * d1 + j;
        const int64_t row_at = t.z * p.sC + int64_t(t.m0 + row) * p.ldc + t.n0;
        const int32_t columns = p.N - t.n0;
        with_activation<kActRuntime>(p.epi.act, [&](auto act) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float sb = __uint_as_float(ptx::ld_shared_u32(sb0 + 4u * (c + 32 * k)));
                const float bias = __uint_as_float(ptx::ld_shared_u32(bias0 + 4u * (c + 32 * k)));
                const float o = epi_act(fmaf(sb, float(v[k]) * sa, bias), decltype(act)::value, p.epi.slope);
                if (c + 32 * k < columns)
                    epi_store(p.C, row_at + c + 32 * k, o, p.epi.out_type);
            }
        });
    }
}

// The finishing warps: every tile but the CTA's last, whose terms they fetch.
template <int MT>
__device__ __forceinline__ bool few_rows_finish(const S8Params &p, FewPlace &f)
{
    using Cfg = S8FewCfg<MT>;
    constexpr int FT = 32 * Cfg::FINISHERS;
    const int ft = int(threadIdx.x) - 32 * Cfg::WARPS;
    uint32_t set = 0, phase = 0;
    for (int32_t tile = f.cluster; tile < f.tiles; tile += f.clusters) {
        const S8Tile t = few_rows_terms<MT>(p, f, tile, ft);
        f.last = tile;
        f.last_set = int32_t(set);
        if (f.tiles - tile <= f.clusters)
            break;
        const uint32_t sums = f.sums0 + set * uint32_t(Cfg::SUMS * 4);
        bool ok = s8_wait<false>(f.sums_full0 + 8u * set, phase, f.flag, p, kStatusEpilogue);
        ok = __all_sync(0xffffffffu, ptx::named_bar_and(1, FT, ok));
        if (!ok)
            return false;
        if (f.ranks > 1) {
            // This CTA's sums are complete: so says one thread to every CTA.
            if (ft < f.ranks)
                ptx::mbar_arrive_cluster(ptx::mapa_shared(f.ready0 + 8u * set, uint32_t(ft)));
            ok = s8_wait<false, true>(f.ready0 + 8u * set, phase, f.flag, p, kStatusReduce);
            ok = __all_sync(0xffffffffu, ptx::named_bar_and(1, FT, ok));
            if (!ok)
                return false;
        }
        few_rows_share<MT>(p, f, t, sums, ft, FT);
        ptx::named_bar_sync(1, FT);  // the sums and the terms have been read here
        if (f.tiles - tile > 2 * f.clusters) {  // (else the set is not used again)
            if (f.ranks > 1) {
                // ... and in every CTA of the cluster, before they are cleared.
                if (ft < f.ranks)
                    ptx::mbar_arrive_cluster(ptx::mapa_shared(f.taken0 + 8u * set, uint32_t(ft)));
                ok = s8_wait<false, true>(f.taken0 + 8u * set, phase, f.flag, p, kStatusReduce);
                ok = __all_sync(0xffffffffu, ptx::named_bar_and(1, FT, ok));
                if (!ok)
                    return false;
            }
            for (int i = ft; i < Cfg::SUMS / 4; i += FT)
                ptx::st_shared_v4(sums + 16u * i, 0u, 0u, 0u, 0u);
            ptx::named_bar_sync(1, FT);
            if (ft == 0)
                ptx::mbar_arrive(f.sums_free0 + 8u * set);
        }
        set ^= 1u;
        if (set == 0)
            phase ^= 1u;
    }
    return true;
}

// The multiplying warps.
template <int MT>
__device__ __forceinline__ bool few_rows_multiply(const CUtensorMap &map_a, const CUtensorMap &map_b,
                                                  const S8Params &p, FewPlace &f, uint32_t full0,
                                                  uint32_t ring_b, uint32_t ring_a, int32_t *sums0, int warp, int lane)
{
    using Cfg = S8FewCfg<MT>;
    constexpr uint32_t S = Cfg::STAGES;
    constexpr int NB = 2 * MT;  // blocks of eight rows
    const int g = lane >> 2, t4 = lane & 3;
    const int half = warp & 1;
    // This CTA's k-blocks, and the warp's first of them.
    const int32_t first = f.rank * p.kb_each + min(f.rank, p.kb_more);
    const int32_t end = first + p.kb_each + (f.rank < p.kb_more);
    const int32_t begin = first + (warp >> 1);

    // The warp's loads run S blocks ahead of its MMAs.
    int32_t next_tile = f.cluster, next_k = begin;
    S8Tile pt = {};
    if (next_tile < f.tiles)
        pt = few_rows_tile<MT>(p, f, next_tile);
    uint32_t issued = 0;  // stages that hold or await a block
    auto issue = [&](uint32_t stage) {
        if (next_k >= end) {
            if (begin >= end)
                return;  // (no block of any tile is this warp's)
            next_k = begin;
            next_tile += f.clusters;
            if (next_tile < f.tiles)
                pt = few_rows_tile<MT>(p, f, next_tile);
        }
        if (next_tile >= f.tiles) {
            next_k = end;  // (comes back here; the tile only grows)
            return;
        }
        if (lane == 0) {
            const uint32_t fb = full0 + 8u * stage;
            ptx::mbar_arrive_expect_tx(fb, Cfg::B_BYTES + Cfg::A_BYTES);
            ptx::tma_load_3d(ring_b + stage * Cfg::B_BYTES, &map_b, fb, pt.n0 + 128 * half, next_k * Cfg::BK, pt.z);
            ptx::tma_load_3d(ring_a + stage * Cfg::A_BYTES, &map_a, fb, next_k * Cfg::BK, pt.m0, pt.z);
        }
        __syncwarp();
        next_k += Cfg::KWARPS;
        ++issued;
    };
#pragma unroll 1
    for (uint32_t s = 0; s < S; ++s)
        issue(s);
    few_rows_start<MT>(f);  // (while those are on their way)

    uint32_t stage = 0, phase = 0, set = 0, set_phase = 0;
    bool ok = true;
    for (int32_t tile = f.cluster; ok && tile < f.tiles; tile += f.clusters) {
        int32_t *const sums = sums0 + set * Cfg::SUMS + half * Cfg::HALF_SUMS;
        f.last = tile;
        f.last_set = int32_t(set);
        bool mine = false;  // the set is this tile's
        const int octets = (few_rows_tile<MT>(p, f, tile).rows + 7) / 8;
        float acc[NB][8][4];
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int j = 0; j < 8; ++j)
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    acc[n][j][d] = 0.f;
        auto take = [&]() {  // the set's last tile has left it
            if (!mine)
                ok = __all_sync(0xffffffffu, s8_wait<false>(f.sums_free0 + 8u * set, set_phase ^ 1u, f.flag, p, kStatusReduce));
            mine = true;
            return ok;
        };
        auto flush = [&]() {
            if (!take())
                return;
#pragma unroll
            for (int n = 0; n < NB; ++n) {
                if (n >= octets)
                    break;
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        atomicAdd(sums + few_rows_sum(n, g & 1, 2 * t4 + (d & 1), 2 * j + (d >> 1), g >> 1),
                                  __float2int_rn(acc[n][j][d]));
                        acc[n][j][d] = 0.f;
                    }
            }
        };
        int held = 0;
        for (int32_t kb = begin; kb < end; kb += Cfg::KWARPS) {
            ok = __all_sync(0xffffffffu, s8_wait<false>(full0 + 8u * stage, phase, f.flag, p, kStatusProducer));
            if (!ok)
                break;
            --issued;
            const uint32_t sb = ring_b + stage * Cfg::B_BYTES, sa = ring_a + stage * Cfg::A_BYTES;
#pragma unroll 1
            for (int kk = 0; kk < 2; ++kk) {
                uint32_t a[NB][2];
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    codes_to_f16(ptx::ld_shared_u32(sa + uint32_t((8 * n + g) * Cfg::BK + 16 * kk + 4 * t4)), a[n][0],
                                 a[n][1]);
                uint32_t r[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t k = uint32_t(16 * kk + 4 * t4 + i);
                    const uint4 u = ptx::ld_shared_v4(sb + k * 128u + ((uint32_t(g) ^ (k & 7u)) << 4));
                    r[i][0] = u.x;
                    r[i][1] = u.y;
                    r[i][2] = u.z;
                    r[i][3] = u.w;
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    auto columns = [&](auto half_word) {
                        constexpr int B = decltype(half_word)::value;
                        const uint32_t b[4] = {code_pair<B>(r[0][x], r[1][x]), code_pair<B + 1>(r[0][x], r[1][x]),
                                               code_pair<B>(r[2][x], r[3][x]), code_pair<B + 1>(r[2][x], r[3][x])};
                        ptx::mma_16816(acc[0][2 * x + B / 2], b, a[0][0], a[0][1]);
#pragma unroll
                        for (int n = 1; n < NB; ++n)
                            ptx::mma_16816_if(n < octets, acc[n][2 * x + B / 2], b, a[n][0], a[n][1]);
                    };
                    columns(ActTag<0>{});
                    columns(ActTag<2>{});
                }
            }
            __syncwarp();  // every lane has read the stage
            issue(stage);
            if (++stage == S) {
                stage = 0;
                phase ^= 1u;
            }
            if (++held == Cfg::FLUSH) {
                flush();
                held = 0;
                if (!ok)
                    break;
            }
        }
        if (ok && held)
            flush();
        // (A warp without a block in the tile waits for the set, too, before
        // it arrives: it could otherwise arrive twice in one phase.)
        if (!ok || !take())
            break;
        __syncwarp();
        if (lane == 0)
            ptx::mbar_arrive(f.sums_full0 + 8u * set);
        set ^= 1u;
        if (set == 0)
            set_phase ^= 1u;
    }
    // No TMA write into shared memory outlives the CTA.
    for (; issued > 0; --issued) {
        s8_wait<false>(full0 + 8u * stage, phase, f.flag, p, kStatusDrain, false);
        if (++stage == S) {
            stage = 0;
            phase ^= 1u;
        }
    }
    return ok;
}

template <int MT>
__global__ void __launch_bounds__(S8FewCfg<MT>::THREADS, 1)
    tsm_s8_few_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                      const S8Params p)
{
    using Cfg = S8FewCfg<MT>;
    constexpr int S = Cfg::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *const base_ptr = smem_raw + (base - raw);
    constexpr uint32_t A0 = Cfg::WARPS * S * Cfg::B_BYTES;
    constexpr uint32_t SUMS0 = A0 + Cfg::WARPS * S * Cfg::A_BYTES;
    constexpr uint32_t CTRL0 = SUMS0 + 2 * Cfg::SUMS * 4;
    static_assert(Cfg::WARPS * S * 8 <= 384, "control block");
    const uint32_t ctrl = base + CTRL0;
    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);
    const int lane = int(threadIdx.x & 31);

    FewPlace f;
    f.sums0 = base + SUMS0;
    f.terms0 = ctrl + Cfg::TERMS_OFF;
    f.sums_full0 = ctrl + 384u;
    f.sums_free0 = ctrl + 400u;
    f.ready0 = ctrl + 416u;
    f.taken0 = ctrl + 432u;
    f.flag = ctrl + 448u;
    f.gtab = ctrl + Cfg::GROUP_TABLE_OFF;
    f.grows = ctrl + Cfg::GROUP_ROWS_OFF;
    f.ranks = p.ranks;
    f.rank = int32_t(ptx::cluster_ctarank());
    f.cluster = int32_t(ptx::cluster_id());
    f.clusters = int32_t(ptx::n_clusters());
    f.last = -1;
    f.last_set = 0;

    // A multiplying warp's own barriers are all that its first loads need.
    if (warp < Cfg::WARPS && lane == 0) {
        for (int s = 0; s < S; ++s)
            ptx::mbar_init(ctrl + 8u * uint32_t(warp * S + s), 1);
        ptx::fence_mbar_init();
    }
    if (int(threadIdx.x) == 32 * Cfg::WARPS) {
        ptx::prefetch_tensormap(&map_a);
        ptx::prefetch_tensormap(&map_b);
        for (uint32_t i = 0; i < 2; ++i) {
            ptx::mbar_init(f.sums_full0 + 8u * i, Cfg::WARPS);
            ptx::mbar_init(f.sums_free0 + 8u * i, 1);
            ptx::mbar_init(f.ready0 + 8u * i, uint32_t(p.ranks));
            ptx::mbar_init(f.taken0 + 8u * i, uint32_t(p.ranks));
        }
        ptx::st_shared_u32(f.flag, 0u);
        ptx::fence_mbar_init();
    }
    __syncwarp();
    // (Relaxed, and before the first loads: a release would wait for those, 2.8
    // us.  The barriers' fence has published all that the others need.)
    if (p.ranks > 1)
        ptx::cluster_arrive_relaxed();
    chain_next();
    chain_wait();
    if (p.group_rows) {
        if (warp == 1)
            build_s8_groups<Cfg::ROWS>(p, f.gtab, f.grows);
        __syncthreads();
    }
    f.tiles = p.group_rows ? int32_t(ptx::ld_shared_u32(f.gtab + 4u * (p.batch - 1)))
                           : p.tiles_m * p.tiles_n * p.batch;
    bool ok = true;
    if (warp < Cfg::WARPS) {
        ptx::regs_inc<Cfg::MMA_REGS>();
        ok = few_rows_multiply<MT>(map_a, map_b, p, f, ctrl + uint32_t(warp * S) * 8u,
                                   base + uint32_t(warp * S) * Cfg::B_BYTES,
                                   base + A0 + uint32_t(warp * S) * Cfg::A_BYTES,
                                   reinterpret_cast<int32_t *>(base_ptr + SUMS0), warp, lane);
        ptx::regs_dec<Cfg::LAUNCH_REGS>();
        if (p.ranks > 1)
            ptx::cluster_wait();
    } else {
        ptx::regs_dec<Cfg::FINISH_REGS>();
        few_rows_start<MT>(f);
        if (p.ranks > 1)
            ptx::cluster_wait();  // the other CTAs' barriers exist
        ok = few_rows_finish<MT>(p, f);
        ptx::regs_inc<Cfg::LAUNCH_REGS>();
    }
    // The CTA's last tile has nothing to hide behind, and every warp takes part
    // in finishing it (four warps alone took 2.1 us for 16 rows, these 1.0).
    __syncwarp();
    ok = __syncthreads_and(ok);
    if (p.ranks > 1)
        ptx::cluster_sync();  // the cluster's sums are complete
    if (ok && f.last >= 0)
        few_rows_share<MT>(p, f, few_rows_tile<MT>(p, f, f.last), f.sums0 + uint32_t(f.last_set) * uint32_t(Cfg::SUMS * 4),
                           int(threadIdx.x), Cfg::THREADS);
    __syncwarp();
    if (p.ranks > 1) {  // no CTA leaves while another may still reach into it
        ptx::cluster_arrive_relaxed();
        ptx::cluster_wait();
    }
}

// ------------------------------------------------------------- counts alone

// Report counts outside [0, M], for a grouped launch whose sums are empty: the
// fill that does its work only clamps them.
__global__ void __launch_bounds__(kMaxGroupsPerLaunch)
    tsm_s8_counts_kernel(const int32_t *group_rows, int32_t groups, int32_t M, uint32_t *status)
{
    chain_next();
    chain_wait();
    const int32_t g = int32_t(threadIdx.x);
    const int32_t rows = g < groups ? __ldcg(group_rows + g) : 0;
    if (rows < 0 || rows > M)
        atomicOr(status, kStatusGroupRows);
}

// ------------------------------------------------------------- repacking

// One thread per 16 bytes of the packed rows (zeros past a row's end).
__global__ void __launch_bounds__(256)
    tsm_pack_s8_kernel(const int8_t *src, int64_t s_ld, int64_t s_stride, int8_t *dst, int64_t d_ld, int64_t d_stride,
                       int64_t rows, int64_t cols, int64_t batch)
{
    chain_next();
    chain_wait();
    const int64_t chunks = d_ld / 16;
    const int64_t total = batch * rows * chunks;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += int64_t(gridDim.x) * blockDim.x) {
        const int64_t row = i / chunks;
        const int64_t c = (i - row * chunks) * 16;
        const int64_t z = row / rows, r = row - z * rows;
        const uint8_t *s = reinterpret_cast<const uint8_t *>(src) + z * s_stride + r * s_ld + c;
        uint32_t w[4] = {0, 0, 0, 0};
        if (c + 20 <= cols) {
            // Five aligned words cover the 16 bytes: the first starts at most
            // three bytes early, so it is taken byte by byte.
            const int off = int(reinterpret_cast<uintptr_t>(s) & 3u);
            if (off == 0) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    w[k] = reinterpret_cast<const uint32_t *>(s)[k];
            } else {
                const uint32_t *a = reinterpret_cast<const uint32_t *>(s - off) + 1;
                uint32_t prev = 0;
                for (int b = off; b < 4; ++b)
                    prev |= uint32_t(s[b - off]) << (8 * b);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t next = a[k];
                    w[k] = __funnelshift_r(prev, next, 8 * off);
                    prev = next;
                }
            }
        } else {
            for (int k = 0; k < 16 && c + k < cols; ++k)
                w[k >> 2] |= uint32_t(s[k]) << (8 * (k & 3));
        }
        *reinterpret_cast<uint4 *>(dst + z * d_stride + r * d_ld + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <int MT>
cudaError_t set_few(S8Capacity *cap)
{
    cudaError_t e = cudaFuncSetAttribute(tsm_s8_few_kernel<MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         S8FewCfg<MT>::SMEM_BYTES);
    for (int i = 0; e == cudaSuccess && i < S8Capacity::KINDS; ++i) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(unsigned(i + 1), 1, 1);
        cfg.blockDim = dim3(S8FewCfg<MT>::THREADS, 1, 1);
        cfg.dynamicSmemBytes = S8FewCfg<MT>::SMEM_BYTES;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = unsigned(i + 1);
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&cap->clusters[i], tsm_s8_few_kernel<MT>, &cfg);
    }
    return e;
}

template <int MT>
cudaError_t launch_few(const CUtensorMap &map_a, const CUtensorMap &map_b, const S8Params &p, int grid,
                       cudaStream_t stream)
{
    return launch_chained(tsm_s8_few_kernel<MT>, dim3(unsigned(grid * p.ranks)), S8FewCfg<MT>::THREADS,
                          S8FewCfg<MT>::SMEM_BYTES, unsigned(p.ranks), stream, map_a, map_b, p);
}

}  // namespace

cudaError_t set_s8_attributes(S8Capacity *cap)
{
    cudaError_t e = set_s8_tiled<kActNone>();
    if (e == cudaSuccess)
        e = set_s8_tiled<kActRelu>();
    if (e == cudaSuccess)
        e = set_s8_tiled<kActLeakyRelu>();
    if (e == cudaSuccess)
        e = set_s8_tiled<kActGelu>();
    if (e == cudaSuccess)
        e = set_s8_tiled<kActGeluTanh>();
    if (e == cudaSuccess)
        e = set_s8_tiled<kActSilu>();
    if (e == cudaSuccess)
        e = set_few<1>(cap);
    if (e == cudaSuccess)
        e = set_few<2>(cap);
    return e;
}

cudaError_t launch_s8(const CUtensorMap &map_a, const CUtensorMap &map_b, const S8Params &p, S8Kind kind, int grid,
                      cudaStream_t stream)
{
    switch (kind) {
    case S8Kind::kFew16: return launch_few<1>(map_a, map_b, p, grid, stream);
    case S8Kind::kFew32: return launch_few<2>(map_a, map_b, p, grid, stream);
    default: break;
    }
    const bool pair = kind == S8Kind::kPair;
    switch (p.epi.act) {
    case kActRelu: return launch_s8_tiled<kActRelu>(map_a, map_b, p, pair, grid, stream);
    case kActLeakyRelu: return launch_s8_tiled<kActLeakyRelu>(map_a, map_b, p, pair, grid, stream);
    case kActGelu: return launch_s8_tiled<kActGelu>(map_a, map_b, p, pair, grid, stream);
    case kActGeluTanh: return launch_s8_tiled<kActGeluTanh>(map_a, map_b, p, pair, grid, stream);
    case kActSilu: return launch_s8_tiled<kActSilu>(map_a, map_b, p, pair, grid, stream);
    default: return launch_s8_tiled<kActNone>(map_a, map_b, p, pair, grid, stream);
    }
}

cudaError_t launch_s8_counts(const S8Params &p, cudaStream_t stream)
{
    return launch_chained(tsm_s8_counts_kernel, dim3(1), kMaxGroupsPerLaunch, 0, 0, stream, p.group_rows, p.batch, p.M,
                          p.status);
}

cudaError_t launch_pack_s8(const int8_t *src, int64_t s_ld, int64_t s_stride, int8_t *dst, int64_t d_ld,
                           int64_t d_stride, int64_t rows, int64_t cols, int64_t batch, int sms,
                           cudaStream_t stream)
{
    const int64_t blocks = (batch * rows * (d_ld / 16) + 255) / 256;
    return launch_chained(tsm_pack_s8_kernel, dim3(unsigned(min(blocks, int64_t(sms) * 32))), 256, 0, 0, stream, src, s_ld,
                          s_stride, dst, d_ld, d_stride, rows, cols, batch);
}

}  // namespace tsm
