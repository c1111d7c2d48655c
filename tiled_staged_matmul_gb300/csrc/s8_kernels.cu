// s8_kernels.cu -- products of 8-bit integers with a scale per row and per
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
#include "gemm_kernel.cuh"
#include "launch.cuh"
#include "ops_internal.h"
#include "s8_ptx.cuh"

namespace tsm {

namespace {

constexpr int kChunkBlocks = 8;  // k-blocks of 128 whose sums the f32 accumulator holds exactly

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

// ------------------------------------------------------------- tiled kernel
//
// One persistent CTA (or CTA pair) per SM (pair of SMs), warp-specialised:
//   warp 0       TMA producer: codes of A (128 rows x 128 k) and B (128 k x 128
//                columns) into the code ring
//   warp 1       MMA issuer (the pair's leader): A from TMEM, B from shared memory
//   warps 4-7    A's codes -> f16 -> TMEM, one row per lane (they never pass
//                through shared memory as f16)
//   warps 8-11   B's codes -> f16 -> the 128-byte swizzled layout of the MMA
//   warps 12-19  two per TMEM lane quarter, one per column half of the tile:
//                accumulator -> 32-bit sums, then the epilogue
// The bound is shared-memory bandwidth: a 256 x 256 x 128 block costs an SM
// 32 KB of codes in, 32 KB out to the converters, 32 KB of f16 B written and
// 32 KB read by the MMAs = 1024 cycles at 128 bytes, just the time its MMAs
// take; with A's f16 in shared memory too it would be 1.5 times that.  A's f16
// ring takes the TMEM columns a second accumulator would need, so the MMAs
// pause while a chunk of 1024 k is read out.  (Two accumulators of half the
// width would not: but the MMA runs at full rate only at its full width, 256
// columns for a pair.)
template <bool PAIR>
struct S8Cfg {
    static constexpr int ROWS = 128;
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int TILE_M = ROWS * CTAS;
    static constexpr int B_COLS = 128;          // columns of B staged by one CTA
    static constexpr int TILE_N = B_COLS * CTAS;  // the MMA's width
    static constexpr int HC = TILE_N / 2;       // columns of one epilogue half
    static constexpr int BK = 128;
    static constexpr int A_CODES = ROWS * BK;   // bytes
    static constexpr int B_CODES = B_COLS * BK;
    static constexpr int CODE_STAGE = A_CODES + B_CODES;
    static constexpr int F_BOX = 64 * BK * 2;   // 64 columns of f16
    static constexpr int F_STAGE = 2 * F_BOX;
    static constexpr int S1 = 3, S2 = 3;        // ring depths
    static constexpr int STAGING = 8 * 32 * 32 * 4;
    static constexpr int CTRL = 2048, GROUP_TABLE_OFF = 1024;
    static constexpr int SMEM_BYTES = 1024 + S1 * CODE_STAGE + S2 * F_STAGE + STAGING + CTRL;
    static_assert(SMEM_BYTES <= 232448, "227 KiB per block");
    static constexpr uint32_t A_COL = 256;      // TMEM: the accumulator, then the f16 A ring
    static_assert(A_COL + S2 * (BK / 2) <= 512 && TILE_N <= 256, "TMEM columns");
    static constexpr int PARTS = 2 * CTAS;      // (CTA, half) parts of a tile
    static constexpr int32_t SLOT_INTS = PARTS * ROWS * HC;
};

constexpr int kWarpA = 4, kWarpB = 8, kWarpDrain = 12, kS8Warps = 20;  // first warps of the roles
constexpr int kS8Threads = 32 * kS8Warps;
// Registers per thread by warpgroup (five of 128 threads): together exactly
// what the block was launched with (640 x 96).
constexpr int kS8RegsIssue = 48, kS8RegsConvert = 56, kS8RegsDrain = 160;
static_assert(128 * kS8RegsIssue + 2 * 128 * kS8RegsConvert + 2 * 128 * kS8RegsDrain <= kS8Threads * 96,
              "register split");

// B's shared-memory descriptor: MN-major, 64-column boxes of BK rows of 128 bytes.
template <bool PAIR>
__device__ __forceinline__ uint64_t desc_b_s8(uint32_t saddr)
{
    return desc_common() | (uint64_t(S8Cfg<PAIR>::F_BOX >> 4) << 16) | uint64_t((saddr & 0x3FFFFu) >> 4);
}

// The schedule in shared memory, read field by field: the registers are for
// the sums.  WARP: a whole warp reads it together, and the compiler is told
// that the values are the warp's (they then need no register per lane).
template <bool WARP>
struct SharedSchedule {
    uint32_t at;
    __device__ __forceinline__ int32_t field(int i) const
    {
        const int32_t v = int32_t(ptx::ld_shared_u32(at + 4u * i));
        return WARP ? __shfl_sync(0xffffffffu, v, 0) : v;
    }
    __device__ __forceinline__ void put(const S8Schedule &s) const
    {
        ptx::st_shared_u32(at, uint32_t(s.tiles));
        ptx::st_shared_u32(at + 4, uint32_t(s.shared));
        ptx::st_shared_u32(at + 8, uint32_t(s.kb));
        ptx::st_shared_u32(at + 12, uint32_t(s.workers));
        ptx::st_shared_u32(at + 16, uint32_t(s.cutters));
    }
    __device__ __forceinline__ int32_t tiles() const { return field(0); }
    __device__ __forceinline__ int32_t kb() const { return field(2); }
    __device__ __forceinline__ int32_t workers() const { return field(3); }
    __device__ __forceinline__ S8Schedule all() const
    {
        S8Schedule s;
        s.tiles = tiles();
        s.shared = field(1);
        s.kb = kb();
        s.workers = workers();
        s.cutters = field(4);
        return s;
    }
};

// One worker's pieces in order: its share of the cut tiles, then whole tiles.
template <bool WARP>
struct PieceWalk {
    int32_t cur, end, next;  // blocks of the cut tiles; next whole tile
    int32_t tile, kb0, kb1;
    __device__ __forceinline__ PieceWalk(const SharedSchedule<WARP> &shared, int32_t w)
    {
        const S8Schedule s = shared.all();
        const bool cuts = s.shared > 0 && w < s.cutters;
        cur = cuts ? s.piece_begin(w) : 0;
        end = cuts ? s.piece_begin(w + 1) : 0;
        next = s.shared + w;
        tile = kb0 = kb1 = 0;
    }
    __device__ __forceinline__ bool advance(const SharedSchedule<WARP> &s)
    {
        kb0 = 0;
        kb1 = s.kb();
        if (cur < end) {
            tile = cur / kb1;
            kb0 = cur - tile * kb1;
            kb1 = min(kb1, kb0 + (end - cur));
            cur += kb1 - kb0;
            return true;
        }
        tile = next;
        next += s.workers();
        return tile < s.tiles();
    }
};

// Where a tile lies.
struct S8Tile {
    int32_t m0, n0, z, rows;
};

__device__ __forceinline__ S8Tile tile_at(int32_t t, const S8Params &p, uint32_t gtab, int tile_m, int tile_n)
{
    S8Tile w;
    int32_t tiles_m = p.tiles_m;
    if (p.group_rows) {
        int32_t lo = 0, hi = p.batch - 1;
        while (lo < hi) {
            const int32_t mid = (lo + hi) >> 1;
            if (int32_t(ptx::ld_shared_u32(gtab + 4u * mid)) > t)
                hi = mid;
            else
                lo = mid + 1;
        }
        const int32_t first = lo ? int32_t(ptx::ld_shared_u32(gtab + 4u * (lo - 1))) : 0;
        tiles_m = (int32_t(ptx::ld_shared_u32(gtab + 4u * lo)) - first) / p.tiles_n;
        t -= first;
        w.z = lo;
        w.rows = min(max(p.group_rows[lo], 0), p.M);
    } else {
        const int32_t per = p.tiles_m * p.tiles_n;
        w.z = t / per;
        t -= w.z * per;
        w.rows = p.M;
    }
    const int32_t group = p.group_m * p.tiles_n;
    const int32_t g = t / group;
    const int32_t first_m = g * p.group_m;
    const int32_t in_group = min(tiles_m - first_m, p.group_m);
    const int32_t r = t - g * group;
    w.m0 = (first_m + r % in_group) * tile_m;
    w.n0 = r / in_group * tile_n;
    return w;
}

// Count one arrival on `word` (a whole warp calls it): true for the last of
// `total`.  The word holds the launch's tag and the count; under another tag
// (whatever the workspace's last user left there) the count is none.  The
// first exchange expects everyone else to have arrived, so that the last one,
// whom the result waits for, is done after one trip to L2.  Any other failed
// exchange means that another of the at most `total` contributors has arrived,
// so the loop ends.  The loop is the warp's, not one lane's, so that the
// compiler need not plan for a warp that has come apart.
__device__ __forceinline__ bool arrive_last(unsigned long long *word, unsigned long long tag, uint32_t total, int lane)
{
    unsigned long long old = (tag << 16) | (total - 1u);
    for (;;) {
        const uint32_t seen = (old >> 16) == tag ? uint32_t(old & 0xffffu) : 0u;
        unsigned long long prev = 0;
        if (lane == 0)
            prev = atomicCAS(word, old, (tag << 16) | (seen + 1u));
        prev = __shfl_sync(0xffffffffu, prev, 0);
        if (prev == old)
            return seen + 1u == total;
        old = prev;
    }
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

// Add a chunk's f32 sums (HC columns of a TMEM lane) to the lane's integers.
// 1.5 * 2^23 + f has f + kMagicBits as its bits while |f| < 2^22, so an
// addition and an integer addition do what a conversion does at an eighth of
// their rate (8192^3: 744 -> 7xx us).  A sum can reach 2^24, though it takes
// codes near the limits with one sign to do so: where one of a warp's passes
// 2^22, the warp converts those eight columns.  Eight columns are on their way
// while eight are added.
constexpr uint32_t kMagicBits = 0x4b400000u;  // of 1.5 * 2^23

template <int HC>
__device__ __forceinline__ void add_chunk(uint32_t acc, int32_t (&sum)[HC])
{
    const float magic = __uint_as_float(kMagicBits);
    uint32_t r[2][8];
    ptx::tmem_ld_32x32b_x8(acc, r[0]);
#pragma unroll
    for (int c = 0; c < HC / 8; ++c) {
        ptx::tmem_wait_ld(r[c & 1]);
        if (c + 1 < HC / 8)
            ptx::tmem_ld_32x32b_x8(acc + 8u * (c + 1), r[(c + 1) & 1]);
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = __uint_as_float(r[c & 1][j]);
        const float top = ptx::max_abs3(ptx::max_abs3(ptx::max_abs3(f[0], f[1], f[2]), f[3], f[4]), f[5],
                                        ptx::max_abs3(f[6], f[7], 0.f));
        if (__any_sync(0xffffffffu, top >= 4194304.f)) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                sum[8 * c + j] += __float2int_rn(f[j]) + int32_t(kMagicBits);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                sum[8 * c + j] += __float_as_int(f[j] + magic);
        }
    }
}

// Arrive on a barrier of the pair's leader.  Released to the CTA only: what the
// arrival stands for is complete in this SM before it is sent -- f16 in its own
// shared memory (the proxy fence) or TMEM (the store wait), or TMEM read out
// (the load wait) -- and is next touched by this SM's own tensor core.
// Released to the cluster, every arrival would first wait for the warp's other
// stores, global ones included: measured 1.34 times the whole kernel's time at
// 8192^3 (1028 against 770 us).
template <bool PAIR>
__device__ __forceinline__ void arrive_leader(uint32_t bar)
{
    if constexpr (PAIR)
        ptx::mbar_arrive_remote(bar);
    else
        ptx::mbar_arrive(bar);
}

// Column scales (times alpha) and biases of four columns.
__device__ __forceinline__ void column_terms(const S8Params &p, int32_t z, int32_t col, float (&sb)[4],
                                             float (&bias)[4])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const bool in = col + k < p.N;
        sb[k] = p.epi.alpha;
        if (p.scale_b && in)
            sb[k] *= __ldg(p.scale_b + z * p.sb_stride + col + k);
        bias[k] = p.epi.bias && in ? __ldg(p.epi.bias + z * p.epi.bias_stride + col + k) : 0.f;
    }
}

// Four values of a row (scaled by the row) through the epilogue into C.
template <int ACT>
__device__ __forceinline__ void put4_as(const S8Params &p, int64_t at, int32_t col, float (&o)[4],
                                        const float (&sb)[4], const float (&bias)[4])
{
#pragma unroll
    for (int k = 0; k < 4; ++k)
        o[k] = epi_act(fmaf(sb[k], o[k], bias[k]), ACT, p.epi.slope);
    if (p.vec_c && col + 3 < p.N) {
        if (p.epi.out_type == kOutF32)
            *reinterpret_cast<float4 *>(static_cast<float *>(p.C) + at) = make_float4(o[0], o[1], o[2], o[3]);
        else
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.C) + at) =
                make_uint2(epi_out16(o[0], p.epi.out_type) | (epi_out16(o[1], p.epi.out_type) << 16),
                           epi_out16(o[2], p.epi.out_type) | (epi_out16(o[3], p.epi.out_type) << 16));
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (col + k < p.N)
            epi_store(p.C, at + k, o[k], p.epi.out_type);
}
// A staged box (32 rows of 32 f32 values, 16-byte chunks swizzled by the row)
// through the epilogue into C: eight lanes take a row's chunks, four rows at a
// time.
__device__ __forceinline__ void store_box(const S8Params &p, const S8Tile &t, uint32_t buf, int32_t row0, int32_t col0,
                                          int lane)
{
    const int32_t col = col0 + 4 * (lane & 7);
    if (col >= p.N)
        return;
    float sb[4], bias[4];
    column_terms(p, t.z, col, sb, bias);
    const int32_t rows = min(32, t.rows - row0);
    with_activation<kActRuntime>(p.epi.act, [&](auto act) {
#pragma unroll 1
        for (int r = lane >> 3; r < rows; r += 4) {
            const uint4 u = ptx::ld_shared_v4(buf + uint32_t(r) * 128u + (uint32_t((lane & 7) ^ (r & 7)) << 4));
            float o[4] = {__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
            put4_as<decltype(act)::value>(p, t.z * p.sC + int64_t(row0 + r) * p.ldc + col, col, o, sb, bias);
        }
    });
}

template <bool PAIR>
__global__ void __launch_bounds__(kS8Threads, 1)
    tsm_s8_tiled_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                        const S8Params p)
{
    using Cfg = S8Cfg<PAIR>;
    constexpr int S1 = Cfg::S1, S2 = Cfg::S2;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *const base_ptr = smem_raw + (base - raw);
    const uint32_t codes0 = base;
    const uint32_t f16_0 = codes0 + S1 * Cfg::CODE_STAGE;
    const uint32_t staging = f16_0 + S2 * Cfg::F_STAGE;
    const uint32_t ctrl = staging + Cfg::STAGING;
    uint8_t *const ctrl_ptr = base_ptr + (ctrl - base);

    // Barriers.  `ready` and `tempty` are used in the pair's leader only.
    const uint32_t full0 = ctrl;               // [S1] codes landed
    const uint32_t empty0 = ctrl + 32u;        // [S1] codes read by the converters
    const uint32_t ready0 = ctrl + 64u;        // [S2] f16 written (both CTAs)
    const uint32_t free0 = ctrl + 96u;         // [S2] MMAs that read the f16 are done
    const uint32_t tfull = ctrl + 128u;        // accumulator complete
    const uint32_t tempty = ctrl + 136u;       // accumulator read out (the leader's: by both CTAs)
    const uint32_t done_bar = ctrl + 160u;     // all MMAs completed
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(ctrl_ptr + 176);
    const uint32_t flag = ctrl + 180u;         // this CTA gives up
    const SharedSchedule<false> sched{ctrl + 256u};
    const SharedSchedule<true> wsched{ctrl + 256u};
    const uint32_t last_flag = ctrl + 184u;    // [2] one per column half
    const uint32_t gtab = ctrl + Cfg::GROUP_TABLE_OFF;

    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);  // (uniform to the compiler)
    const int lane = int(threadIdx.x & 31);
    const uint32_t rank = PAIR ? ptx::cluster_ctarank() : 0u;
    const int32_t worker = int32_t(PAIR ? (blockIdx.x >> 1) : blockIdx.x);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S1; ++s) {
            ptx::mbar_init(full0 + 8u * s, 1);
            ptx::mbar_init(empty0 + 8u * s, 8);
        }
        for (int s = 0; s < S2; ++s) {
            ptx::mbar_init(ready0 + 8u * s, 8 * Cfg::CTAS);
            ptx::mbar_init(free0 + 8u * s, 1);
        }
        ptx::mbar_init(tfull, 1);
        ptx::mbar_init(tempty, 8 * Cfg::CTAS);
        ptx::mbar_init(done_bar, 1);
        ptx::st_shared_u32(flag, 0u);
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&map_a);
        ptx::prefetch_tensormap(&map_b);
    }
    __syncwarp();
    if constexpr (PAIR)
        ptx::cluster_sync();
    chain_next();
    if (warp == 1) {
        ptx::tmem_alloc<PAIR>(ptx::smem_addr(tmem_slot), 512);
        ptx::tmem_relinquish<PAIR>();
    }
    chain_wait();
    if (warp == 2 && p.group_rows) {
        build_group_table(p.group_rows, p.batch, p.M, Cfg::TILE_M, p.tiles_n,
                          reinterpret_cast<uint32_t *>(ctrl_ptr + Cfg::GROUP_TABLE_OFF), p.status);
        __syncwarp();
    }
    if (warp == 2 && lane == 0) {
        S8Schedule s;
        s.plan(p.group_rows ? int32_t(ptx::ld_shared_u32(gtab + 4u * (p.batch - 1))) : p.tiles_m * p.tiles_n * p.batch, p.kb, p.workers);
        sched.put(s);
    }
    ptx::tc_fence_before_sync();
    ptx::cta_sync();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;

    const uint32_t ready_lead0 = PAIR ? ptx::mapa_shared(ready0, 0) : ready0;
    const uint32_t tempty_lead = PAIR ? ptx::mapa_shared(tempty, 0) : tempty;
    const int32_t row_off = int32_t(rank) * Cfg::ROWS;

    if (warp < 4) {
        ptx::regs_dec<kS8RegsIssue>();
        if (warp == 0 && lane == 0) {
            // ---------------- TMA producer
            uint32_t stage = 0, phase = 0;
            uint32_t issued = 0;
            bool ok = true;
            for (PieceWalk<false> w(sched, worker); ok && w.advance(sched);) {
                const S8Tile t = tile_at(w.tile, p, gtab, Cfg::TILE_M, Cfg::TILE_N);
                const int32_t col = t.n0 + int32_t(rank) * 128;
                for (int32_t kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!s8_wait<PAIR>(empty0 + 8u * stage, phase ^ 1u, flag, p, kStatusProducer)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sa = codes0 + stage * Cfg::CODE_STAGE;
                    const uint32_t fb = full0 + 8u * stage;
                    ptx::mbar_arrive_expect_tx(fb, Cfg::CODE_STAGE);
                    ptx::tma_load_3d(sa, &map_a, fb, kb * Cfg::BK, t.m0 + row_off, t.z);
                    ptx::tma_load_3d(sa + Cfg::A_CODES, &map_b, fb, col, kb * Cfg::BK, t.z);
                    ++issued;
                    if (++stage == S1) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // No TMA write into shared memory outlives the CTA.
            // (The last S1 loads: the slots from `stage` on, oldest first.)
            for (int i = 0; i < S1; ++i) {
                if (issued + i >= uint32_t(S1))
                    s8_wait<PAIR>(full0 + 8u * stage, phase ^ 1u, flag, p, kStatusDrain, false);
                if (++stage == S1) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        } else if (warp == 1 && lane == 0 && rank == 0) {
            // ---------------- MMA issuer
            constexpr uint32_t idesc = mma_idesc<Cfg::TILE_N, PAIR>();
            constexpr uint16_t both = PAIR ? 3 : 1;
            uint32_t stage = 0, phase = 0, aphase = 0;
            bool ok = true;
            for (PieceWalk<false> w(sched, worker); ok && w.advance(sched);) {
                int c = 0;  // blocks in the accumulator
                for (int32_t kb = w.kb0; ok && kb < w.kb1; ++kb) {
                    if (!s8_wait<PAIR, PAIR>(ready0 + 8u * stage, phase, flag, p, kStatusMma)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after_sync();
                    const bool last = c == kChunkBlocks - 1 || kb == w.kb1 - 1;
                    const uint32_t a = tmem + Cfg::A_COL + stage * uint32_t(Cfg::BK / 2);
                    if (c == 0) {
                        if (!s8_wait<PAIR, PAIR>(tempty, aphase ^ 1u, flag, p, kStatusMma)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after_sync();
                    }
                    const uint32_t sb = f16_0 + stage * Cfg::F_STAGE;
#pragma unroll
                    for (int kk = 0; kk < Cfg::BK / 16; ++kk)
                        ptx::mma_f16_ts<PAIR>(tmem, a + 8u * kk, desc_b_s8<PAIR>(sb + 2048u * kk), idesc,
                                              (c > 0 || kk > 0) ? 1u : 0u);
                    if (last)
                        ptx::mma_commit<PAIR>(tfull, both);
                    ptx::mma_commit<PAIR>(free0 + 8u * stage, both);
                    if (++stage == S2) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    c = last ? 0 : c + 1;
                    if (last)
                        aphase ^= 1u;
                }
            }
            // Every MMA must finish before TMEM is freed.
            ptx::mma_commit<PAIR>(done_bar, 1);
            s8_wait<PAIR>(done_bar, 0, flag, p, kStatusDrain, false);
        }
        __syncwarp();
    } else if (warp < kWarpDrain) {
        // ---------------- converters
        ptx::regs_dec<kS8RegsConvert>();
        const bool is_a = warp < kWarpB;
        const int q = is_a ? warp - kWarpA : warp - kWarpB;
        uint32_t s1 = 0, p1 = 0, s2 = 0, p2 = 0;
        bool ok = true;
        for (PieceWalk<true> w(wsched, worker); ok && w.advance(wsched);) {
            for (int32_t kb = w.kb0; kb < w.kb1; ++kb) {
                ok = s8_wait<PAIR>(full0 + 8u * s1, p1, flag, p, kStatusProducer) &&
                     s8_wait<PAIR>(free0 + 8u * s2, p2 ^ 1u, flag, p, kStatusProducer);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                const uint32_t codes = codes0 + s1 * Cfg::CODE_STAGE;
                if (is_a) {
                    // Row 32q + lane: eight 16-byte chunks, swizzled by the row.
                    ptx::tc_fence_after_sync();
                    const uint32_t row = codes + uint32_t(32 * q + lane) * 128u;
                    const uint32_t to = tmem + (uint32_t(32 * q) << 16) + Cfg::A_COL + s2 * uint32_t(Cfg::BK / 2);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const uint4 u = ptx::ld_shared_v4(row + (uint32_t((2 * g) ^ (lane & 7)) << 4));
                        const uint4 v = ptx::ld_shared_v4(row + (uint32_t((2 * g + 1) ^ (lane & 7)) << 4));
                        uint32_t r[16];
                        codes_to_f16(u.x, r[0], r[1]);
                        codes_to_f16(u.y, r[2], r[3]);
                        codes_to_f16(u.z, r[4], r[5]);
                        codes_to_f16(u.w, r[6], r[7]);
                        codes_to_f16(v.x, r[8], r[9]);
                        codes_to_f16(v.y, r[10], r[11]);
                        codes_to_f16(v.z, r[12], r[13]);
                        codes_to_f16(v.w, r[14], r[15]);
                        ptx::tmem_st_32x32b_x16(to + 16u * g, r);
                    }
                    __syncwarp();
                    if (lane == 0)
                        ptx::mbar_arrive(empty0 + 8u * s1);
                    ptx::tmem_wait_st();
                    ptx::tc_fence_before_sync();
                } else {
                    // 128 rows (k) of 128 codes, swizzled by the row.  A warp
                    // takes eight rows of one 64-column half at a time: a lane
                    // 16 codes of a row, written as two 16-byte chunks of f16.
                    // Rows k and k ^ 5 share eight lanes: bit 2 keeps their
                    // loads, bit 0 their stores in different banks.
                    const int c = lane & 3, i = lane >> 2;
                    const uint32_t r0 = uint32_t((i >> 1) ^ ((i & 1) * 5));  // row of the eight
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int h = j & 1;
                        const uint32_t k = uint32_t(8 * (4 * q + (j >> 1))) + r0;
                        const uint4 u = ptx::ld_shared_v4(codes + uint32_t(Cfg::A_CODES) + k * 128u +
                                                          (uint32_t(4 * h + c) ^ r0) * 16u);
                        uint32_t r[8];
                        codes_to_f16(u.x, r[0], r[1]);
                        codes_to_f16(u.y, r[2], r[3]);
                        codes_to_f16(u.z, r[4], r[5]);
                        codes_to_f16(u.w, r[6], r[7]);
                        const uint32_t to = f16_0 + s2 * Cfg::F_STAGE + uint32_t(h * Cfg::F_BOX) + k * 128u;
                        const uint32_t first = (uint32_t(2 * c) ^ r0) << 4;
                        ptx::st_shared_v4(to + first, r[0], r[1], r[2], r[3]);
                        ptx::st_shared_v4(to + (first ^ 16u), r[4], r[5], r[6], r[7]);
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        ptx::mbar_arrive(empty0 + 8u * s1);
                }
                __syncwarp();
                if (lane == 0)
                    arrive_leader<PAIR>(ready_lead0 + 8u * s2);
                if (++s1 == S1) {
                    s1 = 0;
                    p1 ^= 1u;
                }
                if (++s2 == S2) {
                    s2 = 0;
                    p2 ^= 1u;
                }
            }
        }
    } else {
        // ---------------- accumulator -> integers -> C
        ptx::regs_inc<kS8RegsDrain>();
        const int e = warp - kWarpDrain;
        const int h = e >> 2;
        const int q = warp & 3;
        const uint32_t acc = tmem + (uint32_t(32 * q) << 16) + uint32_t(h * Cfg::HC);
        const uint32_t buf = staging + uint32_t(e) * 4096u;
        uint32_t aphase = 0;
        bool ok = true;
        for (PieceWalk<true> w(wsched, worker); ok && w.advance(wsched);) {
            // The row's sums.  A chunk adds integer + kMagicBits to each (see
            // add_chunk), so they start that much lower for every chunk.
            int32_t sum[Cfg::HC];
            const uint32_t chunks = uint32_t(w.kb1 - w.kb0 + kChunkBlocks - 1) / kChunkBlocks;
#pragma unroll
            for (int j = 0; j < Cfg::HC; ++j)
                sum[j] = int32_t(0u - chunks * kMagicBits);
            for (int32_t kb = w.kb0; kb < w.kb1; kb += kChunkBlocks) {
                ok = s8_wait<PAIR>(tfull, aphase, flag, p, kStatusEpilogue);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok)
                    break;
                ptx::tc_fence_after_sync();
                add_chunk<Cfg::HC>(acc, sum);
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    arrive_leader<PAIR>(tempty_lead);
                aphase ^= 1u;
            }
            // The four warps go on or give up together (they meet below).
            ok = __all_sync(0xffffffffu, ptx::named_bar_and(1 + h, 128, ok));
            if (!ok)
                break;
            // (Read again rather than kept through the loop above, where
            // registers are short.)
            const uint32_t rank_now = PAIR ? ptx::cluster_ctarank() : 0u;
            const int32_t tid = 32 * q + lane;
            const int32_t me = int32_t(PAIR ? ptx::cta_id() >> 1 : ptx::cta_id());
            S8Tile t = tile_at(w.tile, p, gtab, Cfg::TILE_M, Cfg::TILE_N);
            t.m0 = __shfl_sync(0xffffffffu, t.m0, 0);  // (uniform to the compiler)
            t.n0 = __shfl_sync(0xffffffffu, t.n0, 0);
            t.z = __shfl_sync(0xffffffffu, t.z, 0);
            t.rows = __shfl_sync(0xffffffffu, t.rows, 0);
            const int32_t row0 = t.m0 + int32_t(rank_now) * Cfg::ROWS + 32 * q;  // the warp's first row
            int32_t cut_first = 0, cut_last = -1;  // contributors of a cut tile
            if (w.kb1 - w.kb0 < wsched.kb()) {
                // A piece: its sums go to this worker's slot, and whoever
                // arrives last adds up the others'.  [4-column group][row].
                // A tile's first contributor holds its first block and uses
                // its second slot; the others start in the tile: their first.
                const S8Schedule cut = wsched.all();
                const int32_t first = cut.owner(w.tile * cut.kb);
                const int32_t last = cut.owner((w.tile + 1) * cut.kb - 1);
                const int32_t part = int32_t(rank_now) * 2 + h;
                const int32_t lane_at = part * (Cfg::ROWS * Cfg::HC) + 4 * tid;
                int32_t *const mine = p.partial + (2 * me + (me == first)) * Cfg::SLOT_INTS + lane_at;
                if (row0 < t.rows) {
#pragma unroll
                    for (int j = 0; j < Cfg::HC; j += 4)
                        __stcg(reinterpret_cast<int4 *>(mine + j * Cfg::ROWS),
                               make_int4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]));
                }
                __threadfence();
                ptx::named_bar_sync(1 + h, 128);
                if (q == 0)
                    ptx::st_shared_u32(last_flag + 4u * h, arrive_last(p.arrivals + w.tile * Cfg::PARTS + part, p.tag,
                                                                      uint32_t(last - first + 1), lane));
                ptx::named_bar_sync(1 + h, 128);
                const bool mine_to_sum = __any_sync(0xffffffffu, ptx::ld_shared_u32(last_flag + 4u * h) != 0);
                __threadfence();
                if (!mine_to_sum)
                    continue;
                cut_first = first;
                cut_last = last;
            }
            // Through the warp's staging box: lane = row in, lane = column group out.
            const float sa = p.scale_a && row0 + lane < t.rows ? __ldg(p.scale_a + t.z * p.sa_stride + row0 + lane) : 1.f;
            auto stage = [&](int j, int32_t a, int32_t b, int32_t c, int32_t d) {
                ptx::st_shared_v4(buf + uint32_t(lane) * 128u + (uint32_t((j >> 2) ^ (lane & 7)) << 4),
                                  __float_as_uint(float(a) * sa), __float_as_uint(float(b) * sa),
                                  __float_as_uint(float(c) * sa), __float_as_uint(float(d) * sa));
            };
            const int32_t boxes = row0 < t.rows ? min(Cfg::HC / 32, (p.N - t.n0 - h * Cfg::HC + 31) / 32) : 0;
            if (cut_first <= cut_last) {
                // All contributors' sums, this one's too, a box at a time.
                const int32_t *from = p.partial + (int32_t(rank_now) * 2 + h) * (Cfg::ROWS * Cfg::HC) + 4 * tid;
#pragma unroll 1
                for (int b = 0; b < boxes; ++b, from += 32 * Cfg::ROWS) {
                    int4 x[8] = {};
                    // Two contributors' loads in flight together.
#pragma unroll 2
                    for (int32_t v = cut_first; v <= cut_last; ++v) {
                        const int32_t *theirs = from + (2 * v + (v == cut_first)) * Cfg::SLOT_INTS;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int4 y = __ldcg(reinterpret_cast<const int4 *>(theirs + 4 * i * Cfg::ROWS));
                            x[i].x += y.x;
                            x[i].y += y.y;
                            x[i].z += y.z;
                            x[i].w += y.w;
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        stage(4 * i, x[i].x, x[i].y, x[i].z, x[i].w);
                    __syncwarp();
                    store_box(p, t, buf, row0, t.n0 + h * Cfg::HC + 32 * b, lane);
                    __syncwarp();
                }
                continue;
            }
#pragma unroll 1
            for (int b = 0; b < boxes; ++b) {
#pragma unroll
                for (int bb = 0; bb < Cfg::HC / 32; ++bb)
                    if (b == bb) {
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            stage(j, sum[32 * bb + j], sum[32 * bb + j + 1], sum[32 * bb + j + 2], sum[32 * bb + j + 3]);
                    }
                __syncwarp();
                store_box(p, t, buf, row0, t.n0 + h * Cfg::HC + 32 * b, lane);
                __syncwarp();
            }
        }
    }

    ptx::tc_fence_before_sync();
    ptx::cta_sync();
    if constexpr (PAIR)
        ptx::cluster_sync();
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc<PAIR>(ptx::ld_shared_u32(ctrl + 176u), 512);
    }
}

// ------------------------------------------------------------- few rows
//
// Up to 32 rows of A (a decode step): the product reads every code of B once
// and is bound by that.  A tile is 256 columns; its K is cut over the CTAs of a
// cluster (up to 8 of them, by a time model on the host).  In a CTA,
// independent warps in pairs take 32 k of the tile at a time, one warp for each
// 128 columns, so that a row of B is read 256 bytes at a time (reading 128
// bytes of it ran at 4.6 TB/s, 256 at 6.0, 512 no faster).  Each warp has a TMA
// ring of its own and never waits for another.
//
// Warp-wide f16 MMAs (16 rows x 8 columns x 16 k) run far below the tcgen05
// rate, but 16 or 32 rows need no more: one SM's share of the memory rate is 23
// codes a cycle, 16 x 23 multiply-adds.  B's codes go from shared memory to the
// MMA's operand layout in registers: lane 4g + t takes 16 columns (chunk g) of
// rows 4t ... 4t + 3, and a byte of two rows each makes the f16 pair that it
// has to hold for one column.  Which columns and which k a lane's registers
// stand for is free as long as A's lanes agree, so no transpose is needed: MMA
// j of 16 gets column 16 g + j, and k index 2t, 2t + 1, 2t + 8, 2t + 9 is row
// 4t, 4t + 1, 4t + 2, 4t + 3.
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
    static constexpr int CTRL = 6144, GROUP_TABLE_OFF = 1024, TERMS_OFF = 2048;
    static constexpr int SMEM_BYTES = 1024 + WARPS * STAGES * (B_BYTES + A_BYTES) + 2 * SUMS * 4 + CTRL;
    static_assert(SMEM_BYTES <= 232448 && SMEM_BYTES > 232448 / 2, "227 KiB per block, one block per SM");
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
// row, and chunks of the four columns 32 apart, column j's chunk at j ^ row --
// so that the lanes of an accumulator value (eight rows of four columns 32
// apart) add to different banks, and sixteen threads read sixteen neighbouring
// columns' chunks.
__device__ __forceinline__ constexpr int few_rows_sum(int octet, int d1, int row, int j, int t)
{
    return ((octet * 2 + d1) * 8 + row) * 64 + 4 * (j ^ row) + t;
}

// A CTA's addresses and place in the launch.
struct FewPlace {
    uint32_t sums0, terms0;                       // shared memory: [2][SUMS] ints; scales and biases
    uint32_t sums_full0, sums_free0, ready0, taken0;  // barriers, [2] each
    uint32_t flag, gtab;
    int32_t tiles, cluster, clusters, rank, ranks;
};

// The finishing warps: tile by tile, the cluster's sums of this CTA's share of
// the tile through the epilogue into C.
template <int MT>
__device__ __forceinline__ void few_rows_finish(const S8Params &p, const FewPlace &f, int lane)
{
    using Cfg = S8FewCfg<MT>;
    constexpr int FT = 32 * Cfg::FINISHERS;
    const int ft = int(threadIdx.x) - 32 * Cfg::WARPS;
    const uint32_t sb0 = f.terms0, bias0 = f.terms0 + 4u * Cfg::COLS, sa0 = f.terms0 + 8u * Cfg::COLS;
    uint32_t set = 0, phase = 0;
    for (int32_t tile = f.cluster; tile < f.tiles; tile += f.clusters) {
        const S8Tile t = tile_at(tile, p, f.gtab, Cfg::ROWS, Cfg::COLS);
        // The terms of the epilogue while the sums are on their way.
        for (int c = ft; c < Cfg::COLS; c += FT) {
            const int32_t col = t.n0 + c;
            float sb = p.epi.alpha, bias = 0.f;
            if (p.scale_b && col < p.N)
                sb *= __ldg(p.scale_b + t.z * p.sb_stride + col);
            if (p.epi.bias && col < p.N)
                bias = __ldg(p.epi.bias + t.z * p.epi.bias_stride + col);
            ptx::st_shared_u32(sb0 + 4u * c, __float_as_uint(sb));
            ptx::st_shared_u32(bias0 + 4u * c, __float_as_uint(bias));
        }
        if (ft < Cfg::ROWS)
            ptx::st_shared_u32(sa0 + 4u * ft, __float_as_uint(p.scale_a && ft < t.rows
                                                                  ? __ldg(p.scale_a + t.z * p.sa_stride + ft) : 1.f));
        const uint32_t sums = f.sums0 + set * uint32_t(Cfg::SUMS * 4);
        bool ok = s8_wait<false>(f.sums_full0 + 8u * set, phase, f.flag, p, kStatusEpilogue);
        ok = __all_sync(0xffffffffu, ptx::named_bar_and(1, FT, ok));
        if (!ok)
            return;
        if (f.ranks > 1) {
            // This CTA's sums are complete: so says one thread to every CTA.
            if (ft < f.ranks)
                ptx::mbar_arrive_cluster(ptx::mapa_shared(f.ready0 + 8u * set, uint32_t(ft)));
            ok = s8_wait<false, true>(f.ready0 + 8u * set, phase, f.flag, p, kStatusReduce);
            ok = __all_sync(0xffffffffu, ptx::named_bar_and(1, FT, ok));
            if (!ok)
                return;
        }
        // This CTA's share of the tile, in chunks of four columns 32 apart;
        // rows past the last are left out in eights.
        const int octets = (t.rows + 7) / 8, chunks = 2 * octets * 256;
        const int last = (f.rank + 1) * chunks / f.ranks;
        for (int i = f.rank * chunks / f.ranks + ft; i < last; i += FT) {
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
            const int64_t row_at = t.z * p.sC + row * p.ldc + t.n0;
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
        ptx::named_bar_sync(1, FT);  // the sums and the terms have been read here
        if (f.ranks > 1) {
            // ... and in every CTA of the cluster, before they are cleared.
            if (ft < f.ranks)
                ptx::mbar_arrive_cluster(ptx::mapa_shared(f.taken0 + 8u * set, uint32_t(ft)));
            ok = s8_wait<false, true>(f.taken0 + 8u * set, phase, f.flag, p, kStatusReduce);
            ok = __all_sync(0xffffffffu, ptx::named_bar_and(1, FT, ok));
            if (!ok)
                return;
        }
        for (int i = ft; i < Cfg::SUMS / 4; i += FT)
            ptx::st_shared_v4(sums + 16u * i, 0u, 0u, 0u, 0u);
        ptx::named_bar_sync(1, FT);
        if (ft == 0)
            ptx::mbar_arrive(f.sums_free0 + 8u * set);
        set ^= 1u;
        if (set == 0)
            phase ^= 1u;
    }
}

// The multiplying warps.
template <int MT>
__device__ __forceinline__ void few_rows_multiply(const CUtensorMap &map_a, const CUtensorMap &map_b,
                                                  const S8Params &p, const FewPlace &f, uint32_t full0,
                                                  uint32_t ring_b, uint32_t ring_a, int32_t *sums0, int warp, int lane)
{
    using Cfg = S8FewCfg<MT>;
    constexpr uint32_t S = Cfg::STAGES;
    const int g = lane >> 2, t4 = lane & 3;
    const int half = warp & 1;
    // This CTA's k-blocks, and the warp's first of them.
    const int32_t end = int32_t(int64_t(f.rank + 1) * p.kb / f.ranks);
    const int32_t begin = int32_t(int64_t(f.rank) * p.kb / f.ranks) + (warp >> 1);

    // The warp's loads run S blocks ahead of its MMAs.
    int32_t next_tile = f.cluster, next_k = begin;
    S8Tile pt = {};
    if (next_tile < f.tiles)
        pt = tile_at(next_tile, p, f.gtab, Cfg::ROWS, Cfg::COLS);
    uint32_t issued = 0;  // stages that hold or await a block
    auto issue = [&](uint32_t stage) {
        if (next_k >= end) {
            if (begin >= end)
                return;  // (no block of any tile is this warp's)
            next_k = begin;
            next_tile += f.clusters;
            if (next_tile < f.tiles)
                pt = tile_at(next_tile, p, f.gtab, Cfg::ROWS, Cfg::COLS);
        }
        if (next_tile >= f.tiles) {
            next_k = end;  // (comes back here; the tile only grows)
            return;
        }
        if (lane == 0) {
            const uint32_t fb = full0 + 8u * stage;
            ptx::mbar_arrive_expect_tx(fb, Cfg::B_BYTES + Cfg::A_BYTES);
            ptx::tma_load_3d(ring_b + stage * Cfg::B_BYTES, &map_b, fb, pt.n0 + 128 * half, next_k * Cfg::BK, pt.z);
            ptx::tma_load_3d(ring_a + stage * Cfg::A_BYTES, &map_a, fb, next_k * Cfg::BK, 0, pt.z);
        }
        __syncwarp();
        next_k += Cfg::KWARPS;
        ++issued;
    };
#pragma unroll 1
    for (uint32_t s = 0; s < S; ++s)
        issue(s);

    uint32_t stage = 0, phase = 0, set = 0, set_phase = 0;
    bool ok = true;
    for (int32_t tile = f.cluster; ok && tile < f.tiles; tile += f.clusters) {
        int32_t *const sums = sums0 + set * Cfg::SUMS + half * Cfg::HALF_SUMS;
        bool mine = false;  // the set is this tile's
        float acc[MT][16][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 16; ++j)
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    acc[m][j][d] = 0.f;
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
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int j = 0; j < 16; ++j)
#pragma unroll
                    for (int d = 0; d < 4; ++d) {
                        atomicAdd(sums + few_rows_sum(2 * m + (d >> 1), d & 1, g, j, t4), __float2int_rn(acc[m][j][d]));
                        acc[m][j][d] = 0.f;
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
                uint32_t a[MT][4];
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    codes_to_f16(ptx::ld_shared_u32(sa + uint32_t((16 * m + g) * Cfg::BK + 16 * kk + 4 * t4)),
                                 a[m][0], a[m][2]);
                    codes_to_f16(ptx::ld_shared_u32(sa + uint32_t((16 * m + g + 8) * Cfg::BK + 16 * kk + 4 * t4)),
                                 a[m][1], a[m][3]);
                }
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
                    auto column = [&](auto b) {
                        constexpr int B = decltype(b)::value;
                        const uint32_t b0 = code_pair<B>(r[0][x], r[1][x]);
                        const uint32_t b1 = code_pair<B>(r[2][x], r[3][x]);
#pragma unroll
                        for (int m = 0; m < MT; ++m)
                            ptx::mma_16816(acc[m][4 * x + B], a[m], b0, b1);
                    };
                    column(ActTag<0>{});
                    column(ActTag<1>{});
                    column(ActTag<2>{});
                    column(ActTag<3>{});
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
    f.ranks = p.ranks;
    f.rank = int32_t(ptx::cluster_ctarank());
    f.cluster = int32_t(blockIdx.x) / p.ranks;
    f.clusters = int32_t(gridDim.x) / p.ranks;

    if (threadIdx.x == 0) {
        ptx::prefetch_tensormap(&map_a);
        ptx::prefetch_tensormap(&map_b);
        for (int i = 0; i < Cfg::WARPS * S; ++i)
            ptx::mbar_init(ctrl + 8u * i, 1);
        for (uint32_t i = 0; i < 2; ++i) {
            ptx::mbar_init(f.sums_full0 + 8u * i, Cfg::WARPS);
            ptx::mbar_init(f.sums_free0 + 8u * i, 1);
            ptx::mbar_init(f.ready0 + 8u * i, uint32_t(p.ranks));
            ptx::mbar_init(f.taken0 + 8u * i, uint32_t(p.ranks));
        }
        ptx::st_shared_u32(f.flag, 0u);
        ptx::fence_mbar_init();
    }
    for (int i = int(threadIdx.x); i < 2 * Cfg::SUMS / 4; i += Cfg::THREADS)
        ptx::st_shared_v4(f.sums0 + 16u * i, 0u, 0u, 0u, 0u);
    chain_next();
    chain_wait();
    if (warp == 1 && p.group_rows) {
        build_group_table(p.group_rows, p.batch, p.M, Cfg::ROWS, p.tiles_n,
                          reinterpret_cast<uint32_t *>(base_ptr + CTRL0 + Cfg::GROUP_TABLE_OFF), p.status);
    }
    __syncthreads();
    if (p.ranks > 1)
        ptx::cluster_sync();  // the other CTAs' barriers exist
    f.tiles = p.group_rows ? int32_t(ptx::ld_shared_u32(f.gtab + 4u * (p.batch - 1))) : p.tiles_n * p.batch;
    if (warp < Cfg::WARPS) {
        ptx::regs_inc<Cfg::MMA_REGS>();
        few_rows_multiply<MT>(map_a, map_b, p, f, ctrl + uint32_t(warp * S) * 8u,
                              base + uint32_t(warp * S) * Cfg::B_BYTES, base + A0 + uint32_t(warp * S) * Cfg::A_BYTES,
                              reinterpret_cast<int32_t *>(base_ptr + SUMS0), warp, lane);
    } else {
        ptx::regs_dec<Cfg::FINISH_REGS>();
        few_rows_finish<MT>(p, f, lane);
    }
    __syncwarp();
    if (p.ranks > 1)
        ptx::cluster_sync();  // no CTA leaves while another may still reach into it
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
                    w[k] = __ldg(reinterpret_cast<const uint32_t *>(s) + k);
            } else {
                const uint32_t *a = reinterpret_cast<const uint32_t *>(s - off) + 1;
                uint32_t prev = 0;
                for (int b = off; b < 4; ++b)
                    prev |= uint32_t(__ldg(s - off + b)) << (8 * b);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t next = __ldg(a + k);
                    w[k] = __funnelshift_r(prev, next, 8 * off);
                    prev = next;
                }
            }
        } else {
            for (int k = 0; k < 16 && c + k < cols; ++k)
                w[k >> 2] |= uint32_t(__ldg(s + k)) << (8 * (k & 3));
        }
        *reinterpret_cast<uint4 *>(dst + z * d_stride + r * d_ld + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

template <bool PAIR>
cudaError_t set_tiled()
{
    return cudaFuncSetAttribute(tsm_s8_tiled_kernel<PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                S8Cfg<PAIR>::SMEM_BYTES);
}

template <bool PAIR>
cudaError_t launch_tiled(const CUtensorMap &map_a, const CUtensorMap &map_b, const S8Params &p, int grid,
                         cudaStream_t stream)
{
    return launch_chained(tsm_s8_tiled_kernel<PAIR>, dim3(unsigned(grid)), kS8Threads, S8Cfg<PAIR>::SMEM_BYTES,
                          PAIR ? 2u : 0u, stream, map_a, map_b, p);
}

template <bool PAIR>
S8Shape shape_of()
{
    using Cfg = S8Cfg<PAIR>;
    return S8Shape{Cfg::TILE_M, Cfg::TILE_N, Cfg::BK, int64_t(Cfg::SLOT_INTS) * 4, Cfg::PARTS};
}

}  // namespace

S8Shape s8_shape(S8Kind kind)
{
    switch (kind) {
    case S8Kind::kFew16: return S8Shape{16, 256, 32, 0, 0};
    case S8Kind::kFew32: return S8Shape{32, 256, 32, 0, 0};
    case S8Kind::kOne: return shape_of<false>();
    default: return shape_of<true>();
    }
}

namespace {

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
    cudaError_t e = set_tiled<true>();
    if (e == cudaSuccess)
        e = set_tiled<false>();
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
    case S8Kind::kOne: return launch_tiled<false>(map_a, map_b, p, grid, stream);
    default: return launch_tiled<true>(map_a, map_b, p, 2 * grid, stream);
    }
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
