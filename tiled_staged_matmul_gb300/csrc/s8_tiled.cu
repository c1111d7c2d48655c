// s8_tiled.cu -- the tiled kernels of the 8-bit products (s8_common.cuh says
// what they compute and why in f16), compiled once per activation
// (-DTSM_S8_ACT, gemm_internal.h's kAct* values).
#include "s8_common.cuh"

#ifndef TSM_S8_ACT
#error "compile with -DTSM_S8_ACT=<activation>"
#endif

namespace tsm {

namespace {

constexpr int kAct = TSM_S8_ACT;
constexpr int kChunkBlocks = 8;  // k-blocks of 128 whose sums the f32 accumulator holds exactly

// ------------------------------------------------------------- tiled kernel
//
// One persistent CTA (or CTA pair) per SM (pair of SMs), warp-specialised:
//   warp 0       TMA producer: codes of A (128 rows x 128 k) and B (128 k x 128
//                columns) into the code ring
//   warp 1       MMA issuer (the pair's leader): A from TMEM, B from shared memory
//   warps 4-7    A's codes -> f16 -> TMEM, one row per lane (they never pass
//                through shared memory as f16)
//   warps 8-11   B's codes -> f16 -> the 128-byte swizzled layout of the MMA
//   warps 12-27  four per TMEM lane quarter, one per quarter of the tile's
//                columns: accumulator -> 32-bit sums, then the epilogue (with
//                two per lane quarter, half the columns each, a chunk took 1.05
//                us to add up and 8192^3 665 us, not 647)
// Measured: 8192^3 651 us (1.69 PFLOP/s, 0.89 of the f16 rate measured with
// cuBLAS), 4096 x 14336 x 4096 305 us (0.83), 97 x 14333 x 4095 with one CTA a
// tile 28 us.
//
// The bound is shared-memory bandwidth: a 256 x 256 x 128 block costs an SM
// 32 KB of codes in, 32 KB out to the converters, 32 KB of f16 B written and
// 32 KB read by the MMAs = 1024 cycles at 128 bytes, just the time its MMAs
// take; with A's f16 in shared memory too it would be 1.5 times that.  A's f16
// ring takes the TMEM columns a second accumulator would need, so the MMAs
// pause while a chunk of 1024 k is read out.  (Two accumulators of half the
// width would not: but the MMA runs at full rate only at its full width, 256
// columns for a pair.  One CTA's 128 x 128 tiles run at half of it.)
constexpr int kWarpA = 4, kWarpB = 8, kWarpDrain = 12;  // first warps of the roles
constexpr int kDrainWarps = 16, kS8Warps = kWarpDrain + kDrainWarps;
constexpr int kS8Threads = 32 * kS8Warps;
constexpr int kBarGroup = 1, kBarSetup = 5;  // named barriers: four epilogue groups' (1 ... 4), the setup's
// Registers per thread by warpgroup (seven of 128 threads): together exactly
// what the block was launched with (896 x 72).
constexpr int kS8RegsIssue = 40, kS8RegsConvert = 56, kS8RegsDrain = 88;
static_assert(128 * kS8RegsIssue + 2 * 128 * kS8RegsConvert + 32 * kDrainWarps * kS8RegsDrain <= kS8Threads * 72,
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

// Add a chunk's f32 sums (HC columns of a TMEM lane) to the lane's integers.
// 1.5 * 2^23 + f has f + kMagicBits as its bits while |f| < 2^22, so an
// addition and an integer addition do what a conversion does at an eighth of
// their rate (8192^3: 672 us with conversions, 651 so; 4096 x 14336 x 4096: 317
// and 305).  A sum can reach 2^24, though it takes codes near the limits with one
// sign to do so: where one of a warp's passes 2^22, the warp converts those eight
// columns.
constexpr uint32_t kMagicBits = 0x4b400000u;  // of 1.5 * 2^23

// Returns no less than the largest magnitude added.
template <int HC>
__device__ __forceinline__ float add_chunk(uint32_t acc, int32_t (&sum)[HC])
{
    float largest = 0.f;
    const float magic = __uint_as_float(kMagicBits);
#pragma unroll
    for (int c = 0; c < HC / 8; ++c) {
        uint32_t r[8];
        ptx::tmem_ld_32x32b_x8(acc + 8u * c, r);
        ptx::tmem_wait_ld(r);
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = __uint_as_float(r[j]);
        const float top = ptx::max_abs3(ptx::max_abs3(ptx::max_abs3(f[0], f[1], f[2]), f[3], f[4]), f[5],
                                        ptx::max_abs3(f[6], f[7], 0.f));
        largest = fmaxf(largest, top);
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
    return largest;
}

// Two values as the 16-bit output type stores them, in one conversion.
__device__ __forceinline__ uint32_t out16_pair(float a, float b, int32_t out_type)
{
    if (out_type == kOutBF16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&x);
    }
    const __half2 x = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&x);
}

// The epilogue of a box: 32 rows (a lane each) of 32 columns' sums.  Scaled,
// biased and activated in registers, where a lane's columns are independent
// work (done a row at a time after the exchange, where one value waited for
// another, 4096 x 14336 x 4096 took 1.12 times as long), then through the
// warp's staging space (32 bytes a row, 16-byte chunks swizzled by the row) so
// that the stores cover whole sectors.
__device__ __forceinline__ void finish_box(const S8Params &p, const S8Tile &t, const int32_t (&s32)[32], bool small, float sa,
                                           uint32_t sb_at, uint32_t bias_at, uint32_t buf, int32_t row0, int32_t col0,
                                           int lane)
{
    // Four columns' values.
    auto four = [&](int j, float (&v)[4]) {
        const uint4 s = ptx::ld_shared_v4(sb_at + 4u * j), b = ptx::ld_shared_v4(bias_at + 4u * j);
        const uint32_t sw[4] = {s.x, s.y, s.z, s.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // (Sums below 2^22 become f32 by add_chunk's way, in reverse.)
            const float s1 = small ? __int_as_float(s32[j + i] + int32_t(kMagicBits)) - __uint_as_float(kMagicBits)
                                   : float(s32[j + i]);
            v[i] = epi_act(fmaf(__uint_as_float(sw[i]), s1 * sa, __uint_as_float(bw[i])), kAct, p.epi.slope);
        }
    };
    const int32_t rows = t.rows - row0;
    const uint32_t mine = buf + uint32_t(lane) * 32u, swizzle = uint32_t(lane >> 2) & 1u;
    const bool f32 = p.epi.out_type == kOutF32;
    const int elem = f32 ? 4 : 2;
    const int per_row = 32 / elem;  // columns staged at a time: 8 f32 or 16 16-bit ones
#pragma unroll
    for (int part = 0; part < 4; ++part) {
        if (part >= 2 && !f32)
            break;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint32_t w[4];
            float v[4];
            if (f32) {
                four(8 * part + 4 * c, v);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    w[i] = __float_as_uint(v[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    four((16 * part + 8 * c + 2 * i) & 31, v);
                    w[i] = out16_pair(v[0], v[1], p.epi.out_type);
                    w[i + 1] = out16_pair(v[2], v[3], p.epi.out_type);
                }
            }
            ptx::st_shared_v4(mine + ((uint32_t(c) ^ swizzle) << 4), w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        const int32_t col = col0 + part * per_row;
        char *const c_at = static_cast<char *>(p.C) + (t.z * p.sC + int64_t(row0) * p.ldc + col) * elem;
        if (p.vec_c && col + per_row <= p.N) {
            // Two lanes a row, sixteen rows at a time.
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = 16 * i + (lane >> 1), ch = lane & 1;
                const uint4 u = ptx::ld_shared_v4(buf + uint32_t(r) * 32u + ((uint32_t(ch) ^ (uint32_t(r >> 2) & 1u)) << 4));
                if (r < rows)
                    *reinterpret_cast<uint4 *>(c_at + r * p.ldc * elem + 16 * ch) = u;
            }
        } else {
            // Any pitch, and the last columns: an element a lane (4096 x 4095 x
            // 2048 bf16: four at a time 90 us, one 94).
            const int shift = f32 ? 3 : 4;
#pragma unroll 4
            for (int i = lane; i < 32 * per_row; i += 32) {
                const int r = i >> shift, j = i & (per_row - 1);
                const uint32_t at = buf + uint32_t(r) * 32u + ((uint32_t(j * elem >> 4) ^ (uint32_t(r >> 2) & 1u)) << 4) +
                                    uint32_t(j * elem & 15);
                if (r < rows && col + j < p.N) {
                    if (f32)
                        *reinterpret_cast<uint32_t *>(c_at + (r * p.ldc + j) * 4) = ptx::ld_shared_u32(at);
                    else
                        *reinterpret_cast<uint16_t *>(c_at + (r * p.ldc + j) * 2) = ptx::ld_shared_u16(at);
                }
            }
        }
    }
    __syncwarp();
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
    const uint32_t last_flag = ctrl + 184u;    // [4] one per epilogue group
    const uint32_t gtab = ctrl + Cfg::GROUP_TABLE_OFF, grows = ctrl + Cfg::GROUP_ROWS_OFF;
    const uint32_t tiles0 = ctrl + 512u;  // [16] an epilogue warp's tile
    const uint32_t terms0 = ctrl + Cfg::TERMS_OFF;  // [2][group][columns' scales, biases; rows' scales]

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
        ptx::mbar_init(tempty, kDrainWarps * Cfg::CTAS);
        ptx::mbar_init(done_bar, 1);
        ptx::st_shared_u32(flag, 0u);
        if (!p.group_rows)
            sched.put(p.sched);
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&map_a);
        ptx::prefetch_tensormap(&map_b);
    }
    __syncwarp();
    ptx::cta_sync();  // the barriers are there
    if constexpr (PAIR)
        ptx::cluster_arrive_relaxed();
    chain_next();
    // Unless the tiles are counted on the device, the producer has all it needs
    // by now, and its first loads do not wait for the rest (0.6 us, 1.5 in a
    // pair).
    const bool early = warp == 0 && !p.group_rows;
    if (!early) {
        if constexpr (PAIR)
            ptx::cluster_wait();  // the peer is there, and its barriers
        if (warp == 1) {
            ptx::tmem_alloc<PAIR>(ptx::smem_addr(tmem_slot), 512);
            ptx::tmem_relinquish<PAIR>();
        }
    }
    chain_wait();
    if (!early) {
        if (warp == 2 && p.group_rows) {
            build_s8_groups<Cfg::TILE_M>(p, gtab, grows);
            if (lane == 0) {
                S8Schedule s;
                s.plan(int32_t(ptx::ld_shared_u32(gtab + 4u * (p.batch - 1))), p.kb, p.workers);
                sched.put(s);
            }
        }
        // (All warps that came here: all, or all but the first.)
        ptx::tc_fence_before_sync();
        ptx::named_bar_sync(kBarSetup, p.group_rows ? kS8Threads : kS8Threads - 32);
        ptx::tc_fence_after_sync();
    }
    const uint32_t tmem = early ? 0u : *tmem_slot;

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
                const S8Tile t = tile_at(w.tile, p, gtab, grows, Cfg::TILE_M, Cfg::TILE_N);
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
        if constexpr (PAIR) {
            if (early)
                ptx::cluster_wait();
        }
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
        const uint32_t buf = staging + uint32_t(e) * 1024u;
        uint32_t aphase = 0, turn = 0;
        bool ok = true;
        for (PieceWalk<true> w(wsched, worker); ok && w.advance(wsched);) {
            // The row's sums.  A chunk adds integer + kMagicBits to each (see
            // add_chunk), so they start that much lower for every chunk.
            int32_t sum[Cfg::HC];
            float bound = 0.f;  // no sum is larger
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
                bound += add_chunk<Cfg::HC>(acc, sum);
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    arrive_leader<PAIR>(tempty_lead);
                aphase ^= 1u;
                if (kb != w.kb0)
                    continue;
                // With the first chunk out of the way (it was complete long
                // before the last tile's epilogue was): where the tile is, for
                // later, and its columns' scales and biases and rows' scales on
                // their way.  Two sets in turn, since the group's other warps
                // may still be at the last tile's; they meet below.
                const S8Tile t = tile_at(w.tile, p, gtab, grows, Cfg::TILE_M, Cfg::TILE_N);
                const int32_t i = 32 * q + lane, col = t.n0 + h * Cfg::HC + i;
                const int32_t row = t.m0 + int32_t(PAIR ? ptx::cluster_ctarank() : 0u) * Cfg::ROWS + i;
                const uint32_t at = terms0 + turn * Cfg::TERMS + uint32_t(h) * Cfg::GROUP_TERMS + 4u * i;
                if (i < Cfg::HC)
                    ptx::fetch_f32(at, p.scale_b && col < p.N ? p.scale_b + t.z * p.sb_stride + col : nullptr, 1.f);
                if (i < Cfg::HC)
                    ptx::fetch_f32(at + 4u * Cfg::HC,
                               p.epi.bias && col < p.N ? p.epi.bias + t.z * p.epi.bias_stride + col : nullptr, 0.f);
                ptx::fetch_f32(at + 8u * Cfg::HC, p.scale_a && row < t.rows ? p.scale_a + t.z * p.sa_stride + row : nullptr, 1.f);
                if (lane == 0)
                    ptx::st_shared_v4(tiles0 + 16u * uint32_t(e), uint32_t(t.m0), uint32_t(t.n0), uint32_t(t.z),
                                      uint32_t(t.rows));
                __syncwarp();
            }
            // The four warps go on or give up together (they meet below).
            ptx::fetch_wait();
            ok = __all_sync(0xffffffffu, ptx::named_bar_and(kBarGroup + h, 128, ok));
            if (!ok)
                break;
            // (Read again rather than kept through the loop above, where
            // registers are short.)
            const uint32_t rank_now = PAIR ? ptx::cluster_ctarank() : 0u;
            const int32_t tid = 32 * q + lane;
            const int32_t me = int32_t(PAIR ? ptx::cta_id() >> 1 : ptx::cta_id());
            const uint4 place = ptx::ld_shared_v4(tiles0 + 16u * uint32_t(e));
            S8Tile t;
            t.m0 = __shfl_sync(0xffffffffu, int32_t(place.x), 0);  // (uniform to the compiler)
            t.n0 = __shfl_sync(0xffffffffu, int32_t(place.y), 0);
            t.z = __shfl_sync(0xffffffffu, int32_t(place.z), 0);
            t.rows = __shfl_sync(0xffffffffu, int32_t(place.w), 0);
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
                const int32_t part = int32_t(rank_now) * Cfg::GROUPS + h;
                const int32_t lane_at = part * (Cfg::ROWS * Cfg::HC) + 4 * tid;
                int32_t *const mine = p.partial + (2 * me + (me == first)) * Cfg::SLOT_INTS + lane_at;
                if (row0 < t.rows) {
#pragma unroll
                    for (int j = 0; j < Cfg::HC; j += 4)
                        __stcg(reinterpret_cast<int4 *>(mine + j * Cfg::ROWS),
                               make_int4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]));
                }
                __threadfence();
                ptx::named_bar_sync(kBarGroup + h, 128);
                if (q == 0)
                    ptx::st_shared_u32(last_flag + 4u * h, arrive_last(p.arrivals + w.tile * Cfg::PARTS + part, p.tag,
                                                                      uint32_t(last - first + 1), lane));
                ptx::named_bar_sync(kBarGroup + h, 128);
                const bool mine_to_sum = __any_sync(0xffffffffu, ptx::ld_shared_u32(last_flag + 4u * h) != 0);
                __threadfence();
                if (!mine_to_sum) {
                    turn ^= 1u;
                    continue;
                }
                cut_first = first;
                cut_last = last;
            }
            const int32_t half0 = t.n0 + h * Cfg::HC;
            const uint32_t sb0 = terms0 + turn * Cfg::TERMS + uint32_t(h) * Cfg::GROUP_TERMS, bias0 = sb0 + 4u * Cfg::HC;
            turn ^= 1u;
            const float sa = p.epi.alpha * __uint_as_float(ptx::ld_shared_u32(sb0 + 8u * Cfg::HC + 4u * (32 * q + lane)));
            const bool small = __all_sync(0xffffffffu, bound < 4194304.f);
            const int32_t boxes = row0 < t.rows ? min(Cfg::HC / 32, (p.N - half0 + 31) / 32) : 0;
            if (cut_first <= cut_last) {
                // All contributors' sums, this one's too, a box at a time.
                const int32_t *from = p.partial + (int32_t(rank_now) * Cfg::GROUPS + h) * (Cfg::ROWS * Cfg::HC) + 4 * tid;
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
                    int32_t s32[32];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        s32[4 * i] = x[i].x;
                        s32[4 * i + 1] = x[i].y;
                        s32[4 * i + 2] = x[i].z;
                        s32[4 * i + 3] = x[i].w;
                    }
                    finish_box(p, t, s32, false, sa, sb0 + 128u * b, bias0 + 128u * b, buf, row0, half0 + 32 * b, lane);
                }
                continue;
            }
#pragma unroll
            for (int b = 0; b < Cfg::HC / 32; ++b)
                if (b < boxes) {
                    int32_t s32[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        s32[j] = sum[32 * b + j];
                    finish_box(p, t, s32, small, sa, sb0 + 128u * b, bias0 + 128u * b, buf, row0, half0 + 32 * b, lane);
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

}  // namespace

template <int ACT>
cudaError_t set_s8_tiled()
{
    static_assert(ACT == kAct, "one activation per unit");
    const cudaError_t e = set_tiled<true>();
    return e == cudaSuccess ? set_tiled<false>() : e;
}

template <int ACT>
cudaError_t launch_s8_tiled(const CUtensorMap &map_a, const CUtensorMap &map_b, const S8Params &p, bool pair, int grid,
                            cudaStream_t stream)
{
    return pair ? launch_tiled<true>(map_a, map_b, p, 2 * grid, stream)
                : launch_tiled<false>(map_a, map_b, p, grid, stream);
}

template cudaError_t set_s8_tiled<kAct>();
template cudaError_t launch_s8_tiled<kAct>(const CUtensorMap &, const CUtensorMap &, const S8Params &, bool, int,
                                           cudaStream_t);

}  // namespace tsm
