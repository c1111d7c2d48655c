// fp4_product.cu -- products of microscaled 4-bit floating-point rows:
//
//   C[i][j] = act(alpha * scale_a[i] * scale_b[j] * S[i][j] + bias[j]),
//   S[i][j] = sum over blocks b of  sa[i][b] sb[j][b] * sum over k in b of A[i][k] B[j][k]
//
// A and B are rows of e2m1 codes along k, with a scale per block of 16 (e4m3)
// or 32 (a power of two).  tcgen05.mma takes codes and block scales as they
// are: the codes from shared memory, the scales from TMEM, where tcgen05.cp
// puts a 512-byte scale tile in the order in which it lies in memory.
//
// The product is computed transposed, columns of C (rows of B, the weights) on
// the MMA's 128 TMEM lanes and rows of C (tokens) on its N side, so that one
// kernel serves one token and thousands: a tile is 128 columns by 32, 64 or 128
// rows, or a CTA pair's 256 by 256.  A lane's scale and bias of its column are
// then registers, and a warp's 32 lanes store consecutive elements of a row.
//
// One persistent CTA (or pair) per SM (pair of SMs), warp-specialised:
//   warp 0      TMA producer: codes of both operands and their scale tiles
//   warp 1      MMA issuer (the pair's leader): four MMAs of 64 k a stage
//   warps 2, 3  scales to TMEM (the pair's leader)
//   warps 4-19  epilogue, four per TMEM lane quarter, a quarter of the rows each:
//               a pair's take the sums out of the columns that the next tile needs
//               before they work on any
// A copy of a scale tile to TMEM takes the tensor core 40 cycles, and a 256 x 256
// stage with blocks of 16 has twelve, as long as its MMAs.  Copies that the MMAs'
// own thread issues run one after another with them; those of another thread run
// beside them (8192^3 296 us so, 233 otherwise), with barriers between the two.
// Few rows are bound by reading B once.  Where their tiles are few, too, a tile's K
// is cut over a cluster, whose CTAs add up each other's sums through distributed
// shared memory (1 x 4096 x 4096 7.4 us, 16.0 otherwise); else tiles of a last wave
// that costs too much are cut over the SMs, their sums joined through memory by
// whoever arrives last.  Either way in a fixed order.
#include "fp4_internal.h"
#include "fp4_ptx.cuh"
#include "s8_common.cuh"

namespace tsm {

namespace {

constexpr int kFirstEpi = 4, kEpiWarps = 16, kEpiGroups = 4;
constexpr int kFp4Threads = 32 * (kFirstEpi + kEpiWarps);
constexpr int kFp4BarGroup = 1, kFp4BarSetup = 5;  // named barriers: four epilogue groups' (1 ... 4), the setup's
// The producer tells the epilogue where its pieces lie: it decodes each once, and
// ahead of time.  It is at most the ring's stages, two accumulators and the piece in
// hand ahead, less than this many.
constexpr int kNotes = 16;
struct Fp4Note {
    S8Tile t;
    int32_t tile, kb0, kb1;  // tile -1: no more
};

template <int NT, bool PAIR, int BLK>
struct Fp4Cfg {
    static constexpr int CTAS = PAIR ? 2 : 1;
    static constexpr int COLS = 128;                     // columns of C per CTA
    static constexpr int ROWS = NT / CTAS;               // rows of C staged by one CTA
    static constexpr int TILE_M = NT, TILE_N = COLS * CTAS;
    static constexpr int B_BYTES = COLS * 128;
    static constexpr int A_BYTES = ROWS * 128;
    static constexpr int KT = kFp4BlockK / (4 * BLK);    // scale tiles along a stage's k
    static constexpr int MT = PAIR ? 2 : 1;              // scale tiles along the tile's rows
    static constexpr int SB_BYTES = KT * kScaleTile;
    static constexpr int SA_BYTES = MT * KT * kScaleTile;
    static constexpr int STAGE = B_BYTES + A_BYTES + SB_BYTES + SA_BYTES;
    // The epilogue works on CW rows at a time; a group of four warps takes every
    // fourth such chunk.
    static constexpr int CW = NT < 64 ? 8 : 16;
    static constexpr int CHUNKS = NT / CW / kEpiGroups;
    static_assert(CHUNKS >= 1 && CHUNKS * CW * kEpiGroups == NT, "chunks");
    static constexpr int EPI_ROWS = CHUNKS * CW;         // of one epilogue group
    static constexpr int NOTES_OFF = 3 * 1024, TERMS_OFF = NOTES_OFF + 32 * kNotes;
    static constexpr int COLS_OFF = TERMS_OFF + 2 * NT * 4;
    static constexpr int CTRL = COLS_OFF + 2 * kEpiWarps * 64 * 4;
    static constexpr int FIT = (232448 - 1024 - CTRL) / STAGE;
    static constexpr int S = FIT > 8 ? 8 : FIT;
    static constexpr int SMEM_BYTES = 1024 + S * STAGE + CTRL;
    static_assert(STAGE % 1024 == 0 && S >= 4, "stages");
    static_assert(SMEM_BYTES > 232448 / 2, "one CTA per SM keeps TMEM allocation uncontended");
    // TMEM: two accumulators, then the scales of a few stages.  A pair's
    // accumulators of 256 columns leave no room for those, so the second one starts
    // OVER columns before the first one's end.
    static constexpr int SET_COLS = 4 + 4 * MT;          // B's tile, then A's
    static constexpr int SCALE_COLS = KT * SET_COLS;     // of a stage
    static constexpr int PER = 4 / KT;                   // MMAs that take their scales from one set of tiles
    static constexpr int SLOTS = PAIR && BLK == 16 ? 3 : 4;
    static constexpr int OVER = PAIR ? SLOTS * SCALE_COLS : 0;
    // A group's chunks in columns that both accumulators use.
    static constexpr int EARLY = (OVER + CW * kEpiGroups - 1) / (CW * kEpiGroups);
    static constexpr int ACC1 = NT - OVER;
    static constexpr int SCALE_AT = 512 - SLOTS * SCALE_COLS;
    static_assert(S + 3 < kNotes, "notes");
    static_assert(SLOTS < S, "a slot's last use is known by its stage's");
    static_assert(ACC1 + NT <= SCALE_AT, "TMEM columns");
    static constexpr int PARTS = kEpiGroups * CTAS;
    static constexpr int32_t SLOT = CTAS * NT * COLS;    // floats
    static constexpr Fp4Kind KIND = PAIR       ? Fp4Kind::kPair
                                    : NT == 32 ? Fp4Kind::kRows32
                                    : NT == 64 ? Fp4Kind::kRows64
                                               : Fp4Kind::kRows128;
    static constexpr Fp4Shape SHAPE = fp4_shape(KIND);
    static_assert(SHAPE.tile_m == TILE_M && SHAPE.tile_n == TILE_N && SHAPE.slot_bytes == 4 * SLOT && SHAPE.parts == PARTS,
                  "the host's idea of a tile");
    // The MMA's descriptor: e2m1 x e2m1 (bits 7-9 and 10-12 = 1), both K-major, N
    // / 8 from bit 17, scales e4m3 or e8m0 (bit 23), M / 16 from bit 24.  With two
    // scales a row for 64 k, the upper two of a tile's four are chosen by 2 at bits
    // 4-5 (N side) and 29-30 (M side).
    static constexpr uint32_t IDESC = (1u << 7) | (1u << 10) | (uint32_t(NT >> 3) << 17) | (uint32_t(BLK == 32) << 23) |
                                      (uint32_t(COLS * CTAS >> 4) << 24);
    static constexpr uint32_t UPPER = (2u << 4) | (2u << 29);
};

// A CTA's (or pair's) pieces: the schedule's or, in a cluster that cuts a tile's K,
// the CTA's share of the cluster's one tile.
template <bool WARP>
struct Fp4Walk {
    PieceWalk<WARP> w;
    int32_t tile, kb0, kb1;
    bool split;
    __device__ __forceinline__ Fp4Walk(const SharedSchedule<WARP> &shared, const Fp4Params &p, int32_t worker)
        : w(shared, worker), tile(-1), kb0(0), kb1(0), split(p.ranks > 1)
    {
    }
    __device__ __forceinline__ bool advance(const SharedSchedule<WARP> &shared, const Fp4Params &p)
    {
        if (split) {
            if (tile >= 0)
                return false;
            const int32_t rank = int32_t(ptx::cluster_ctarank());
            tile = int32_t(ptx::cluster_id());
            kb0 = rank * p.kb / p.ranks;
            kb1 = (rank + 1) * p.kb / p.ranks;
            return true;
        }
        const bool more = w.advance(shared);
        tile = w.tile;
        kb0 = w.kb0;
        kb1 = w.kb1;
        return more;
    }
};

// Shared-memory descriptor of a scale tile: 32 rows of 16 bytes, no swizzle,
// groups of eight rows 128 bytes apart.
__device__ __forceinline__ uint64_t desc_scales(uint32_t saddr)
{
    return (uint64_t(128 >> 4) << 32) | (uint64_t(1) << 46) | uint64_t((saddr & 0x3FFFFu) >> 4);
}

// CW rows of a lane's column of C: scaled, biased, activated.  sa_at: the rows'
// scales; sb: the column's, with alpha in it.
template <int CW>
__device__ __forceinline__ void scale_and_activate(const Fp4Params &p, float (&v)[CW], uint32_t sa_at, float sb, float bias)
{
#pragma unroll
    for (int j = 0; j < CW; j += 4) {
        const uint4 s = ptx::ld_shared_v4(sa_at + 4u * j);
        ptx::mul_fma2(v[j], v[j + 1], __uint_as_float(s.x), __uint_as_float(s.y), sb, bias);
        ptx::mul_fma2(v[j + 2], v[j + 3], __uint_as_float(s.z), __uint_as_float(s.w), sb, bias);
    }
    with_activation<kActRuntime>(p.epi.act, [&](auto act) {
        if constexpr (decltype(act)::value == kActSilu) {
#pragma unroll
            for (int j = 0; j < CW; j += 2)
                ptx::silu2(v[j], v[j + 1]);
        } else {
#pragma unroll
            for (int j = 0; j < CW; ++j)
                v[j] = epi_act(v[j], decltype(act)::value, p.epi.slope);
        }
    });
}

// CW values of a lane's column to `rows` rows of C from element `at` on (`left`: the
// columns that are there from the lane's own on).  16-bit types go in pairs of
// columns where they are aligned: neighbour lanes exchange values, so that even
// lanes store two columns of one row, odd lanes of the next.  FULL: all rows and
// columns are there.
template <int CW, bool FULL>
__device__ __forceinline__ void store_rows(const Fp4Params &p, const float (&v)[CW], int64_t at, int32_t rows, int32_t left, int lane)
{
    if (p.epi.out_type == kOutF32) {
        float *c = static_cast<float *>(p.C) + at;
        if (FULL || left > 0) {
#pragma unroll
            for (int j = 0; j < CW; ++j, c += p.ldc)
                if (FULL || j < rows)
                    *c = v[j];
        }
        return;
    }
    uint16_t *c = static_cast<uint16_t *>(p.C) + at;
    if (p.vec_c) {
        const int odd = lane & 1;
        const uint32_t halves = odd ? 0x3276u : 0x5410u;
        c += odd * (p.ldc - 1);
        uint32_t two[CW / 2];
        if (p.epi.out_type == kOutBF16) {
#pragma unroll
            for (int j = 0; j < CW; j += 2)
                two[j / 2] = out16_pair(v[j], v[j + 1], kOutBF16);
        } else {
#pragma unroll
            for (int j = 0; j < CW; j += 2)
                two[j / 2] = out16_pair(v[j], v[j + 1], kOutF16);
        }
#pragma unroll
        for (int j = 0; j < CW; j += 2)
            two[j / 2] = __byte_perm(two[j / 2], __shfl_xor_sync(0xffffffffu, two[j / 2], 1), halves);
        const int64_t step = 2 * p.ldc;
#pragma unroll
        for (int j = 0; j < CW; j += 2, c += step) {
            if (FULL) {
                *reinterpret_cast<uint32_t *>(c) = two[j / 2];
            } else if (j + odd < rows) {
                if (left + odd > 1)
                    *reinterpret_cast<uint32_t *>(c) = two[j / 2];
                else if (left + odd == 1)
                    *c = uint16_t(two[j / 2]);
            }
        }
    } else if (FULL || left > 0) {
#pragma unroll
        for (int j = 0; j < CW; ++j, c += p.ldc)
            if (FULL || j < rows)
                *c = uint16_t(epi_out16(v[j], p.epi.out_type));
    }
}

template <int NT, bool PAIR, int BLK>
__global__ void __launch_bounds__(kFp4Threads, 1)
    tsm_fp4_kernel(const __grid_constant__ Fp4Maps maps, const Fp4Params p)
{
    using Cfg = Fp4Cfg<NT, PAIR, BLK>;
    constexpr int S = Cfg::S;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const uint32_t ctrl = base + S * Cfg::STAGE;
    // Barriers.  `full`, `tempty` and `over` are used in the pair's leader only.
    const uint32_t full0 = ctrl;               // [S] a stage has landed (both CTAs')
    const uint32_t empty0 = ctrl + 64u;        // [S] the MMAs that read it are done
    const uint32_t tfull0 = ctrl + 128u;       // [2] accumulator complete
    const uint32_t tempty0 = ctrl + 144u;      // [2] accumulator read out
    const uint32_t over = ctrl + 160u;         // the columns that both accumulators share are read out
    const uint32_t done_bar = ctrl + 168u;     // all MMAs completed
    const uint32_t tmem_slot = ctrl + 176u;
    const uint32_t flag = ctrl + 180u;         // this CTA gives up
    const uint32_t last_flag = ctrl + 184u;    // [4] one per epilogue group
    const uint32_t sfull0 = ctrl + 200u;       // [SLOTS] a stage's scales are in TMEM
    const uint32_t sdone_bar = ctrl + 232u;    // all copies of scales completed
    const SharedSchedule<false> sched{ctrl + 256u};
    const SharedSchedule<true> wsched{ctrl + 256u};
    const uint32_t gtab = ctrl + 1024u, grows = ctrl + 2048u;
    const uint32_t note0 = ctrl + 320u;        // [kNotes] a note has been written
    const uint32_t sums0 = ctrl + 512u;        // [epilogue warp] a cluster's CTAs' sums are in shared memory
    const uint32_t notes = ctrl + Cfg::NOTES_OFF;
    const uint32_t terms0 = ctrl + Cfg::TERMS_OFF;  // [2][group][its rows' scales]
    const uint32_t cols0 = ctrl + Cfg::COLS_OFF;    // [2][epilogue warp][its columns' scales, biases]

    const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x >> 5), 0);  // (uniform to the compiler)
    const int lane = int(threadIdx.x & 31);
    const uint32_t rank = PAIR ? ptx::cluster_ctarank() : 0u;
    const int32_t worker = int32_t(PAIR ? (blockIdx.x >> 1) : blockIdx.x);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            ptx::mbar_init(full0 + 8u * s, 1);
            ptx::mbar_init(empty0 + 8u * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(tfull0 + 8u * b, 1);
            ptx::mbar_init(tempty0 + 8u * b, kEpiWarps * Cfg::CTAS);
        }
        for (int i = 0; i < Cfg::SLOTS; ++i)
            ptx::mbar_init(sfull0 + 8u * i, 2);
        for (int i = 0; i < kNotes; ++i)
            ptx::mbar_init(note0 + 8u * i, 1);
        for (int i = 0; !PAIR && i < kEpiWarps; ++i)
            ptx::mbar_init(sums0 + 8u * i, uint32_t(p.ranks));
        if (PAIR)
            ptx::mbar_init(over, kEpiWarps * Cfg::CTAS);
        ptx::mbar_init(done_bar, 1);
        ptx::mbar_init(sdone_bar, 2);
        ptx::st_shared_u32(flag, 0u);
        if (!p.group_rows)
            sched.put(p.sched);
        ptx::fence_mbar_init();
        ptx::prefetch_tensormap(&maps.a);
        ptx::prefetch_tensormap(&maps.b);
        ptx::prefetch_tensormap(&maps.scales_a);
        ptx::prefetch_tensormap(&maps.scales_b);
    }
    __syncwarp();
    ptx::cta_sync();  // the barriers are there
    const bool split = !PAIR && p.ranks > 1;
    if (PAIR || split)
        ptx::cluster_arrive_relaxed();
    chain_next();
    if constexpr (PAIR)
        ptx::cluster_wait();  // the peer is there, and its barriers
    // Unless the tiles are counted on the device, the producer has all it needs
    // by now, and its first loads do not wait for the rest.
    const bool early = warp == 0 && !p.group_rows;
    if (!early && warp == 1) {
        ptx::tmem_alloc<PAIR>(tmem_slot, 512);
        ptx::tmem_relinquish<PAIR>();
    }
    chain_wait();
    if (!early) {
        if (warp == 2 && p.group_rows) {
            build_s8_groups<Cfg::TILE_M>(p, gtab, grows);
            if (lane == 0) {
                S8Schedule s;
                s.plan(int32_t(ptx::ld_shared_u32(gtab + 4u * (p.batch - 1))), p.kb, p.workers, p.sched_price, p.sched_part);
                sched.put(s);
            }
        }
        // (All warps that came here: all, or all but the first.)
        ptx::tc_fence_before_sync();
        ptx::named_bar_sync(kFp4BarSetup, p.group_rows ? kFp4Threads : kFp4Threads - 32);
        ptx::tc_fence_after_sync();
    }
    const uint32_t tmem = early ? 0u : __shfl_sync(0xffffffffu, ptx::ld_shared_u32(tmem_slot), 0);

    if (warp == 0) {
        if (lane == 0) {
            // ---------------- TMA producer (each CTA fills its own stages)
            const uint32_t full_lead0 = PAIR ? ptx::mapa_shared(full0, 0) : full0;
            uint32_t stage = 0, phase = 0, issued = 0;
            bool ok = true;
            auto load = [&](uint32_t to, const CUtensorMap &map, uint32_t bar, int32_t c0, int32_t c1, int32_t c2) {
                if constexpr (PAIR)
                    ptx::tma_load_3d_pair(to, &map, bar, c0, c1, c2);
                else
                    ptx::tma_load_3d(to, &map, bar, c0, c1, c2);
            };
            uint32_t note = 0;
            const auto tell = [&](const S8Tile &t, int32_t tile, int32_t kb0, int32_t kb1) {
                const uint32_t to = notes + 32u * (note % kNotes);
                ptx::st_shared_v4(to, uint32_t(t.m0), uint32_t(t.n0), uint32_t(t.z), uint32_t(t.rows));
                ptx::st_shared_v4(to + 16u, uint32_t(tile), uint32_t(kb0), uint32_t(kb1), 0u);
                ptx::mbar_arrive(note0 + 8u * (note % kNotes));
                ++note;
            };
            for (Fp4Walk<false> w(sched, p, worker); ok && w.advance(sched, p);) {
                const S8Tile t = tile_at(w.tile, p, gtab, grows, Cfg::TILE_M, Cfg::TILE_N);
                tell(t, w.tile, w.kb0, w.kb1);
                const int32_t col = t.n0 + int32_t(rank) * Cfg::COLS, row = t.m0 + int32_t(rank) * Cfg::ROWS;
                const int32_t sb_row = t.z * p.scale_rows_b + col / 128, sa_row = t.z * p.scale_rows_a + t.m0 / 128;
                for (int32_t kb = w.kb0; kb < w.kb1; ++kb) {
                    if (!s8_wait<PAIR>(empty0 + 8u * stage, phase ^ 1u, flag, p, kStatusProducer)) {
                        ok = false;
                        break;
                    }
                    const uint32_t to = base + stage * Cfg::STAGE;
                    const uint32_t fb = full_lead0 + 8u * stage;
                    // Both CTAs' bytes are counted on the leader's barrier.
                    if (rank == 0)
                        ptx::mbar_arrive_expect_tx(full0 + 8u * stage, Cfg::CTAS * Cfg::STAGE);
                    load(to, maps.b, fb, kb * 128, col, t.z);
                    load(to + Cfg::B_BYTES, maps.a, fb, kb * 128, row, t.z);
                    load(to + Cfg::B_BYTES + Cfg::A_BYTES, maps.scales_b, fb, 0, kb * Cfg::KT, sb_row);
                    load(to + Cfg::B_BYTES + Cfg::A_BYTES + Cfg::SB_BYTES, maps.scales_a, fb, 0, kb * Cfg::KT, sa_row);
                    ++issued;
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            tell({}, -1, 0, 0);
            if (rank == 0) {
                // No TMA write into shared memory outlives the CTA (the pair):
                // the last S loads, the stages from `stage` on, oldest first.
                for (int i = 0; i < S; ++i) {
                    if (issued + i >= uint32_t(S))
                        s8_wait<PAIR>(full0 + 8u * stage, phase ^ 1u, flag, p, kStatusDrain, false);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            } else if (ptx::ld_shared_u32(flag)) {
                // The peer's loads are counted in the leader only: after giving
                // up, a fixed time for them to land.
                const uint64_t t0 = ptx::globaltimer_ns();
                while (ptx::globaltimer_ns() - t0 < 200000ull) {
                }
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            // ---------------- MMA issuer: the warp in step, its first lane issues
            const bool on = lane == 0;
            const auto wait = [&](bool good) { return __all_sync(0xffffffffu, good) != 0; };
            constexpr uint16_t both = PAIR ? 3 : 1;
            uint32_t stage = 0, phase = 0, acc = 0, aphase = 0, turn = 0, slot = 0, sphase = 0;
            bool ok = true;
            for (Fp4Walk<true> w(wsched, p, worker); ok && w.advance(wsched, p);) {
                ok = wait(s8_wait<PAIR, PAIR>(tempty0 + 8u * acc, aphase ^ 1u, flag, p, kStatusMma));
                if (PAIR && ok)
                    ok = wait(s8_wait<PAIR, PAIR>(over, turn ^ 1u, flag, p, kStatusMma));
                if (!ok)
                    break;
                ptx::tc_fence_after_sync();
                const uint32_t d = tmem + acc * uint32_t(Cfg::ACC1);
                for (int32_t kb = w.kb0; kb < w.kb1; ++kb) {
                    ok = wait(s8_wait<PAIR>(full0 + 8u * stage, phase, flag, p, kStatusMma) &&
                              s8_wait<PAIR>(sfull0 + 8u * slot, sphase, flag, p, kStatusMma));
                    if (!ok)
                        break;
                    ptx::tc_fence_after_sync();
                    const uint32_t sb = base + stage * Cfg::STAGE, sa = sb + Cfg::B_BYTES;
                    const uint32_t scales = tmem + Cfg::SCALE_AT + slot * uint32_t(Cfg::SCALE_COLS);
                    // (What lies past K is zeros.)
                    const int32_t left = p.K - kb * kFp4BlockK;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t tsb = scales + uint32_t(kk / Cfg::PER * Cfg::SET_COLS);
                        if (64 * kk < left)
                            ptx::mma_fp4<PAIR, BLK>(on, d, desc_a(sb + 32u * kk), desc_a(sa + 32u * kk),
                                                    Cfg::IDESC | (kk % Cfg::PER ? Cfg::UPPER : 0u), tsb, tsb + 4u,
                                                    (kb > w.kb0 || kk > 0) ? 1u : 0u);
                    }
                    ptx::mma_commit_if<PAIR>(on, empty0 + 8u * stage, both);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++slot == uint32_t(Cfg::SLOTS)) {
                        slot = 0;
                        sphase ^= 1u;
                    }
                }
                if (!ok)
                    break;
                ptx::mma_commit_if<PAIR>(on, tfull0 + 8u * acc, both);
                turn ^= 1u;
                acc ^= 1u;
                if (acc == 0)
                    aphase ^= 1u;
            }
            // Every MMA must finish before TMEM is freed.
            ptx::mma_commit_if<PAIR>(on, done_bar, 1);
            s8_wait<PAIR>(done_bar, 0, flag, p, kStatusDrain, false);
        }
        __syncwarp();
    } else if (warp < kFirstEpi) {
        if (rank == 0) {
            // ---------------- scales to TMEM: the warp in step, as above
            const bool on = lane == 0;
            const auto wait = [&](bool good) { return __all_sync(0xffffffffu, good) != 0; };
            uint32_t stage = 0, phase = 0, slot = 0, count = 0;
            // The stage SLOTS before, whose MMAs read the same slot: where they end
            // it is free.
            uint32_t old_stage = 0, old_phase = 0;
            bool ok = true;
            for (Fp4Walk<true> w(wsched, p, worker); ok && w.advance(wsched, p);) {
                for (int32_t kb = w.kb0; kb < w.kb1; ++kb) {
                    ok = wait(s8_wait<PAIR>(full0 + 8u * stage, phase, flag, p, kStatusMma) &&
                              (count < uint32_t(Cfg::SLOTS) || s8_wait<PAIR>(empty0 + 8u * old_stage, old_phase, flag, p, kStatusMma)));
                    if (!ok)
                        break;
                    ptx::tc_fence_after_sync();
                    const uint32_t ssb = base + stage * Cfg::STAGE + Cfg::B_BYTES + Cfg::A_BYTES, ssa = ssb + Cfg::SB_BYTES;
                    const uint32_t to = tmem + Cfg::SCALE_AT + slot * uint32_t(Cfg::SCALE_COLS);
#pragma unroll
                    for (int i0 = 0; i0 < Cfg::KT; i0 += 2) {
                        const int i = i0 + (warp & 1);
                        ptx::tmem_cp_scales<PAIR>(on, to + uint32_t(i * Cfg::SET_COLS), desc_scales(ssb + uint32_t(i * kScaleTile)));
#pragma unroll
                        for (int m = 0; m < Cfg::MT; ++m)
                            ptx::tmem_cp_scales<PAIR>(on, to + uint32_t(i * Cfg::SET_COLS + 4 + 4 * m),
                                                      desc_scales(ssa + uint32_t((m * Cfg::KT + i) * kScaleTile)));
                    }
                    ptx::mma_commit_if<PAIR>(on, sfull0 + 8u * slot, 1);
                    if (++stage == S) {
                        stage = 0;
                        phase ^= 1u;
                    }
                    if (++slot == uint32_t(Cfg::SLOTS))
                        slot = 0;
                    if (++count > uint32_t(Cfg::SLOTS) && ++old_stage == S) {
                        old_stage = 0;
                        old_phase ^= 1u;
                    }
                }
            }
            // So must every copy.
            ptx::mma_commit_if<PAIR>(on, sdone_bar, 1);
            s8_wait<PAIR>(sdone_bar, 0, flag, p, kStatusDrain, false);
        }
        __syncwarp();
    } else {
        // ---------------- epilogue
        constexpr int CW = Cfg::CW, EARLY = Cfg::EARLY;
        const int h = (warp - kFirstEpi) >> 2, q = warp & 3;
        uint32_t acc = 0, aphase = 0, note = 0;
        bool met = !split;
        // The group's chunks of a tile, those in the columns that both accumulators
        // use first: the last ones of the first, the first ones of the second.
        const auto row_of = [&](int i, uint32_t a) {
            return PAIR && a == 0 ? (kEpiGroups * (Cfg::CHUNKS - i) - 1 - h) * CW : (kEpiGroups * i + h) * CW;
        };
        const auto rows_of = [&](uint32_t a) {
            return terms0 + (a * uint32_t(kEpiGroups) + uint32_t(h)) * uint32_t(4 * Cfg::EPI_ROWS);
        };
        const auto cols_of = [&](uint32_t a) {
            return cols0 + (a * uint32_t(kEpiWarps) + uint32_t(warp - kFirstEpi)) * 256u + 4u * uint32_t(lane);
        };
        const auto read = [&]() {
            const uint32_t from = notes + 32u * (note % kNotes);
            const uint4 x = ptx::ld_shared_v4(from), y = ptx::ld_shared_v4(from + 16u);
            return Fp4Note{{int32_t(x.x), int32_t(x.y), int32_t(x.z), int32_t(x.w)}, int32_t(y.x), int32_t(y.y), int32_t(y.z)};
        };
        // The next piece's scales and bias, on their way while this one's sums are
        // stored.
        bool ok = true;
        const auto look_ahead = [&](uint32_t a) {
            ok = s8_wait<PAIR>(note0 + 8u * (note % kNotes), (note / kNotes) & 1u, flag, p, kStatusEpilogue);
            if (!ok)
                return;
            const Fp4Note n = read();
            if (n.tile < 0)
                return;
            const int32_t col = n.t.n0 + int32_t(rank) * Cfg::COLS + 32 * q + lane;
            // A quarter of the group's rows each.
            const int at = q * (Cfg::EPI_ROWS / 4) + lane;
            const int32_t row = n.t.m0 + row_of(at / CW, a) + at % CW;
            if (lane < Cfg::EPI_ROWS / 4)
                ptx::fetch_f32(rows_of(a) + 4u * uint32_t(at),
                               p.scale_a && row < n.t.rows ? p.scale_a + n.t.z * p.sa_stride + row : nullptr, 1.f);
            ptx::fetch_f32(cols_of(a), p.scale_b && col < p.N ? p.scale_b + n.t.z * p.sb_stride + col : nullptr, 1.f);
            ptx::fetch_f32(cols_of(a) + 128u, p.epi.bias && col < p.N ? p.epi.bias + n.t.z * p.epi.bias_stride + col : nullptr, 0.f);
        };
        look_ahead(acc);
        for (;;) {
            Fp4Note w = {{}, -1, 0, 0};
            if (ok)
                w = read();
            ++note;
            ok = w.tile >= 0 && s8_wait<PAIR>(tfull0 + 8u * acc, aphase, flag, p, kStatusEpilogue);
            // The group's warps go on or stop together (they meet below), and have
            // each other's terms.
            ptx::fetch_wait();
            if (!__all_sync(0xffffffffu, ptx::named_bar_and(kFp4BarGroup + h, 128, ok)))
                break;
            const S8Tile &t = w.t;
            const int32_t col = t.n0 + int32_t(rank) * Cfg::COLS + 32 * q + lane;
            const int32_t rows = t.rows - t.m0;
            const uint32_t sa0 = rows_of(acc);
            const float sb = p.epi.alpha * __uint_as_float(ptx::ld_shared_u32(cols_of(acc)));
            const float bias = __uint_as_float(ptx::ld_shared_u32(cols_of(acc) + 128u));
            const bool whole = w.kb1 - w.kb0 == p.kb;
            ptx::tc_fence_after_sync();
            const uint32_t from = tmem + (uint32_t(32 * q) << 16) + acc * uint32_t(Cfg::ACC1);
            const int64_t at = int64_t(t.z) * p.sC + int64_t(t.m0) * p.ldc + col;
            const auto release = [&](uint32_t bar) {
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0)
                    arrive_leader<PAIR>(PAIR ? ptx::mapa_shared(bar, 0) : bar);
            };
            const bool full_columns = t.n0 + int32_t(rank) * Cfg::COLS + Cfg::COLS <= p.N;
            const auto finish = [&](float (&v)[CW], int i, int32_t row) {
                scale_and_activate(p, v, sa0 + uint32_t(4 * CW * i), sb, bias);
                if (full_columns && row + CW <= rows)
                    store_rows<CW, true>(p, v, at + row * p.ldc, CW, 0, lane);
                else
                    store_rows<CW, false>(p, v, at + row * p.ldc, rows - row, p.N - col, lane);
            };
            if (whole) {
                float early[EARLY ? EARLY : 1][CW];
                if constexpr (EARLY > 0) {
#pragma unroll
                    for (int i = 0; i < EARLY; ++i)
                        ptx::tmem_ld_cols(from + uint32_t(row_of(i, acc)), early[i]);
                    release(over);
                }
                look_ahead(acc ^ 1u);
                // (Unrolled: the chunks' buffers are registers.)
#pragma unroll
                for (int i = 0; i < Cfg::CHUNKS; ++i) {
                    const int32_t row = row_of(i, acc);
                    float v[CW];
                    if (i >= EARLY && row < rows)
                        ptx::tmem_ld_cols(from + uint32_t(row), v);
                    if (i == Cfg::CHUNKS - 1)
                        release(tempty0 + 8u * acc);
#pragma unroll
                    for (int k = 0; k < EARLY; ++k)
                        if (i == k) {
#pragma unroll
                            for (int j = 0; j < CW; ++j)
                                v[j] = early[k][j];
                        }
                    if (row < rows)
                        finish(v, i, row);
                }
            } else if (split) {
                // A share of the tile's K.  The sums go to the ring's place in shared
                // memory ([row][column]; all of this CTA's MMAs are done with it), each
                // chunk is added up by one CTA, in the order of K, by the warp that
                // has the same columns and rows in each.
                ptx::cluster_wait();  // the others are there, and their barriers
                met = true;
                const uint32_t mine = base + uint32_t(32 * q + lane) * 4u;
#pragma unroll 1
                for (int i = 0; i < Cfg::CHUNKS; ++i) {
                    const int32_t row = row_of(i, acc);
                    if (row < rows) {
                        float v[CW];
                        ptx::tmem_ld_cols(from + uint32_t(row), v);
#pragma unroll
                        for (int j = 0; j < CW; ++j)
                            ptx::st_shared_u32(mine + uint32_t(row + j) * 512u, __float_as_uint(v[j]));
                    }
                }
                __syncwarp();
                const uint32_t bar = sums0 + 8u * uint32_t(warp - kFirstEpi);
                if (lane < p.ranks)
                    ptx::mbar_arrive_cluster(ptx::mapa_shared(bar, uint32_t(lane)));
                ok = __all_sync(0xffffffffu, s8_wait<PAIR, true>(bar, 0, flag, p, kStatusReduce));
#pragma unroll 1
                for (int i = 0; ok && i < Cfg::CHUNKS; ++i) {
                    const int32_t row = row_of(i, acc);
                    if (row < rows && (row / CW) % p.ranks == int32_t(ptx::cluster_ctarank())) {
                        float v[CW];
#pragma unroll
                        for (int j = 0; j < CW; ++j)
                            v[j] = 0.f;
                        // (Four CTAs' loads in flight together.)
#pragma unroll 4
                        for (int32_t r = 0; r < p.ranks; ++r) {
                            const uint32_t theirs = ptx::mapa_shared(mine + uint32_t(row) * 512u, uint32_t(r));
#pragma unroll
                            for (int j = 0; j < CW; ++j)
                                if (row + j < rows)
                                    v[j] += __uint_as_float(ptx::ld_cluster_u32(theirs + 512u * uint32_t(j)));
                        }
                        finish(v, i, row);
                    }
                }
                look_ahead(acc ^ 1u);
            } else {
                // A piece: its sums go to this worker's slot ([row][column]), and
                // whoever arrives last adds up the contributors', in their order.
                // A tile's first contributor holds its first block and uses its
                // second slot; the others start in the tile: their first.
                const S8Schedule cut = wsched.all();
                const int32_t first = cut.owner(w.tile * cut.kb), last = cut.owner((w.tile + 1) * cut.kb - 1);
                float *const parts = p.partial + int32_t(rank) * NT * Cfg::COLS + 32 * q + lane;
                float *const to = parts + int64_t(2 * worker + (worker == first)) * Cfg::SLOT;
#pragma unroll 1
                for (int i = 0; i < Cfg::CHUNKS; ++i) {
                    const int32_t row = row_of(i, acc);
                    if (row < rows) {
                        float v[CW];
                        ptx::tmem_ld_cols(from + uint32_t(row), v);
#pragma unroll
                        for (int j = 0; j < CW; ++j)
                            if (row + j < rows)
                                __stcg(to + (row + j) * Cfg::COLS, v[j]);
                    }
                }
                if (PAIR)
                    release(over);
                release(tempty0 + 8u * acc);
                look_ahead(acc ^ 1u);
                __threadfence();
                ptx::named_bar_sync(kFp4BarGroup + h, 128);
                // (A pair's first accumulator is taken from its end: the groups the other way round.)
                const int part = int(rank) * kEpiGroups + (PAIR && acc == 0 ? kEpiGroups - 1 - h : h);
                if (q == 0)
                    ptx::st_shared_u32(last_flag + 4u * h, arrive_last(p.arrivals + w.tile * Cfg::PARTS + part, p.tag,
                                                                      uint32_t(last - first + 1), lane));
                ptx::named_bar_sync(kFp4BarGroup + h, 128);
                const bool mine = __any_sync(0xffffffffu, ptx::ld_shared_u32(last_flag + 4u * h) != 0);
                __threadfence();
                if (mine) {
#pragma unroll 1
                    for (int i = 0; i < Cfg::CHUNKS; ++i) {
                        const int32_t row = row_of(i, acc);
                        if (row < rows) {
                            float v[CW];
#pragma unroll
                            for (int j = 0; j < CW; ++j)
                                v[j] = 0.f;
                            // (Two contributors' loads in flight together.)
#pragma unroll 2
                            for (int32_t k = first; k <= last; ++k) {
                                const float *theirs = parts + int64_t(2 * k + (k == first)) * Cfg::SLOT + row * Cfg::COLS;
#pragma unroll
                                for (int j = 0; j < CW; ++j)
                                    if (row + j < rows)
                                        v[j] += __ldcg(theirs + j * Cfg::COLS);
                            }
                            finish(v, i, row);
                        }
                    }
                }
            }
            acc ^= 1u;
            if (acc == 0)
                aphase ^= 1u;
        }
        ptx::fetch_wait();
        if (!met)
            ptx::cluster_wait();
    }

    ptx::tc_fence_before_sync();
    if (split && warp < kFirstEpi)
        ptx::cluster_wait();  // (the meeting that began at the start; the epilogue's warps have been there)
    ptx::cta_sync();
    if (PAIR || split)
        ptx::cluster_sync();  // no CTA leaves while another may still read its sums or signal it
    if (warp == 1) {
        __syncwarp();
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc<PAIR>(ptx::ld_shared_u32(tmem_slot), 512);
    }
}

// fn with the tile and block of a kernel fixed at compile time.
template <int NT, bool PAIR, int BLK>
struct Fp4Tag {
    static constexpr int rows = NT, block = BLK;
    static constexpr bool pair = PAIR;
};
template <int BLK, typename F>
cudaError_t with_kind(Fp4Kind kind, F &&fn)
{
    switch (kind) {
    case Fp4Kind::kRows32: return fn(Fp4Tag<32, false, BLK>{});
    case Fp4Kind::kRows64: return fn(Fp4Tag<64, false, BLK>{});
    case Fp4Kind::kRows128: return fn(Fp4Tag<128, false, BLK>{});
    default: return fn(Fp4Tag<256, true, BLK>{});
    }
}

}  // namespace

cudaError_t set_fp4_attributes(Fp4Capacity *cap)
{
    for (const Fp4Kind kind : {Fp4Kind::kRows32, Fp4Kind::kRows64, Fp4Kind::kRows128, Fp4Kind::kPair}) {
        const auto set = [&](auto tag) {
            using T = decltype(tag);
            const auto kernel = tsm_fp4_kernel<T::rows, T::pair, T::block>;
            constexpr int smem = Fp4Cfg<T::rows, T::pair, T::block>::SMEM_BYTES;
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            // (Both block sizes' kernels have one CTA on an SM, and alike clusters.)
            for (int i = 0; e == cudaSuccess && !T::pair && T::block == 16 && i < Fp4Capacity::RANKS; ++i) {
                cudaLaunchConfig_t cfg = {};
                cfg.gridDim = dim3(unsigned(i + 1), 1, 1);
                cfg.blockDim = dim3(kFp4Threads, 1, 1);
                cfg.dynamicSmemBytes = smem;
                cudaLaunchAttribute attr;
                attr.id = cudaLaunchAttributeClusterDimension;
                attr.val.clusterDim.x = unsigned(i + 1);
                attr.val.clusterDim.y = 1;
                attr.val.clusterDim.z = 1;
                cfg.attrs = &attr;
                cfg.numAttrs = 1;
                e = cudaOccupancyMaxActiveClusters(&cap->clusters[int(kind)][i], kernel, &cfg);
            }
            return e;
        };
        cudaError_t e = with_kind<16>(kind, set);
        if (e == cudaSuccess)
            e = with_kind<32>(kind, set);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

cudaError_t launch_fp4(const Fp4Maps &maps, const Fp4Params &p, Fp4Kind kind, int block, int grid, cudaStream_t stream)
{
    const auto run = [&](auto tag) {
        using T = decltype(tag);
        const unsigned cluster = T::pair ? 2u : unsigned(p.ranks);
        return launch_chained(tsm_fp4_kernel<T::rows, T::pair, T::block>, dim3(unsigned(grid) * cluster), kFp4Threads,
                              Fp4Cfg<T::rows, T::pair, T::block>::SMEM_BYTES, cluster > 1 ? cluster : 0u, stream, maps, p);
    };
    return block == 16 ? with_kind<16>(kind, run) : with_kind<32>(kind, run);
}

}  // namespace tsm
