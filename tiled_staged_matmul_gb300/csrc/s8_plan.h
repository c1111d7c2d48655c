// s8_plan.h -- how an 8-bit product is launched: the kernel, its tiles and their
// schedule, and the workspace.  Host arithmetic only: no CUDA call is made.
#pragma once

#include "ops_internal.h"

#include <algorithm>

namespace tsm {

// An operand the tensor-memory accelerator can address (no copy needed).
inline bool addressable(const int8_t *x, int64_t ld, int64_t stride, int64_t rows, int64_t batch)
{
    return (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && (rows == 1 || ld % 16 == 0) && (batch == 1 || stride % 16 == 0);
}

// CTAs per cluster of a few-rows launch: the least estimated time over 1 to 8.
// A CTA's rate is its share of the memory's, or what its warps can multiply if
// that is less; its pairs of warps (8, or 4 for two blocks of rows) take whole
// blocks; adding up their sums takes 1 us.  The launch waits for the cluster
// with the most tiles.  Finishing a tile takes 2 us, 3 where its sums pass
// between CTAs; it hides behind the next tile if that takes longer.  (Within 6 %
// of the best of the eight on nine shapes, 1 x 4096 x 4096 to 16 x 57344 x 8192;
// the worst of them took up to four times as long.)
inline int few_rows_ranks(int64_t tiles, int32_t kb, const S8Capacity &cap, bool two, int *clusters)
{
    const double block = 8192.0;                   // bytes of 32 k x 256 columns
    const double memory = 6.0e6;                   // bytes per us, all CTAs
    const double most = two ? 38.0e3 : 45.0e3;     // bytes per us, one CTA
    const int pairs = two ? 4 : 8;
    int best = 1;
    double best_us = 0.0;
    for (int i = 0; i < S8Capacity::KINDS; ++i) {
        const int ranks = i + 1;
        if (cap.clusters[i] <= 0 || (i > 0 && ranks > kb))
            continue;
        const int64_t n = std::min<int64_t>(tiles, cap.clusters[i]);
        const double rate = std::min(most, memory / double(n * ranks));
        const double finish = ranks > 1 ? 3.0 : 2.0;
        const int64_t steps = ((kb + ranks - 1) / ranks + pairs - 1) / pairs;
        const double each = std::max(finish, double(steps * pairs) * block / rate + 1.0);
        const double us = double((tiles + n - 1) / n) * each + finish;
        if (i == 0 || us < best_us) {
            best = ranks;
            best_us = us;
            *clusters = int(n);
        }
    }
    return best;
}

// The tiled kernel: a CTA per 128 x 128 tile, or a pair per 256 x 256, which does
// twice the work at one SM's time for a block and a pair's longer start.  By the
// time of the busiest worker: 5 us and 0.66 a block of 128 k, or 6.5 and 0.75
// (the nearer of two on 20 shapes from 140 x 1072 x 272 to 512 x 14336 x 4096, us
// as single CTAs and pairs: 140 x 1072 x 272 8.1 and 10.4, 512 x 4096 x 4096 26.8
// and 33.8, 256 x 256 x 65536 42 and 52, 300 x 5008 x 8192 46.9 and 42.7, 2048^3
// 28.8 and 20.7).  A grouped launch's tiles are counted on the device; all of
// the groups' rows are taken to be there.
inline S8Kind tiled_kind(const S8Params &p, int sms)
{
    S8Kind best = S8Kind::kPair;
    double best_us = 0.0;
    for (const S8Kind kind : {S8Kind::kPair, S8Kind::kOne}) {
        const bool pair = kind == S8Kind::kPair;
        const S8Shape shape = s8_shape(kind);
        const int64_t tiles = (int64_t(p.M) + shape.tile_m - 1) / shape.tile_m *
                              ((int64_t(p.N) + shape.tile_n - 1) / shape.tile_n) * p.batch;
        if (tiles > S8Schedule::kMaxTiles)
            continue;
        S8Schedule s = {};
        s.plan(int32_t(tiles), int32_t((int64_t(p.K) + shape.block_k - 1) / shape.block_k), pair ? sms / 2 : sms);
        const double us = pair ? 6.5 + 0.75 * double(s.blocks()) : 5.0 + 0.66 * double(s.blocks());
        if (best_us == 0.0 || us < best_us) {
            best = kind;
            best_us = us;
        }
    }
    return best;
}

// A launch of a product whose sizes are all positive.
struct S8Plan {
    S8Kind kind;
    S8Shape shape;
    int32_t tiles_m, tiles_n, kb;
    int32_t workers;            // CTAs, or pairs, that share a tiled launch
    int32_t ranks;              // few rows: CTAs of a cluster
    int grid;                   // few rows: clusters; tiled: workers
    S8Schedule sched;           // tiled, not grouped
    bool pack_a, pack_b;        // copied to rows lda2 / ldb2 bytes apart first
    int64_t lda2, ldb2;
    // Workspace: the copies, the pieces' sums, the arrival words.
    int64_t bytes_a, bytes_b, bytes_p, bytes_w;

    bool few() const { return kind == S8Kind::kFew16 || kind == S8Kind::kFew32; }

    // False: more tiles than a launch can count.
    bool make(const S8Params &p, int sms, const S8Capacity &cap)
    {
        *this = {};
        // Few rows by M.  As few rows and as tiles, us: 16 x 4096 x 4096 10.5 and
        // 16.2, 16 x 14336 x 4096 18.1 and 26.1, 32 x 1024 x 1024 8.8 and 9.9, 32 x
        // 4096 x 4096 13.0 and 16.2, 32 x 57344 x 8192 121 and 130, 32 x 14336 x 4096
        // 26.4 and 25.9, 32 x 4096 x 14336 28.3 and 27.2; the few-rows kernel holds
        // no more than 32.
        // In groups of up to 32 rows most have far fewer, so those are cut into
        // sixteens and only the rows there are cost anything.  64 groups by 1408
        // columns and 2048 k, as sixteens and as tiles: 192 rows in all 43.8 and
        // 64.2, 16 each 49.9 and 64.9; but 32 each, which only the device knows, 89
        // and 65.  Groups with room for more go to the tiles whatever their counts:
        // 192 rows in all take 65 us where there is room for 33 to 128, 77 for 512.
        kind = p.M <= 16 || (p.group_rows && p.M <= 32) ? S8Kind::kFew16
               : p.M <= 32                              ? S8Kind::kFew32
                                                        : tiled_kind(p, sms);
        shape = s8_shape(kind);
        tiles_m = int32_t((int64_t(p.M) + shape.tile_m - 1) / shape.tile_m);
        tiles_n = int32_t((int64_t(p.N) + shape.tile_n - 1) / shape.tile_n);
        kb = int32_t((int64_t(p.K) + shape.block_k - 1) / shape.block_k);
        workers = kind == S8Kind::kPair ? sms / 2 : sms;
        ranks = 1;
        const int64_t tiles = int64_t(tiles_m) * tiles_n * p.batch;
        if (tiles > S8Schedule::kMaxTiles)
            return false;
        if (few()) {
            // (A grouped launch's tiles are counted on the device; the estimate is
            // for one block of rows in every group.)
            ranks = few_rows_ranks(p.group_rows ? int64_t(tiles_n) * p.batch : tiles, kb, cap,
                                   kind == S8Kind::kFew32, &grid);
        } else {
            sched.plan(int32_t(tiles), kb, workers);
            grid = p.group_rows ? workers
                                : int(std::max<int64_t>(sched.shared ? sched.cutters : 0,
                                                        std::min<int64_t>(sched.tiles, workers)));
        }
        pack_a = !addressable(p.A, p.lda, p.sA, p.M, p.batch);
        pack_b = !addressable(p.B, p.ldb, p.sB, p.K, p.batch);
        const auto up = [](int64_t x, int64_t m) { return (x + m - 1) / m * m; };
        lda2 = up(p.K, 16);
        ldb2 = up(p.N, 16);
        bytes_a = pack_a ? up(int64_t(p.batch) * p.M * lda2, 256) : 0;
        bytes_b = pack_b ? up(int64_t(p.batch) * p.K * ldb2, 256) : 0;
        // (A grouped launch's tiles are counted on the device: any number up to these.)
        const int64_t cut = few() ? 0 : p.group_rows ? 2 * int64_t(workers) : sched.shared;
        bytes_p = cut ? 2 * int64_t(workers) * shape.slot_bytes : 0;
        bytes_w = cut * shape.parts * 8;
        return true;
    }
};

}  // namespace tsm
