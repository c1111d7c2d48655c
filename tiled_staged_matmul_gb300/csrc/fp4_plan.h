// fp4_plan.h -- how a product of 4-bit rows is launched: the kernel, its tiles
// and their schedule, and the workspace.  Host arithmetic only: no CUDA call is
// made.
#pragma once

#include "fp4_internal.h"
#include "s8_plan.h"

#include <algorithm>

namespace tsm {

// A launch of a product whose sizes are all positive.
struct Fp4Plan {
    Fp4Kind kind;
    Fp4Shape shape;
    int32_t tiles_m, tiles_n, kb;
    int32_t workers;            // CTAs, or pairs, that share a launch
    int32_t ranks;              // CTAs of a cluster that cuts a tile's K
    int grid;                   // workers, or clusters
    S8Schedule sched;           // not grouped
    bool pack_a, pack_b;        // copied to rows lda2 / ldb2 bytes apart first
    int64_t lda2, ldb2;
    // Workspace: the copies, the pieces' sums, the arrival words.
    int64_t bytes_a, bytes_b, bytes_p, bytes_w;

    // Tiles, schedule and grid for one kind of kernel.  False: more tiles than a
    // launch can count.
    bool lay_out(Fp4Kind kind_, const Fp4Params &p, int sms, const Fp4Capacity &cap)
    {
        kind = kind_;
        shape = fp4_shape(kind);
        tiles_m = int32_t((int64_t(p.M) + shape.tile_m - 1) / shape.tile_m);
        tiles_n = int32_t((int64_t(p.N) + shape.tile_n - 1) / shape.tile_n);
        kb = int32_t((int64_t(p.K) + kFp4BlockK - 1) / kFp4BlockK);
        workers = kind == Fp4Kind::kPair ? sms / 2 : sms;
        const int64_t tiles = int64_t(tiles_m) * tiles_n * p.batch;
        if (tiles > S8Schedule::kMaxTiles)
            return false;
        // As many CTAs to a tile as leave all tiles in one round.
        ranks = 1;
        for (int r = 2; kind != Fp4Kind::kPair && !p.group_rows && r <= Fp4Capacity::RANKS && 2 * r <= kb; ++r)
            if (tiles <= cap.clusters[int(kind)][r - 1])
                ranks = r;
        sched.plan(int32_t(tiles), kb, workers, shape.price, shape.part);
        if (ranks > 1)
            sched.shared = 0;
        grid = p.group_rows ? workers
               : ranks > 1  ? int(tiles)
                            : int(std::max<int64_t>(sched.shared ? sched.cutters : 0, std::min<int64_t>(sched.tiles, workers)));
        return true;
    }

    // False: more tiles than a launch can count.
    bool make(const Fp4Params &p, const uint8_t *A, int64_t lda, int64_t sA, const uint8_t *B, int64_t ldb, int64_t sB, int sms,
              const Fp4Capacity &cap)
    {
        *this = {};
        const Fp4Kind rows = p.M <= 32 ? Fp4Kind::kRows32 : p.M <= 64 ? Fp4Kind::kRows64 : Fp4Kind::kRows128;
        // A CTA pair's tiles do four times the work of a CTA's of 128 rows, but there
        // are a quarter as many, and no cluster cuts them.  By the time of the busiest
        // worker, us, a block of K at a time; cutting a pair's tile adds the reading of
        // its contributors' sums.  As single CTAs and pairs, us: 150 x 1000 x 1000 7.7 and
        // 7.8, 256 x 4096 x 4096 10.5 and 12.4, 300 x 5000 x 8192 14.8 and 18.5, 512 x 512 x
        // 65536 21.2 and 49.1, 1024 x 1024 x 65536 43.6 and 53.4, 1500 x 1500 x 65536 76.2
        // and 81.8, 256 x 28672 x 8192 37.2 and 35.7, 512 x 8192 x 8192 24.2 and 18.8,
        // 2048 x 2048 x 16384 41.3 and 28.7, 4096^3 40.8 and 31.0.  The constants choose
        // the shorter in each of these.
        // Groups with room for more than 128 rows take pairs, whatever their counts,
        // which only the device knows: 64 experts' prompt 63.7 and 62.0, 8 experts'
        // 550 and 375, but 16 small ones' 24 and 27.
        if (p.M <= 128) {
            if (!lay_out(rows, p, sms, cap))
                return false;
        } else if (p.group_rows || !lay_out(rows, p, sms, cap)) {
            if (!lay_out(Fp4Kind::kPair, p, sms, cap))
                return false;
        } else {
            const double one = ranks > 1 ? 7.5 + 0.5 * ranks + 0.274 * double((kb + ranks - 1) / ranks)
                                         : 6.8 + 0.27 * double(sched.blocks());
            const Fp4Plan single = *this;
            const auto two = [this] {
                return 7.0 + (sched.shared ? 0.42 * double(sched.blocks()) + 3.0 * sched.cutters / sched.shared
                                           : 0.385 * double(sched.blocks()));
            };
            if (!lay_out(Fp4Kind::kPair, p, sms, cap) || one < two())
                *this = single;
        }
        const auto up = [](int64_t x, int64_t m) { return (x + m - 1) / m * m; };
        const int64_t width = (int64_t(p.K) + 1) / 2;
        pack_a = !addressable(reinterpret_cast<const int8_t *>(A), lda, sA, p.M, p.batch);
        pack_b = !addressable(reinterpret_cast<const int8_t *>(B), ldb, sB, p.N, p.batch);
        lda2 = ldb2 = up(width, 16);
        bytes_a = pack_a ? up(int64_t(p.batch) * p.M * lda2, 256) : 0;
        bytes_b = pack_b ? up(int64_t(p.batch) * p.N * ldb2, 256) : 0;
        // (A grouped launch's tiles are counted on the device: any number up to these.)
        const int64_t cut = p.group_rows ? 2 * int64_t(workers) : sched.shared;
        bytes_p = cut ? 2 * int64_t(workers) * shape.slot_bytes : 0;
        bytes_w = cut * shape.parts * 8;
        return true;
    }
};

}  // namespace tsm
