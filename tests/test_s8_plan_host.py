"""How the 8-bit products are launched (csrc/s8_plan.h): host arithmetic,
compiled by itself into a small program and asked here, so nothing is allocated
or launched."""
import os
import subprocess

import pytest

from tiled_staged_matmul_gb300.csrc import build as tsm_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMS = 152

PROGRAM = r"""
#include "s8_plan.h"
#include <cstdio>

using namespace tsm;

int main()
{
    // The most clusters of 1 to 8 CTAs that 152 SMs hold.
    S8Capacity cap;
    for (int i = 0; i < S8Capacity::KINDS; ++i)
        cap.clusters[i] = 152 / (i + 1);
    long long M, N, K, batch, lda, ldb, sA, sB, a, b, grouped;
    while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", &M, &N, &K, &batch, &lda, &ldb, &sA, &sB,
                      &a, &b, &grouped) == 11) {
        static const int32_t counts[1] = {0};
        S8Params p = {};
        p.A = reinterpret_cast<const int8_t *>(a);
        p.B = reinterpret_cast<const int8_t *>(b);
        p.M = int32_t(M);
        p.N = int32_t(N);
        p.K = int32_t(K);
        p.batch = int32_t(batch);
        p.lda = lda;
        p.ldb = ldb;
        p.sA = sA;
        p.sB = sB;
        p.group_rows = grouped ? counts : nullptr;
        S8Plan s;
        const bool ok = s.make(p, 152, cap);
        std::printf("%d %d %d %d %d %d %d %d %d %lld %lld %lld %lld\n", int(ok), int(s.kind), s.tiles_m, s.tiles_n, s.kb,
                    s.ranks, s.grid, int(s.sched.shared), int(s.sched.cutters), (long long)s.bytes_a,
                    (long long)s.bytes_b, (long long)s.bytes_p, (long long)s.bytes_w);
    }
    return 0;
}
"""
FIELDS = ("ok", "kind", "tiles_m", "tiles_n", "kb", "ranks", "grid", "shared", "cutters", "bytes_a", "bytes_b",
          "bytes_p", "bytes_w")
KINDS = ("few16", "few32", "one", "pair")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """Plans of a list of problems, one dict each."""
    where = tmp_path_factory.mktemp("s8_plan")
    src, exe = str(where / "plan.cu"), str(where / "plan")
    with open(src, "w") as f:
        f.write(PROGRAM)
    subprocess.run([tsm_build._nvcc(), "-std=c++17", *tsm_build.ARCH, "-I", tsm_build.HERE, "-o", exe, src], check=True,
                   capture_output=True, text=True)

    def ask(problems):
        lines = []
        for q in problems:
            M, N, K, batch = q["M"], q["N"], q["K"], q.get("batch", 1)
            lda, ldb = q.get("lda", up(K, 16)), q.get("ldb", up(N, 16))
            lines.append(" ".join(map(str, (M, N, K, batch, lda, ldb, q.get("sA", M * lda if batch > 1 else 0),
                                            q.get("sB", K * ldb if batch > 1 else 0), q.get("a", 1 << 32),
                                            q.get("b", 1 << 33), int(q.get("grouped", False))))))
        out = subprocess.run([exe], input="\n".join(lines), check=True, capture_output=True, text=True).stdout
        answers = [dict(zip(FIELDS, map(int, line.split()))) for line in out.splitlines()]
        assert len(answers) == len(problems)
        for a in answers:
            a["kind"] = KINDS[a["kind"]]
        return answers

    return ask


def up(n, m):
    return -(-n // m) * m


# Row counts whose product with the batch passes 31 and 32 bits.
@pytest.mark.parametrize("batch,M,N,K", [(65536, 32768, 16, 8), (65536, 65536, 8, 24), (1 << 17, 1 << 15, 1, 1),
                                         (1 << 20, 4096, 3, 40), (1 << 28, 32, 1, 3), (3, 1 << 30, 1, 5)])
def test_packed_copies_have_room_for_every_row(plans, batch, M, N, K):
    a, = plans([{"M": M, "N": N, "K": K, "batch": batch, "lda": K + 1 - K % 2, "ldb": N + 1 - N % 2, "b": (1 << 33) + 1}])
    assert a["ok"]
    assert a["bytes_a"] == up(batch * M * up(K, 16), 256)
    assert a["bytes_b"] == up(batch * K * up(N, 16), 256)
    if batch * M * up(K, 16) >= 1 << 32:
        assert a["bytes_a"] >= 1 << 32


def test_nothing_is_copied_that_can_be_read_in_place(plans):
    for q, copies in (({"M": 40, "N": 48, "K": 32}, (0, 0)), ({"M": 40, "N": 48, "K": 31, "lda": 31}, (1, 0)),
                      ({"M": 40, "N": 47, "K": 32, "ldb": 47}, (0, 1)), ({"M": 40, "N": 48, "K": 32, "a": 8}, (1, 0)),
                      ({"M": 1, "N": 48, "K": 31, "lda": 31}, (0, 0)), ({"M": 40, "N": 47, "K": 1, "ldb": 47}, (0, 0)),
                      ({"M": 40, "N": 48, "K": 32, "batch": 2, "sA": 40 * 32 + 8}, (1, 0))):
        a, = plans([q])
        assert (a["bytes_a"] > 0, a["bytes_b"] > 0) == tuple(map(bool, copies)), q


def test_too_many_tiles_are_refused(plans):
    most, past = plans([{"M": 256, "N": 256, "K": 16, "batch": 1 << 30}, {"M": 256, "N": 257, "K": 16, "batch": 1 << 30}])
    assert most["ok"] and not past["ok"]


# What the GPU tests of the products take for granted.
def test_the_tests_reach_every_kernel(plans):
    by_size = [((1, 300, 500), "few16"), ((16, 256, 2048), "few16"), ((20, 77, 96), "few32"), ((32, 144, 5000), "few32"),
               ((33, 40, 333), "one"), ((70, 260, 1100), "one"), ((180, 516, 2100), "one"), ((513, 65, 4097), "one"),
               ((1500, 2100, 1200), "pair"), ((1537, 2049, 1025), "pair"), ((900, 3000, 2000), "pair"),
               ((4000, 4100, 130), "pair"), ((1300, 2500, 700), "pair"), ((300, 5008, 8192), "pair")]
    for (size, want), a in zip(by_size, plans([dict(zip("MNK", s)) for s, _ in by_size])):
        assert a["kind"] == want, size
    small, large = plans([{"M": 32, "N": 130, "K": 257, "batch": 6, "grouped": True},
                          {"M": 300, "N": 1024, "K": 520, "batch": 40, "grouped": True}])
    assert small["kind"] == "few16" and small["tiles_m"] == 2 and large["kind"] == "pair"


def test_schedules_hold_together(plans):
    """Grids within the device, cuts only where more than one worker shares a
    tile, and room for two sets of sums a worker."""
    problems = [{"M": M, "N": N, "K": K} for M in (1, 16, 17, 32, 33, 129, 700, 4097) for N in (1, 300, 5000, 60000)
                for K in (1, 128, 1030, 16384, 131071)]
    for q, a in zip(problems, plans(problems)):
        slots = {"one": SMS * 2 * 65536, "pair": SMS // 2 * 2 * 262144}.get(a["kind"], 0)
        assert a["ok"] and 1 <= a["ranks"] <= 8 and a["grid"] >= 1, q
        if a["kind"].startswith("few"):
            assert a["grid"] * a["ranks"] <= SMS and a["ranks"] <= a["kb"], q
            assert a["bytes_p"] == a["bytes_w"] == 0, q
        else:
            workers = SMS // 2 if a["kind"] == "pair" else SMS
            assert a["grid"] <= workers and a["cutters"] <= workers and a["shared"] < 2 * workers, q
            assert a["bytes_p"] == (slots if a["shared"] else 0), q
            assert a["bytes_w"] == a["shared"] * (8 if a["kind"] == "pair" else 4) * 8, q
