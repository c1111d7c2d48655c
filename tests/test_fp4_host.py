"""What the choice of experts and the 4-bit operators refuse, found on the host
before any CUDA call: fake, never-dereferenced device addresses."""
import ctypes
import os
import subprocess

import pytest

from tiled_staged_matmul_gb300.csrc import build as tsm_build

A0, B0, C0, D0, E0, F0 = (0x7f0000000000 + 0x10000000 * i for i in range(6))


@pytest.fixture(scope="module")
def b():
    tsm_build.build()
    from tiled_staged_matmul_gb300 import binding
    return binding


def status(b, st):
    return b.gemm_status_string(st)


def test_exports(b):
    lib = ctypes.CDLL(b.LIB_PATH)
    for name in ("choose_experts", "choose_experts_grad", "fp4_quantize_rows", "gemm_fp4_scaled", "gemm_fp4_grouped_scaled"):
        assert hasattr(lib, name) and hasattr(b, name)


# (logits, type, bias, ids, weights, tokens, experts, topk, ld, score, groups, keep, best)
@pytest.mark.parametrize("args,want", [
    ((0, 0, 0, C0, D0, 4, 8, 2, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, 0, D0, 4, 8, 2, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, 0, 4, 8, 2, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 3, 0, C0, D0, 4, 8, 2, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, -1, 8, 2, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 1 << 31, 8, 2, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 0, 0, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 1025, 2, 1025), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 8, 9, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 64, 33, 64), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 8, -1, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 8, 2, 7), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 8, 2, 8, 2), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 8, 2, 8, 0, 0), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 8, 2, 8, 0, 3), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 66, 2, 66, 0, 33), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 516, 2, 516, 0, 3, 2), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 8, 2, 8, 0, 4, 0), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 8, 2, 8, 0, 4, 5), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 8, 2, 8, 0, 4, 2, 3), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 8, 2, 8, 0, 4, 2, 0), "GEMM_ERR_INVALID_VALUE"),
    ((A0 + 2, 0, 0, C0, D0, 4, 8, 2, 8), "GEMM_ERR_MISALIGNED"),
    ((A0 + 1, 1, 0, C0, D0, 4, 8, 2, 8), "GEMM_ERR_MISALIGNED"),
    ((A0, 0, B0 + 2, C0, D0, 4, 8, 2, 8), "GEMM_ERR_MISALIGNED"),
    ((A0, 0, 0, C0 + 1, D0, 4, 8, 2, 8), "GEMM_ERR_MISALIGNED"),
    ((A0, 0, 0, C0, C0 + 16, 4, 8, 2, 8), "GEMM_ERR_ALIAS"),
    ((A0, 0, 0, A0 + 64, D0, 4, 8, 2, 8), "GEMM_ERR_ALIAS"),
    ((A0, 0, D0 + 8, C0, D0, 4, 8, 2, 8), "GEMM_ERR_ALIAS"),
    ((A0, 0, 0, B0, C0, 5, 8, 2, 1 << 61), "GEMM_ERR_ALIAS"),
    ((0, 0, 0, 0, 0, 0, 8, 2, 8), "GEMM_OK"),
    ((0, 0, 0, 0, 0, 4, 8, 0, 8), "GEMM_OK"),
])
def test_choice(b, args, want):
    assert status(b, b.choose_experts(*args)) == want


# (dweights, logits, type, ids, dlogits, tokens, experts, topk, ld, ld_d, score)
@pytest.mark.parametrize("args,want", [
    ((0, B0, 0, C0, D0, 4, 8, 2, 8, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, 0, C0, D0, 4, 8, 2, 8, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, 0, 0, D0, 4, 8, 2, 8, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, 0, C0, 0, 4, 8, 2, 8, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, -1, C0, D0, 4, 8, 2, 8, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, 0, C0, D0, 4, 8, 2, 7, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, 0, C0, D0, 4, 8, 2, 8, 7), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, 0, C0, D0, 4, 8, 2, 8, 8, 7), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, 0, C0, D0, 4, 2000, 2, 2000, 2000), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, 0, C0, D0 + 2, 4, 8, 2, 8, 8), "GEMM_ERR_MISALIGNED"),
    ((A0 + 2, B0, 0, C0, D0, 4, 8, 2, 8, 8), "GEMM_ERR_MISALIGNED"),
    ((A0, B0, 0, C0, B0, 4, 8, 2, 8, 8), "GEMM_ERR_ALIAS"),
    ((A0, B0, 0, C0, C0 + 16, 4, 8, 2, 8, 8), "GEMM_ERR_ALIAS"),
    ((A0, B0, 0, C0, A0, 4, 8, 2, 8, 8), "GEMM_ERR_ALIAS"),
    ((B0, C0, 0, D0, A0, 5, 8, 2, 8, 1 << 61), "GEMM_ERR_ALIAS"),
    ((0, 0, 0, 0, 0, 0, 8, 2, 8, 8), "GEMM_OK"),
])
def test_choice_gradient(b, args, want):
    assert status(b, b.choose_experts_grad(*args)) == want


# (X, type, block, q, block_scales, scales, group_rows, M, K, ldx, ldq, sX, sQ, scale_stride, batch)
@pytest.mark.parametrize("args,want", [
    ((0, 1, 16, B0, C0, D0, 0, 4, 64, 64, 32), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 1, 16, 0, C0, D0, 0, 4, 64, 64, 32), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 1, 16, B0, 0, D0, 0, 4, 64, 64, 32), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 1, 16, B0, C0, 0, 0, 4, 64, 64, 32), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 5, 16, B0, C0, D0, 0, 4, 64, 64, 32), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 1, 8, B0, C0, D0, 0, 4, 64, 64, 32), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 1, 0, B0, C0, D0, 0, 4, 64, 64, 32), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 1, 16, B0, C0, D0, 0, -4, 64, 64, 32), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 1, 16, B0, C0, D0, 0, 4, 64, 63, 32), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 1, 16, B0, C0, D0, 0, 4, 65, 65, 32), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 1, 32, B0, C0, 0, 0, 1, 1 << 31, 1 << 31, 1 << 30), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 1, 32, B0, C0, 0, 0, 1 << 16, 64, 64, 32, 1 << 22, 1 << 21, 0, 1 << 15), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 1, 16, B0, C0, D0, 0, 4, 64, 64, 32, 256, 127, 4, 2), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 1, 16, B0, C0, D0, 0, 4, 64, 64, 32, 256, 128, 3, 2), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 1, 16, B0, C0, D0, 0, 4, 64, 64, 32, -1, 128, 4, 2), "GEMM_ERR_INVALID_VALUE"),
    ((A0 + 1, 1, 16, B0, C0, D0, 0, 4, 64, 64, 32), "GEMM_ERR_MISALIGNED"),
    ((A0, 1, 16, B0, C0 + 8, D0, 0, 4, 64, 64, 32), "GEMM_ERR_MISALIGNED"),
    ((A0, 1, 16, B0, C0, D0 + 2, 0, 4, 64, 64, 32), "GEMM_ERR_MISALIGNED"),
    ((A0, 1, 16, B0, C0, D0, E0 + 2, 4, 64, 64, 32), "GEMM_ERR_MISALIGNED"),
    ((A0, 1, 16, A0 + 16, C0, D0, 0, 4, 64, 64, 32), "GEMM_ERR_ALIAS"),
    ((A0, 1, 16, B0, B0 + 96, D0, 0, 4, 64, 64, 32), "GEMM_ERR_ALIAS"),
    ((A0, 1, 16, B0, C0, C0 + 496, 0, 4, 64, 64, 32), "GEMM_ERR_ALIAS"),
    ((A0, 1, 16, B0, C0, D0, D0 + 4, 4, 64, 64, 32), "GEMM_ERR_ALIAS"),
    ((A0, 1, 32, B0, C0, 0, 0, 5, 64, 1 << 62, 32), "GEMM_ERR_ALIAS"),
    ((B0, 1, 32, A0, C0, 0, 0, 5, 64, 64, 1 << 62), "GEMM_ERR_ALIAS"),
    ((0, 1, 16, 0, 0, 0, 0, 0, 64, 64, 32), "GEMM_OK"),
    ((0, 1, 32, 0, 0, 0, 0, 4, 64, 64, 32, 0, 0, 0, 0), "GEMM_OK"),
])
def test_quantisation(b, args, want):
    assert status(b, b.fp4_quantize_rows(*args)) == want


# (A, B, C, block scales of A, of B, scale_a, scale_b, block, M, N, K, lda, ldb, ldc, sA, sB, sC, ...)
@pytest.mark.parametrize("args,want", [
    ((0, B0, C0, D0, E0, 0, 0, 16, 4, 8, 64, 32, 32, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, C0, D0, E0, 0, 0, 16, 4, 8, 64, 32, 32, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, 0, D0, E0, 0, 0, 16, 4, 8, 64, 32, 32, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, 0, E0, 0, 0, 16, 4, 8, 64, 32, 32, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, D0, 0, 0, 0, 16, 4, 8, 64, 32, 32, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, D0, E0, 0, 0, 64, 4, 8, 64, 32, 32, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, D0, E0, 0, 0, 16, -4, 8, 64, 32, 32, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, D0, E0, 0, 0, 16, 4, 8, 64, 31, 32, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, D0, E0, 0, 0, 16, 4, 8, 65, 33, 32, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, D0, E0, 0, 0, 16, 4, 8, 64, 32, 32, 7), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, D0, E0, 0, 0, 16, 4, 8, (1 << 23) + 2, 1 << 23, 1 << 23, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, D0, E0, 0, 0, 16, 2**31 - 1, 8, 64, 32, 32, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, D0, E0, 0, 0, 16, 4, 8, 64, 32, 32, 8, 0, 256, 32, 0, 0, 2), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, D0, E0, 0, 0, 16, 4, 8, 64, 32, 32, 8, 128, 256, 32, -1, 0, 2), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0 + 2, D0, E0, 0, 0, 16, 4, 8, 64, 32, 32, 8), "GEMM_ERR_MISALIGNED"),
    ((A0, B0, C0, D0 + 8, E0, 0, 0, 16, 4, 8, 64, 32, 32, 8), "GEMM_ERR_MISALIGNED"),
    ((A0, B0, C0, D0, E0 + 4, 0, 0, 16, 4, 8, 64, 32, 32, 8), "GEMM_ERR_MISALIGNED"),
    ((A0, B0, C0, D0, E0, F0 + 2, 0, 16, 4, 8, 64, 32, 32, 8), "GEMM_ERR_MISALIGNED"),
    ((A0, B0, C0, D0, E0, 0, 0, 16, 4, 8, 64, 32, 32, 8, 128, 256, 31, 0, 0, 2), "GEMM_ERR_ALIAS"),
    ((A0, B0, A0 + 64, D0, E0, 0, 0, 16, 4, 8, 64, 32, 32, 8), "GEMM_ERR_ALIAS"),
    ((A0, B0, D0 + 496, D0, E0, 0, 0, 16, 4, 8, 64, 32, 32, 8), "GEMM_ERR_ALIAS"),
    ((A0, B0, C0, D0, E0, C0 + 4, 0, 16, 4, 8, 64, 32, 32, 8), "GEMM_ERR_ALIAS"),
    ((A0, B0, C0, D0, E0, 0, 0, 16, 5, 8, 64, 1 << 62, 32, 8), "GEMM_ERR_ALIAS"),
    ((B0, C0, A0, D0, E0, 0, 0, 16, 5, 8, 64, 32, 32, 1 << 62), "GEMM_ERR_ALIAS"),
    ((0, 0, 0, 0, 0, 0, 0, 16, 0, 8, 64, 32, 32, 8), "GEMM_OK"),
    ((0, 0, 0, 0, 0, 0, 0, 32, 4, 0, 64, 32, 32, 8), "GEMM_OK"),
])
def test_product(b, args, want):
    assert status(b, b.gemm_fp4_scaled(*args)) == want


def test_product_epilogue_and_groups(b):
    head = (A0, B0, C0, D0, E0, 0, 0, 16)
    assert status(b, b.gemm_fp4_scaled(*head, 4, 8, 64, 32, 32, 8, epi=b.epilogue(activation=9))) == "GEMM_ERR_INVALID_VALUE"
    assert status(b, b.gemm_fp4_scaled(*head, 4, 8, 64, 32, 32, 8, epi=b.epilogue(out_type=3))) == "GEMM_ERR_INVALID_VALUE"
    tail = (4, 8, 64, 32, 32, 8, 128, 256, 32)
    assert status(b, b.gemm_fp4_grouped_scaled(*head, 0, 2, *tail)) == "GEMM_ERR_INVALID_VALUE"
    assert status(b, b.gemm_fp4_grouped_scaled(*head, F0 + 1, 2, *tail)) == "GEMM_ERR_MISALIGNED"
    assert status(b, b.gemm_fp4_grouped_scaled(*head, 0, 0, *tail)) == "GEMM_OK"
    # Scale tiles of all matrices are counted in 32 bits.
    assert status(b, b.gemm_fp4_grouped_scaled(*head, F0, 1 << 24, 1 << 15, 8, 64, 32, 32, 8, 1 << 20, 256, 1 << 18)) \
        == "GEMM_ERR_INVALID_VALUE"


def test_python_arguments(b):
    """What the torch calls find before they reach the library."""
    import torch
    x = torch.zeros((4, 64))
    with pytest.raises(ValueError):
        b.quantize_fp4(x)  # not on a GPU
    with pytest.raises(ValueError):
        b.quantize_fp4(x, block=8)
    with pytest.raises(TypeError):
        b.quantize_fp4(x.int())
    with pytest.raises(TypeError):
        b.moe_choose(x.int(), 2)
    with pytest.raises(ValueError):
        b.moe_choose(x, 2)
    with pytest.raises(ValueError):
        b.moe_choose_grad(torch.zeros((4, 2)), x, torch.zeros((4, 2), dtype=torch.int32))
    u = torch.zeros((4, 32), dtype=torch.uint8)
    tiles = torch.zeros((1, 1, 512), dtype=torch.uint8)
    with pytest.raises(TypeError):
        b.gemm_fp4(b.Fp4Rows(u.int(), tiles, None, 16), b.Fp4Rows(u, tiles, None, 16))
    with pytest.raises(ValueError):
        b.gemm_fp4(b.Fp4Rows(u, tiles, None, 24), b.Fp4Rows(u, tiles, None, 24))
    with pytest.raises(ValueError):
        b.gemm_fp4(b.Fp4Rows(u, tiles, None, 16), b.Fp4Rows(u, tiles, None, 16))


PROGRAM = r"""
#include "fp4_plan.h"
#include <cstdio>

using namespace tsm;

int main()
{
    Fp4Capacity cap;
    for (auto &kind : cap.clusters)
        for (int i = 0; i < Fp4Capacity::RANKS; ++i)
            kind[i] = 152 / (i + 1);
    long long M, N, K, batch, lda, ldb, a, b, grouped;
    while (std::scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld", &M, &N, &K, &batch, &lda, &ldb, &a, &b, &grouped) == 9) {
        static const int32_t counts[1] = {0};
        Fp4Params p = {};
        p.M = int32_t(M);
        p.N = int32_t(N);
        p.K = int32_t(K);
        p.batch = int32_t(batch);
        p.group_rows = grouped ? counts : nullptr;
        Fp4Plan s;
        const bool ok = s.make(p, reinterpret_cast<const uint8_t *>(a), lda, M * lda, reinterpret_cast<const uint8_t *>(b), ldb,
                               N * ldb, 152, cap);
        // Every worker's piece lies in at most two tiles of its own to sum, and
        // the pieces together are the cut tiles.
        bool sound = true;
        const int64_t blocks = int64_t(s.sched.shared) * s.kb;
        if (s.sched.shared) {
            sound = s.sched.piece_begin(0) == 0 && s.sched.piece_begin(s.sched.cutters) == blocks;
            for (int w = 0; w < s.sched.cutters; ++w) {
                const int32_t begin = s.sched.piece_begin(w), end = s.sched.piece_begin(w + 1);
                sound = sound && begin < end && end - begin < 2 * s.kb && s.sched.owner(begin) == w && s.sched.owner(end - 1) == w;
            }
        }
        std::printf("%d %d %d %d %d %d %d %d %d %lld %lld %lld %lld %d\n", int(ok), int(s.kind), s.tiles_m, s.tiles_n, s.kb, s.ranks, s.grid,
                    int(s.sched.shared), int(s.sched.cutters), (long long)s.bytes_a, (long long)s.bytes_b, (long long)s.bytes_p,
                    (long long)s.bytes_w, int(sound));
    }
    return 0;
}
"""
FIELDS = ("ok", "kind", "tiles_m", "tiles_n", "kb", "ranks", "grid", "shared", "cutters", "bytes_a", "bytes_b", "bytes_p", "bytes_w",
          "sound")


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    where = tmp_path_factory.mktemp("fp4_plan")
    src, exe = str(where / "plan.cu"), str(where / "plan")
    with open(src, "w") as f:
        f.write(PROGRAM)
    here = os.path.dirname(os.path.abspath(tsm_build.__file__))
    subprocess.run([tsm_build._nvcc(), "-std=c++17", "-I", here, "-o", exe, src], check=True)

    def ask(problems):
        lines = "\n".join(" ".join(map(str, p)) for p in problems)
        out = subprocess.run([exe], input=lines, capture_output=True, text=True, check=True).stdout
        return [dict(zip(FIELDS, map(int, line.split()))) for line in out.splitlines()]

    return ask


def test_plans_are_sound(plans):
    """Over all kinds of sizes: the schedule covers the work, the workspace holds
    every worker's two slots, and copies are made where they are needed only."""
    slot = (16384, 32768, 65536, 262144)
    parts = (4, 4, 4, 8)
    sizes = [(M, N, K) for M in (1, 16, 32, 33, 64, 65, 128, 129, 1000, 8191) for N in (1, 128, 1000, 14336)
             for K in (1, 256, 4010, 16384, 1 << 23)]
    for grouped in (0, 1):
        problems = [(M, N, K, bt, 1 << 23, 1 << 23, A0, B0, grouped) for M, N, K in sizes for bt in (1, 3)]
        for p, s in zip(problems, plans(problems)):
            assert s["ok"] and s["sound"], (p, s)
            assert s["bytes_a"] == 0 and s["bytes_b"] == 0
            k = s["kind"]
            workers = 76 if k == 3 else 152
            assert s["grid"] * s["ranks"] <= workers
            assert s["ranks"] == 1 or (s["shared"] == 0 and s["grid"] == s["tiles_m"] * s["tiles_n"] * p[3]
                                       and s["kb"] >= 2 * s["ranks"] and k < 3 and not grouped)
            if grouped:
                assert s["grid"] == workers and s["bytes_p"] == 2 * workers * slot[k]
            if s["shared"] or grouped:
                assert s["bytes_p"] == 2 * workers * slot[k]
                assert s["bytes_w"] == (2 * workers if grouped else s["shared"]) * parts[k] * 8
                assert s["shared"] < 2 * workers and s["cutters"] <= workers
            else:
                assert s["bytes_p"] == 0


def test_copies(plans):
    for lda, ldb, a, b_, pa, pb in ((32, 32, A0, B0, 0, 0), (40, 32, A0, B0, 1, 0), (32, 33, A0, B0, 0, 1),
                                    (32, 32, A0 + 8, B0 + 1, 1, 1)):
        s = plans([(5, 7, 64, 2, lda, ldb, a, b_, 0)])[0]
        assert s["bytes_a"] == (512 if pa else 0) and s["bytes_b"] == (512 if pb else 0)


def test_too_many_tiles(plans):
    assert not plans([(2**31 - 600, 2**31 - 600, 64, 1, 32, 32, A0, B0, 0)])[0]["ok"]


def test_tiles_are_cut_where_it_pays(plans):
    """The sizes with which the GPU tests reach each way of cutting a tile's K: over
    a cluster, or over the workers, for every kind of kernel."""
    from test_fp4_cut_gpu import CUT
    for (M, N, K), (kind, ranks, cut) in CUT.items():
        s = plans([(M, N, K, 1, 1 << 23, 1 << 23, A0, B0, 0)])[0]
        assert s["kind"] == kind and (s["ranks"] > 1) == (ranks > 1) and (s["shared"] > 0) == cut, (M, N, K, s)
