"""The host checks of the expert token movement and of the 8-bit products:
every case is refused (or found empty) before any CUDA call is made, so the
addresses are never touched."""
import ctypes
import os
import re

import pytest

from tiled_staged_matmul_gb300.csrc import build as tsm_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A0, B0, C0, D0, E0 = (0x7f0000000000 + i * 0x10000000 for i in range(5))


@pytest.fixture(scope="module")
def b():
    tsm_build.build()
    from tiled_staged_matmul_gb300 import binding
    return binding


def status(b, st):
    return b.gemm_status_string(st)


def test_exports(b):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "tsm_gemm.h")).read(), flags=re.S)
    names = set(re.findall(r"\b((?:moe|quantize)_\w+|gemm_s8_\w+)\s*\(", text))
    assert names == {"moe_route_slots", "moe_dispatch_rows", "moe_dispatch_rows_grad", "moe_combine_rows",
                     "moe_combine_rows_grad", "quantize_rows_s8", "gemm_s8_scaled", "gemm_s8_grouped_scaled"}
    lib = ctypes.CDLL(b.LIB_PATH)
    assert all(hasattr(lib, n) for n in names)


@pytest.mark.parametrize("args,want", [
    ((A0, 2, B0, C0, 4, 2, 8, 4), "GEMM_ERR_INVALID_VALUE"),            # 2-byte ids
    ((A0, 4, B0, C0, -1, 2, 8, 4), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 4, B0, C0, 4, 2, 1025, 4), "GEMM_ERR_INVALID_VALUE"),         # too many groups
    ((A0, 4, B0, C0, 1 << 20, 1 << 11, 8, 4), "GEMM_ERR_INVALID_VALUE"),  # 2^31 choices
    ((A0, 4, B0, C0, 4, 2, 1024, 1 << 21), "GEMM_ERR_INVALID_VALUE"),   # 2^31 rows
    ((A0, 4, 0, C0, 4, 2, 8, 4), "GEMM_ERR_INVALID_VALUE"),             # no slots
    ((A0 + 4, 8, B0, C0, 4, 2, 8, 4), "GEMM_ERR_MISALIGNED"),
    ((A0, 4, A0 + 8, C0, 4, 2, 8, 4), "GEMM_ERR_ALIAS"),                # slots on ids
    ((A0, 4, B0, B0, 4, 2, 8, 4), "GEMM_ERR_ALIAS"),                    # counts on slots
    ((0, 4, 0, 0, 0, 2, 0, 4), "GEMM_OK"),
])
def test_route(b, args, want):
    assert status(b, b.moe_route_slots(*args)) == want


@pytest.mark.parametrize("args,want", [
    ((A0, 3, B0, C0, 4, 2, 8, 16, 16, 16), "GEMM_ERR_INVALID_VALUE"),   # 3-byte elements
    ((A0, 2, B0, C0, 4, 2, -8, 16, 16, 16), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 2, B0, C0, 4, 2, 8, 16, 15, 16), "GEMM_ERR_INVALID_VALUE"),   # pitch below the width
    ((A0, 2, B0, C0, 4, 2, 8, 16, 16, 15), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 2, 0, C0, 4, 2, 8, 16, 16, 16), "GEMM_ERR_INVALID_VALUE"),
    ((A0 + 1, 2, B0, C0, 4, 2, 8, 16, 16, 16), "GEMM_ERR_MISALIGNED"),
    ((A0, 2, B0 + 2, C0, 4, 2, 8, 16, 16, 16), "GEMM_ERR_MISALIGNED"),
    ((A0, 2, B0, A0 + 64, 4, 2, 8, 16, 16, 16), "GEMM_ERR_ALIAS"),
    ((A0, 2, B0, C0, 0, 2, 8, 16, 16, 16), "GEMM_OK"),
    ((A0, 2, B0, 0, 4, 2, 0, 16, 16, 16), "GEMM_OK"),
    ((0, 2, 0, 0, 4, 2, 8, 0, 0, 0), "GEMM_OK"),
])
def test_dispatch(b, args, want):
    assert status(b, b.moe_dispatch_rows(*args)) == want


@pytest.mark.parametrize("args,want", [
    ((A0, 5, B0, 0, C0, 4, 2, 8, 16, 16, 16), "GEMM_ERR_INVALID_VALUE"),  # unknown type
    ((A0, 1, B0, 0, 0, 4, 2, 8, 16, 16, 16), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 1, B0, D0 + 2, C0, 4, 2, 8, 16, 16, 16), "GEMM_ERR_MISALIGNED"),
    ((A0, 1, B0, D0, A0, 4, 2, 8, 16, 16, 16), "GEMM_ERR_ALIAS"),
    ((A0, 1, B0, C0, C0, 4, 2, 8, 16, 16, 16), "GEMM_ERR_ALIAS"),         # out on the weights
    ((A0, 1, B0, 0, C0, 0, 2, 8, 16, 16, 16), "GEMM_OK"),
])
def test_combine(b, args, want):
    assert status(b, b.moe_combine_rows(*args)) == want


@pytest.mark.parametrize("args,want", [
    ((A0, B0, 7, C0, D0, E0, 0, 4, 2, 8, 16, 16, 16, 16), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, 1, C0, D0, E0, 0, 4, 2, 8, 16, 16, 16, 12), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, 0, C0, D0, E0 + 2, 0, 4, 2, 8, 16, 16, 16, 16), "GEMM_ERR_MISALIGNED"),
    ((A0, B0, 1, C0, D0, B0, 0, 4, 2, 8, 16, 16, 16, 16), "GEMM_ERR_ALIAS"),
    ((A0, B0, 1, C0, D0, E0, D0, 4, 2, 8, 16, 16, 16, 16), "GEMM_ERR_ALIAS"),  # dweights on weights
    ((A0, B0, 1, C0, D0, E0, 0, 0, 2, 8, 16, 16, 16, 16), "GEMM_OK"),
])
def test_combine_grad(b, args, want):
    assert status(b, b.moe_combine_rows_grad(*args)) == want


@pytest.mark.parametrize("args,want", [
    ((A0, "f64", B0, C0, 0, 4, 16, 16, 16), "GEMM_ERR_INVALID_VALUE"),
    ((A0, "f16", B0, C0, 0, 4, 16, 15, 16), "GEMM_ERR_INVALID_VALUE"),
    ((A0, "f16", B0, C0, 0, 4, 16, 16, 15), "GEMM_ERR_INVALID_VALUE"),
    ((A0, "f16", B0, C0, 0, 4, 16, 16, 16, 64, 60, 4, 2), "GEMM_ERR_INVALID_VALUE"),  # matrices of q overlap
    ((A0, "f16", B0, C0, 0, 4, 16, 16, 16, 64, 64, 3, 2), "GEMM_ERR_INVALID_VALUE"),  # scales overlap
    ((A0 + 1, "f16", B0, C0, 0, 4, 16, 16, 16), "GEMM_ERR_MISALIGNED"),
    ((A0, "f16", A0, C0, 0, 4, 16, 16, 16), "GEMM_ERR_ALIAS"),
    ((A0, "f16", B0, 0, 0, 4, 16, 16, 16), "GEMM_ERR_INVALID_VALUE"),
    ((A0, "f16", B0, C0, 0, 0, 16, 16, 16), "GEMM_OK"),
])
def test_quantize(b, args, want):
    args = tuple(9 if a == "f64" else a for a in args)
    assert status(b, b.quantize_rows_s8(*args)) == want


@pytest.mark.parametrize("args,want", [
    ((A0, B0, C0, 0, 0, -1, 4, 4, 4, 4, 4), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, 0, 0, 4, 4, 131072, 131072, 4, 4), "GEMM_ERR_INVALID_VALUE"),  # sums past 32 bits
    ((A0, B0, C0, 0, 0, 4, 4, 8, 7, 4, 4), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, 0, 0, 4, 8, 4, 4, 7, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, 0, 0, 4, 8, 4, 4, 8, 7), "GEMM_ERR_INVALID_VALUE"),
    ((A0, 0, C0, 0, 0, 4, 8, 4, 4, 8, 8), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0 + 2, 0, 0, 4, 8, 4, 4, 8, 8), "GEMM_ERR_MISALIGNED"),
    ((A0, B0, C0, D0 + 1, 0, 4, 8, 4, 4, 8, 8), "GEMM_ERR_MISALIGNED"),
    ((A0, B0, B0, 0, 0, 4, 8, 4, 4, 8, 8), "GEMM_ERR_ALIAS"),
    ((A0, B0, C0, C0 + 16, 0, 4, 8, 4, 4, 8, 8), "GEMM_ERR_ALIAS"),     # a scale inside C
    ((A0, B0, C0, 0, 0, 4, 8, 4, 4, 8, 8, 16, 32, 16, 0, 0, 2), "GEMM_ERR_ALIAS"),  # batches of C overlap
    ((A0, B0, C0, 0, 0, 4, 8, 4, 4, 8, 8, 0, 32, 32, 0, 0, 2), "GEMM_ERR_INVALID_VALUE"),
    ((A0, B0, C0, 0, 0, 4, 8, 4, 4, 8, 8, 16, 32, 32, -1, 0, 2), "GEMM_ERR_INVALID_VALUE"),
    ((0, 0, 0, 0, 0, 0, 8, 4, 4, 8, 8), "GEMM_OK"),
    ((0, 0, 0, 0, 0, 4, 0, 4, 4, 8, 8), "GEMM_OK"),
])
def test_product(b, args, want):
    assert status(b, b.gemm_s8_scaled(*args)) == want


def test_product_epilogue_and_groups(b):
    assert status(b, b.gemm_s8_scaled(A0, B0, C0, 0, 0, 4, 8, 4, 4, 8, 8, epi=b.epilogue(activation=9))) \
        == "GEMM_ERR_INVALID_VALUE"
    assert status(b, b.gemm_s8_scaled(A0, B0, C0, 0, 0, 4, 8, 4, 4, 8, 8, epi=b.epilogue(out_type=3))) \
        == "GEMM_ERR_INVALID_VALUE"
    tail = (4, 8, 4, 4, 8, 8, 16, 32, 32, 0, 0)
    assert status(b, b.gemm_s8_grouped_scaled(A0, B0, C0, 0, 0, 0, 2, *tail)) == "GEMM_ERR_INVALID_VALUE"
    assert status(b, b.gemm_s8_grouped_scaled(A0, B0, C0, 0, 0, D0 + 1, 2, *tail)) == "GEMM_ERR_MISALIGNED"
    assert status(b, b.gemm_s8_grouped_scaled(A0, B0, C0, 0, 0, 0, 0, *tail)) == "GEMM_OK"


# Pitches and strides whose spans pass 64 bits: what wraps there would look like
# a small buffer.  The written buffer lies above, so that the true span meets it.
FAR = 1 << 62


@pytest.mark.parametrize("call,args", [
    ("moe_dispatch_rows", (A0, 2, B0, C0, 5, 2, 8, 16, FAR, 16)),
    ("moe_dispatch_rows", (B0, 2, C0, A0, 5, 2, 5, 16, 16, FAR)),
    ("moe_dispatch_rows_grad", (A0, 1, B0, C0, 5, 2, 5, 16, FAR, 16)),
    ("moe_combine_rows", (A0, 0, B0, D0, C0, 5, 2, 5, 16, FAR, 16)),
    ("moe_combine_rows", (B0, 1, C0, D0, A0, 5, 2, 8, 16, 16, FAR)),
    ("moe_combine_rows_grad", (A0, B0, 1, C0, D0, E0, 0, 5, 2, 8, 16, FAR, 16, 16)),
    ("moe_combine_rows_grad", (B0, A0, 1, C0, D0, E0, 0, 5, 2, 5, 16, 16, FAR, 16)),
    ("moe_combine_rows_grad", (B0, C0, 1, D0, E0, A0, 0, 5, 2, 5, 16, 16, 16, FAR)),
    ("quantize_rows_s8", (A0, 1, B0, C0, 0, 5, 16, FAR, 16)),
    ("quantize_rows_s8", (B0, 1, A0, C0, 0, 5, 16, 16, FAR)),
    ("quantize_rows_s8", (A0, 1, B0, C0, 0, 4, 16, 16, 16, FAR, 64, 4, 5)),
    ("quantize_rows_s8", (B0, 1, C0, A0, 0, 4, 16, 16, 16, 64, 64, FAR, 5)),
    ("gemm_s8_scaled", (A0, B0, C0, 0, 0, 5, 8, 4, FAR, 8, 8)),
    ("gemm_s8_scaled", (B0, A0, C0, 0, 0, 5, 8, 5, 5, FAR, 8)),
    ("gemm_s8_scaled", (B0, C0, A0, 0, 0, 5, 8, 4, 4, 8, FAR)),
    ("gemm_s8_scaled", (A0, B0, C0, 0, 0, 4, 8, 4, 4, 8, 8, FAR, 32, 32, 0, 0, 5)),
    ("gemm_s8_scaled", (B0, C0, D0, A0, 0, 4, 8, 4, 4, 8, 8, 16, 32, 32, FAR, 0, 5)),
    ("gemm_s8_scaled", (B0, C0, A0, 0, 0, 5, 8, 4, 4, 8, FAR, 20, 32, 32, 0, 0, 2)),
])
def test_spans_past_64_bits(b, call, args):
    assert status(b, getattr(b, call)(*args)) == "GEMM_ERR_ALIAS"
