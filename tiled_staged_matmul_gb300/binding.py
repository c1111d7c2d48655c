"""ctypes binding of the C ABI in ``include/tsm_gemm.h``.

Argument marshalling only: every step of the GEMM runs in ``libtsm_gemm.so``.
Importing this module loads the library and raises ``ImportError`` when it
has not been built -- there is no fallback path.

The raw functions keep the C names (``gemm_f16_f32acc`` ...) and take device
pointers as integers.  ``gemm`` and ``gemm_host`` are conveniences over torch
tensors: torch only provides the memory and the stream.
"""
from __future__ import annotations

import ctypes
import os

from .csrc import build as _build

LIB_PATH = _build.LIB_PATH

GEMM_OK = 0
GEMM_ERR_INVALID_VALUE = 1
GEMM_ERR_MISALIGNED = 2
GEMM_ERR_ALIAS = 3
GEMM_ERR_UNSUPPORTED_DEVICE = 4
GEMM_ERR_CUDA = 5
GEMM_ERR_DEVICE_TIMEOUT = 6


class GemmOptions(ctypes.Structure):
    _fields_ = [("split_k", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("timeout_ms", ctypes.c_int32), ("inject_stall", ctypes.c_int32),
                ("tile_m", ctypes.c_int32), ("splitk_reduce", ctypes.c_int32),
                ("l2_prefetch", ctypes.c_int32), ("split_tail", ctypes.c_int32),
                ("trace", ctypes.c_void_p), ("red_cluster", ctypes.c_int32)]


ACTIVATIONS = {"none": 0, "relu": 1, "leaky_relu": 2, "gelu": 3, "gelu_tanh": 4, "silu": 5}
OUT_TYPES = {"f32": 0, "f16": 1, "bf16": 2}


class GemmEpilogue(ctypes.Structure):
    _fields_ = [("alpha", ctypes.c_float), ("bias", ctypes.c_void_p),
                ("bias_stride", ctypes.c_int64), ("activation", ctypes.c_int32),
                ("slope", ctypes.c_float), ("out_type", ctypes.c_int32)]


def epilogue(alpha=1.0, bias=0, bias_stride=0, activation="none", slope=0.01, out_type="f32"):
    """A ``GemmEpilogue``: ``activation`` and ``out_type`` by name or number,
    ``bias`` a device pointer (0 = none)."""
    act = ACTIVATIONS.get(activation, activation)
    out = OUT_TYPES.get(out_type, out_type)
    return GemmEpilogue(float(alpha), int(bias) or None, int(bias_stride), int(act), float(slope),
                        int(out))


class GemmPlanInfo(ctypes.Structure):
    _fields_ = [("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32),
                ("tile_k", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("split_k", ctypes.c_int32), ("tiles_m", ctypes.c_int32),
                ("tiles_n", ctypes.c_int32), ("k_blocks", ctypes.c_int32),
                ("units", ctypes.c_int64), ("grid", ctypes.c_int32),
                ("group_m", ctypes.c_int32), ("stage_bytes", ctypes.c_int64),
                ("smem_bytes", ctypes.c_int64), ("workspace_bytes", ctypes.c_int64),
                ("fused_reduce", ctypes.c_int32), ("tail_tiles", ctypes.c_int32),
                ("tail_split", ctypes.c_int32), ("tail_narrow", ctypes.c_int32),
                ("red_cluster", ctypes.c_int32)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class GemmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{gemm_status_string(status)}: {message}")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build the CUDA library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(LIB_PATH)
    i64, i32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
    lib.gemm_f16_f32acc.restype = ctypes.c_int
    lib.gemm_f16_f32acc.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i64, vp]
    lib.gemm_f16_f32acc_batched.restype = ctypes.c_int
    lib.gemm_f16_f32acc_batched.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i64,
                                            i64, i64, i64, i64, vp]
    lib.gemm_f16_f32acc_opts.restype = ctypes.c_int
    lib.gemm_f16_f32acc_opts.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i64,
                                         i64, i64, i64, i64, ctypes.POINTER(GemmOptions), vp]
    lib.gemm_plan.restype = ctypes.c_int
    lib.gemm_plan.argtypes = [i64, i64, i64, i64, ctypes.POINTER(GemmOptions), i32,
                              ctypes.POINTER(GemmPlanInfo)]
    lib.gemm_plan_grouped.restype = ctypes.c_int
    lib.gemm_plan_grouped.argtypes = [i64, i64, i64, i64, ctypes.POINTER(GemmOptions), i32,
                                      ctypes.POINTER(GemmPlanInfo)]
    lib.gemm_get_device_status.restype = ctypes.c_int
    lib.gemm_get_device_status.argtypes = [vp]
    lib.gemm_last_error_string.restype = ctypes.c_char_p
    lib.gemm_last_error_string.argtypes = []
    lib.gemm_status_string.restype = ctypes.c_char_p
    lib.gemm_status_string.argtypes = [ctypes.c_int]
    lib.gemm_version.restype = ctypes.c_int32
    lib.gemm_version.argtypes = []
    lib.gemm_f16_f32acc_grouped.restype = ctypes.c_int
    lib.gemm_f16_f32acc_grouped.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64,
                                            i64, i64, i64, vp]
    lib.gemm_f16_f32acc_grouped_opts.restype = ctypes.c_int
    lib.gemm_f16_f32acc_grouped_opts.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, i64,
                                                 i64, i64, i64, i64, ctypes.POINTER(GemmOptions),
                                                 vp]
    lib.gemm_f16_fused.restype = ctypes.c_int
    lib.gemm_f16_fused.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, i64, i64, i64,
                                   ctypes.POINTER(GemmEpilogue), ctypes.POINTER(GemmOptions), vp]
    lib.gemm_f16_grouped_fused.restype = ctypes.c_int
    lib.gemm_f16_grouped_fused.argtypes = [vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, i64,
                                           i64, i64, ctypes.POINTER(GemmEpilogue),
                                           ctypes.POINTER(GemmOptions), vp]
    lib.rowsum_f32acc.restype = ctypes.c_int
    lib.rowsum_f32acc.argtypes = [vp, i32, vp, i64, i64, i64, i64, vp]
    lib.gemv_f16_f32acc.restype = ctypes.c_int
    lib.gemv_f16_f32acc.argtypes = [vp, vp, vp, i64, i64, i64, i64, vp]
    lib.moe_route_slots.restype = ctypes.c_int
    lib.moe_route_slots.argtypes = [vp, i32, vp, vp, i64, i64, i64, i64, vp]
    lib.moe_dispatch_rows.restype = ctypes.c_int
    lib.moe_dispatch_rows.argtypes = [vp, i32, vp, vp, i64, i64, i64, i64, i64, i64, vp]
    lib.moe_dispatch_rows_grad.restype = ctypes.c_int
    lib.moe_dispatch_rows_grad.argtypes = [vp, i32, vp, vp, i64, i64, i64, i64, i64, i64, vp]
    lib.moe_combine_rows.restype = ctypes.c_int
    lib.moe_combine_rows.argtypes = [vp, i32, vp, vp, vp, i64, i64, i64, i64, i64, i64, vp]
    lib.moe_combine_rows_grad.restype = ctypes.c_int
    lib.moe_combine_rows_grad.argtypes = [vp, vp, i32, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, vp]
    lib.quantize_rows_s8.restype = ctypes.c_int
    lib.quantize_rows_s8.argtypes = [vp, i32, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, i64, vp]
    lib.gemm_s8_scaled.restype = ctypes.c_int
    lib.gemm_s8_scaled.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, i64, i64, i64,
                                   i64, i64, ctypes.POINTER(GemmEpilogue), vp]
    lib.gemm_s8_grouped_scaled.restype = ctypes.c_int
    lib.gemm_s8_grouped_scaled.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i64, i64, i64, i64,
                                           i64, i64, i64, i64, ctypes.POINTER(GemmEpilogue), vp]
    lib.gemm_f16_f32acc_splitk_noalloc.restype = ctypes.c_int
    lib.gemm_f16_f32acc_splitk_noalloc.argtypes = [vp, vp, vp, i64, i64, i64, i64, i64, i64,
                                                   i32, vp]
    return lib


_lib = _load()


def _opts(split_k=0, tile_n=0, timeout_ms=0, inject_stall=0, tile_m=0, splitk_reduce=0):
    return GemmOptions(int(split_k), int(tile_n), int(timeout_ms), int(inject_stall), int(tile_m),
                       int(splitk_reduce))


# ------------------------------------------------------------------ raw C names

def gemm_f16_f32acc(A, B, C, M, N, K, lda, ldb, ldc, stream=0) -> int:
    return _lib.gemm_f16_f32acc(A, B, C, M, N, K, lda, ldb, ldc, stream)


def gemm_f16_f32acc_batched(A, B, C, M, N, K, lda, ldb, ldc, strideA, strideB, strideC,
                            batch, stream=0) -> int:
    return _lib.gemm_f16_f32acc_batched(A, B, C, M, N, K, lda, ldb, ldc, strideA, strideB,
                                        strideC, batch, stream)


def gemm_f16_f32acc_opts(A, B, C, M, N, K, lda, ldb, ldc, strideA, strideB, strideC, batch,
                         opts: GemmOptions | None = None, stream=0) -> int:
    p = ctypes.byref(opts) if opts is not None else None
    return _lib.gemm_f16_f32acc_opts(A, B, C, M, N, K, lda, ldb, ldc, strideA, strideB,
                                     strideC, batch, p, stream)


def gemm_f16_f32acc_grouped(A, B, C, group_rows, groups, M, N, K, lda, ldb, ldc, strideA,
                            strideB, strideC, stream=0) -> int:
    return _lib.gemm_f16_f32acc_grouped(A, B, C, group_rows, groups, M, N, K, lda, ldb, ldc,
                                        strideA, strideB, strideC, stream)


def gemm_f16_f32acc_grouped_opts(A, B, C, group_rows, groups, M, N, K, lda, ldb, ldc, strideA,
                                 strideB, strideC, opts: GemmOptions | None = None,
                                 stream=0) -> int:
    p = ctypes.byref(opts) if opts is not None else None
    return _lib.gemm_f16_f32acc_grouped_opts(A, B, C, group_rows, groups, M, N, K, lda, ldb, ldc,
                                             strideA, strideB, strideC, p, stream)


def gemm_f16_fused(A, B, C, M, N, K, lda, ldb, ldc, strideA, strideB, strideC, batch,
                   epi: GemmEpilogue | None = None, opts: GemmOptions | None = None,
                   stream=0) -> int:
    e = ctypes.byref(epi) if epi is not None else None
    o = ctypes.byref(opts) if opts is not None else None
    return _lib.gemm_f16_fused(A, B, C, M, N, K, lda, ldb, ldc, strideA, strideB, strideC, batch,
                               e, o, stream)


def gemm_f16_grouped_fused(A, B, C, group_rows, groups, M, N, K, lda, ldb, ldc, strideA, strideB,
                           strideC, epi: GemmEpilogue | None = None,
                           opts: GemmOptions | None = None, stream=0) -> int:
    e = ctypes.byref(epi) if epi is not None else None
    o = ctypes.byref(opts) if opts is not None else None
    return _lib.gemm_f16_grouped_fused(A, B, C, group_rows, groups, M, N, K, lda, ldb, ldc, strideA,
                                       strideB, strideC, e, o, stream)


def rowsum_f32acc(X, elem_type, out, R, C, row_stride, col_stride, stream=0) -> int:
    return _lib.rowsum_f32acc(X, OUT_TYPES.get(elem_type, elem_type), out, R, C, row_stride,
                              col_stride, stream)


def gemv_f16_f32acc(A, x, y, M, K, lda, incx=1, stream=0) -> int:
    return _lib.gemv_f16_f32acc(A, x, y, M, K, lda, incx, stream)


def gemm_f16_f32acc_splitk_noalloc(A, B, C, M, N, K, lda, ldb, ldc, split_k=0, stream=0) -> int:
    """The entry point that allocates nothing (split-K partials in a fixed
    16 MiB device array inside the library); see include/tsm_gemm.h."""
    return _lib.gemm_f16_f32acc_splitk_noalloc(A, B, C, M, N, K, lda, ldb, ldc, split_k, stream)


def moe_route_slots(expert_ids, id_bytes, slots, counts, tokens, topk, groups, capacity, stream=0) -> int:
    return _lib.moe_route_slots(expert_ids, id_bytes, slots, counts, tokens, topk, groups, capacity, stream)


def moe_dispatch_rows(x, elem_bytes, slots, rows_out, tokens, topk, rows, width, ldx, ld_rows, stream=0) -> int:
    return _lib.moe_dispatch_rows(x, elem_bytes, slots, rows_out, tokens, topk, rows, width, ldx, ld_rows, stream)


def moe_dispatch_rows_grad(drows, elem_type, slots, dx, tokens, topk, rows, width, ld_rows, ldx, stream=0) -> int:
    return _lib.moe_dispatch_rows_grad(drows, elem_type, slots, dx, tokens, topk, rows, width, ld_rows, ldx, stream)


def moe_combine_rows(rows_in, elem_type, slots, weights, out, tokens, topk, rows, width, ld_rows, ld_out,
                    stream=0) -> int:
    return _lib.moe_combine_rows(rows_in, elem_type, slots, weights, out, tokens, topk, rows, width, ld_rows, ld_out,
                            stream)


def moe_combine_rows_grad(dout, rows_in, elem_type, slots, weights, drows, dweights, tokens, topk, rows, width,
                         ld_dout, ld_rows, ld_drows, stream=0) -> int:
    return _lib.moe_combine_rows_grad(dout, rows_in, elem_type, slots, weights, drows, dweights, tokens, topk, rows,
                                 width, ld_dout, ld_rows, ld_drows, stream)


def quantize_rows_s8(X, elem_type, q, scales, group_rows, M, K, ldx, ldq, strideX=0, strideQ=0, scale_stride=0,
                     batch=1, stream=0) -> int:
    return _lib.quantize_rows_s8(X, OUT_TYPES.get(elem_type, elem_type), q, scales, group_rows, M, K, ldx, ldq,
                                 strideX, strideQ, scale_stride, batch, stream)


def gemm_s8_scaled(A, B, C, scale_a, scale_b, M, N, K, lda, ldb, ldc, strideA=0, strideB=0, strideC=0,
                   scale_a_stride=0, scale_b_stride=0, batch=1, epi: GemmEpilogue | None = None,
                   stream=0) -> int:
    e = ctypes.byref(epi) if epi is not None else None
    return _lib.gemm_s8_scaled(A, B, C, scale_a, scale_b, M, N, K, lda, ldb, ldc, strideA, strideB, strideC,
                               scale_a_stride, scale_b_stride, batch, e, stream)


def gemm_s8_grouped_scaled(A, B, C, scale_a, scale_b, group_rows, groups, M, N, K, lda, ldb, ldc, strideA,
                           strideB, strideC, scale_a_stride, scale_b_stride, epi: GemmEpilogue | None = None,
                           stream=0) -> int:
    e = ctypes.byref(epi) if epi is not None else None
    return _lib.gemm_s8_grouped_scaled(A, B, C, scale_a, scale_b, group_rows, groups, M, N, K, lda, ldb, ldc,
                                       strideA, strideB, strideC, scale_a_stride, scale_b_stride, e, stream)


def gemm_plan(M, N, K, batch=1, opts: GemmOptions | None = None, num_sms=0) -> dict:
    info = GemmPlanInfo()
    p = ctypes.byref(opts) if opts is not None else None
    st = _lib.gemm_plan(M, N, K, batch, p, num_sms, ctypes.byref(info))
    if st != GEMM_OK:
        raise GemmError(st, gemm_last_error_string())
    return info.as_dict()


def gemm_plan_grouped(M, N, K, groups=1, opts: GemmOptions | None = None, num_sms=0) -> dict:
    info = GemmPlanInfo()
    p = ctypes.byref(opts) if opts is not None else None
    st = _lib.gemm_plan_grouped(M, N, K, groups, p, num_sms, ctypes.byref(info))
    if st != GEMM_OK:
        raise GemmError(st, gemm_last_error_string())
    return info.as_dict()


def gemm_get_device_status(stream=0) -> int:
    return _lib.gemm_get_device_status(stream)


def gemm_last_error_string() -> str:
    return _lib.gemm_last_error_string().decode()


def gemm_status_string(status: int) -> str:
    return _lib.gemm_status_string(int(status)).decode()


def gemm_version() -> int:
    return _lib.gemm_version()


def check(status: int) -> None:
    if status != GEMM_OK:
        raise GemmError(status, gemm_last_error_string())


# ------------------------------------------------------------------ torch conveniences

def _stream_handle(stream):
    if stream is None:
        # (torch.cuda.current_stream() builds a Stream object, ten times as long)
        import torch
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _on_stream(stream, call, *args, **kwargs):
    """``call`` with ``stream`` (a torch stream or a handle) as torch's current
    one.  What a call allocates, fills or copies in torch goes to the current
    stream, with nothing that orders it with kernels on another: results could
    be filled over, or lie in memory that the current stream still works on.
    The tensors it returns belong to ``stream``."""
    import torch
    handle = _stream_handle(stream)
    if handle == _stream_handle(None):
        return call(*args, **kwargs)
    if isinstance(stream, int):
        # (0 and 1 both name the default stream.)
        stream = torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return call(*args, **kwargs)


def gemm(A, B, out=None, *, alpha=1.0, bias=None, activation="none", slope=0.01, out_dtype=None,
         split_k=0, tile_n=0, tile_m=0, timeout_ms=0, inject_stall=0, stream=None):
    """``out = activation(alpha * (A @ B) + bias)`` for f16 CUDA tensors A
    (M x K) and B (K x N); ``out`` is f32 unless ``out_dtype`` (or the given
    ``out``) says torch.float16 / torch.bfloat16.

    3-D tensors (batch x M x K, batch x K x N) run as one batched call;
    ``bias`` is an f32 CUDA tensor of N values (or batch x N).  Rows may be
    padded (``stride(-2) >= size(-1)``) but the last stride must be 1.
    Returns ``out`` (allocated with ``torch.empty`` when not given)."""
    import torch
    if out is None and stream is not None:
        return _on_stream(stream, gemm, A, B, alpha=alpha, bias=bias, activation=activation, slope=slope,
                          out_dtype=out_dtype, split_k=split_k, tile_n=tile_n, tile_m=tile_m,
                          timeout_ms=timeout_ms, inject_stall=inject_stall)
    if A.dtype != torch.float16 or B.dtype != torch.float16:
        raise TypeError("A and B must be torch.float16")
    batched = A.dim() == 3
    if A.dim() != B.dim() or A.dim() not in (2, 3):
        raise ValueError("A and B must both be 2-D or both 3-D")
    M, K = A.shape[-2], A.shape[-1]
    K2, N = B.shape[-2], B.shape[-1]
    if K != K2:
        raise ValueError(f"inner sizes differ: {K} vs {K2}")
    batch = A.shape[0] if batched else 1
    if batched and B.shape[0] != batch:
        raise ValueError("batch sizes differ")
    dtype = out.dtype if out is not None else (out_dtype or torch.float32)
    out_names = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
    if dtype not in out_names:
        raise TypeError("out must be torch.float32, torch.float16 or torch.bfloat16")
    if out is None:
        # rows padded to a 16-byte pitch (the TMA's rule); the view hides it
        per16 = 16 // torch.tensor([], dtype=dtype).element_size()
        ldc_alloc = max(per16, -(-N // per16) * per16)
        shape = (batch, M, ldc_alloc) if batched else (M, ldc_alloc)
        out = torch.empty(shape, dtype=dtype, device=A.device)[..., :N]
    for t, name in ((A, "A"), (B, "B"), (out, "out")):
        if t.numel() and t.stride(-1) != 1:
            raise ValueError(f"{name} must have a unit last stride")
    # Any row pitch works; pitches that are not multiples of 16 bytes (and
    # unaligned bases) cost the library a repacking copy.
    lda = A.stride(-2) if M > 1 else max(K, 1)
    ldb = B.stride(-2) if K > 1 else max(N, 1)
    ldc = out.stride(-2) if M > 1 else max(N, 1)
    sA = A.stride(0) if batched else 0
    sB = B.stride(0) if batched else 0
    sC = out.stride(0) if batched else 0
    opts = _opts(split_k, tile_n, timeout_ms, inject_stall, tile_m)
    if bias is not None:
        if bias.dtype != torch.float32 or not bias.is_cuda or bias.shape[-1] != N:
            raise ValueError("bias must be a CUDA float32 tensor of N values (or batch x N)")
        if bias.stride(-1) != 1:
            raise ValueError("bias must have a unit last stride")
    epi = epilogue(alpha, bias.data_ptr() if bias is not None else 0,
                   bias.stride(0) if bias is not None and bias.dim() == 2 else 0,
                   activation, slope, out_names[dtype])
    st = gemm_f16_fused(A.data_ptr(), B.data_ptr(), out.data_ptr(), M, N, K, lda, ldb, ldc, sA, sB,
                        sC, batch, epi, opts, _stream_handle(stream))
    check(st)
    return out


def grouped_gemm(A, B, group_rows, out=None, *, alpha=1.0, bias=None, activation="none",
                 slope=0.01, out_dtype=None, tile_n=0, tile_m=0, stream=None):
    """Grouped (Mixture-of-Experts) GEMM on CUDA tensors: for each group g,
    ``out[g, :group_rows[g]] = A[g, :group_rows[g]] @ B[g]``.

    A is groups x M x K and B groups x K x N (f16), ``group_rows`` a CUDA
    int32 tensor of ``groups`` row counts in [0, M].  Rows at or past a
    group's count keep the contents of ``out`` (zeros when ``out`` is not
    given).  Returns ``out`` (groups x M x N, f32)."""
    import torch
    if stream is not None and (out is None or not group_rows.is_contiguous()):
        return _on_stream(stream, grouped_gemm, A, B, group_rows, out, alpha=alpha, bias=bias,
                          activation=activation, slope=slope, out_dtype=out_dtype, tile_n=tile_n,
                          tile_m=tile_m)
    if A.dtype != torch.float16 or B.dtype != torch.float16:
        raise TypeError("A and B must be torch.float16")
    if A.dim() != 3 or B.dim() != 3 or A.shape[0] != B.shape[0] or A.shape[2] != B.shape[1]:
        raise ValueError("A must be G x M x K and B G x K x N")
    if group_rows.dtype != torch.int32 or not group_rows.is_cuda or group_rows.numel() != A.shape[0]:
        raise ValueError("group_rows must be a CUDA int32 tensor of one count per group")
    G, M, K = A.shape
    N = B.shape[2]
    dtype = out.dtype if out is not None else (out_dtype or torch.float32)
    out_names = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
    if dtype not in out_names:
        raise TypeError("out must be torch.float32, torch.float16 or torch.bfloat16")
    if out is None:
        per16 = 16 // torch.tensor([], dtype=dtype).element_size()
        ldc_alloc = max(per16, -(-N // per16) * per16)
        out = torch.zeros((G, M, ldc_alloc), dtype=dtype, device=A.device)[..., :N]
    if tuple(out.shape) != (G, M, N):
        raise ValueError("out must be a G x M x N tensor")
    for t, name in ((A, "A"), (B, "B"), (out, "out")):
        if t.numel() and t.stride(-1) != 1:
            raise ValueError(f"{name} must have a unit last stride")
    rows = group_rows.contiguous()
    opts = _opts(0, tile_n, 0, 0, tile_m)
    if bias is not None and (bias.dtype != torch.float32 or not bias.is_cuda
                             or bias.shape[-1] != N or bias.stride(-1) != 1):
        raise ValueError("bias must be a CUDA float32 tensor of N values (or groups x N)")
    epi = epilogue(alpha, bias.data_ptr() if bias is not None else 0,
                   bias.stride(0) if bias is not None and bias.dim() == 2 else 0,
                   activation, slope, out_names[dtype])
    st = gemm_f16_grouped_fused(A.data_ptr(), B.data_ptr(), out.data_ptr(), rows.data_ptr(),
                                G, M, N, K, A.stride(1), B.stride(1), out.stride(1),
                                A.stride(0), B.stride(0), out.stride(0), epi, opts,
                                _stream_handle(stream))
    check(st)
    return out


def rowsum(X, out=None, *, stream=None):
    """Row sums of a 2-D CUDA tensor (f32, f16 or bf16; any strides): an f32
    tensor of X.shape[0] values, summed in f32 in a fixed order."""
    import torch
    if out is None and stream is not None:
        return _on_stream(stream, rowsum, X)
    names = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
    if X.dtype not in names or X.dim() != 2 or not X.is_cuda:
        raise ValueError("X must be a 2-D CUDA tensor of float32, float16 or bfloat16")
    R, C = X.shape
    if out is None:
        out = torch.empty(R, dtype=torch.float32, device=X.device)
    if out.dtype != torch.float32 or out.numel() != R or (R and out.stride(0) != 1):
        raise ValueError("out must be a contiguous float32 tensor of X.shape[0] values")
    check(rowsum_f32acc(X.data_ptr(), names[X.dtype], out.data_ptr(), R, C, X.stride(0),
                        X.stride(1), _stream_handle(stream)))
    return out


def gemv(A, x, out=None, *, stream=None):
    """``A @ x`` for an f16 CUDA matrix A (unit last stride) and f16 vector x
    (any stride): an f32 vector."""
    import torch
    if out is None and stream is not None:
        return _on_stream(stream, gemv, A, x)
    if A.dtype != torch.float16 or x.dtype != torch.float16 or A.dim() != 2 or x.dim() != 1:
        raise ValueError("A must be a 2-D and x a 1-D torch.float16 CUDA tensor")
    M, K = A.shape
    if x.numel() != K:
        raise ValueError("x must hold A.shape[1] values")
    if K and A.stride(1) != 1:
        raise ValueError("A must have a unit last stride")
    if out is None:
        out = torch.empty(M, dtype=torch.float32, device=A.device)
    check(gemv_f16_f32acc(A.data_ptr(), x.data_ptr(), out.data_ptr(), M, K,
                          A.stride(0) if M > 1 else max(K, 1), x.stride(0) if K > 1 else 1,
                          _stream_handle(stream)))
    return out


# Mixture-of-Experts: token rows to their experts and back.  The experts' side
# is a groups x capacity x width tensor, the layout grouped_gemm takes.

# (The checks below are ordered so that contiguous CUDA tensors, the usual
# case, pass with few attribute reads: a decode step's calls take the GPU two
# or three microseconds each.  torch.empty between two launches costs half of
# what Tensor.new_empty does.)

_ELEM_TYPES = {}


def _elem_type(dtype):
    if not _ELEM_TYPES:
        import torch
        _ELEM_TYPES.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
    code = _ELEM_TYPES.get(dtype)
    if code is None:
        raise TypeError(f"rows must be torch.float32, torch.float16 or torch.bfloat16, not {dtype}")
    return code


def _slots_of(slots):
    """(tokens, topk) of a slots tensor."""
    import torch
    if slots.dtype != torch.int32 or not slots.is_cuda or slots.dim() != 2 or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous CUDA int32 tensor of tokens x topk values")
    return slots.shape


def _token_pitch(x, tokens, width, dtype, name):
    """The row pitch of a tokens x width tensor."""
    if x.dim() != 2 or not x.is_cuda or x.dtype != dtype or x.shape != (tokens, width):
        raise ValueError(f"{name} must be a {tokens} x {width} CUDA tensor of {dtype}")
    if x.is_contiguous():
        return width
    if width > 1 and x.numel() and x.stride(1) != 1:
        raise ValueError(f"{name} must have a unit last stride")
    return x.stride(0) if tokens > 1 else width


def _expert_pitch(rows, width, dtype, name):
    """The row pitch of a groups x capacity x width tensor of evenly spaced rows."""
    if rows.dim() != 3 or not rows.is_cuda or rows.dtype != dtype or rows.shape[2] != width:
        raise ValueError(f"{name} must be a groups x capacity x {width} CUDA tensor of {dtype}")
    if rows.is_contiguous():
        return width
    G, cap, _ = rows.shape
    ld = rows.stride(1) if cap > 1 else rows.stride(0) if G > 1 else width
    if rows.numel() and ((width > 1 and rows.stride(2) != 1) or (G > 1 and rows.stride(0) != cap * ld)
                         or (G * cap > 1 and ld < width)):
        raise ValueError(f"{name} must have a unit last stride and evenly spaced rows "
                         "(stride(0) == capacity * stride(1))")
    return max(ld, width)


def _weights_ptr(weights, slots):
    import torch
    if weights is None:
        return 0
    if weights.dtype != torch.float32 or not weights.is_cuda or weights.shape != slots.shape \
            or not weights.is_contiguous():
        raise ValueError("weights must be a contiguous CUDA float32 tensor of tokens x topk values")
    return weights.data_ptr()


def moe_route(expert_ids, groups, capacity, *, stream=None):
    """Rows for the experts' choices: ``(slots, counts)`` for a tokens x topk
    CUDA tensor of expert numbers (int32 or int64).

    ``slots[t, j] = e * capacity + rank`` with ranks in token order, -1 for a
    choice past the capacity or an id outside [0, groups); ``counts`` is what
    ``grouped_gemm`` takes as ``group_rows``.  Both are int32."""
    import torch
    if stream is not None:
        return _on_stream(stream, moe_route, expert_ids, groups, capacity)
    if expert_ids.dtype not in (torch.int32, torch.int64) or not expert_ids.is_cuda or expert_ids.dim() != 2:
        raise ValueError("expert_ids must be a 2-D CUDA tensor of int32 or int64")
    ids = expert_ids if expert_ids.is_contiguous() else expert_ids.contiguous()
    T, k = ids.shape
    slots = torch.empty((T, k), dtype=torch.int32, device=ids.device)
    counts = torch.empty((groups,), dtype=torch.int32, device=ids.device)
    check(_lib.moe_route_slots(ids.data_ptr(), ids.element_size(), slots.data_ptr(), counts.data_ptr(), T, k, groups,
                               capacity, _stream_handle(stream)))
    return slots, counts


def moe_dispatch(x, slots, groups, capacity, out=None, *, stream=None):
    """Copy token rows to their experts: ``out[e, r] = x[t]`` where
    ``slots[t, j] == e * capacity + r``.

    ``x`` is tokens x width (f32, f16, bf16 or int8).  Returns ``out`` (groups
    x capacity x width); rows no slot names keep their contents (zeros when
    ``out`` is not given)."""
    if out is None and stream is not None:
        return _on_stream(stream, moe_dispatch, x, slots, groups, capacity)
    T, k = _slots_of(slots)
    H = x.shape[-1]
    ldx = _token_pitch(x, T, H, x.dtype, "x")
    if out is None:
        out = x.new_zeros((groups, capacity, H))
    if out.shape != (groups, capacity, H):
        raise ValueError(f"out must be a {groups} x {capacity} x {H} tensor")
    ld = _expert_pitch(out, H, x.dtype, "out")
    check(_lib.moe_dispatch_rows(x.data_ptr(), x.element_size(), slots.data_ptr(), out.data_ptr(), T, k,
                                 groups * capacity, H, ldx, ld, _stream_handle(stream)))
    return out


def moe_dispatch_grad(drows, slots, out=None, *, stream=None):
    """The gradient of ``moe_dispatch``: ``dx[t] = sum_j drows[slots[t, j]]``
    for groups x capacity x width ``drows`` (f32, f16 or bf16); summed in f32,
    returned in the rows' type."""
    import torch
    if out is None and stream is not None:
        return _on_stream(stream, moe_dispatch_grad, drows, slots)
    code = _elem_type(drows.dtype)
    T, k = _slots_of(slots)
    G, cap, H = drows.shape
    ld = _expert_pitch(drows, H, drows.dtype, "drows")
    if out is None:
        out = torch.empty((T, H), dtype=drows.dtype, device=drows.device)
        ldo = H
    else:
        ldo = _token_pitch(out, T, H, drows.dtype, "out")
    check(_lib.moe_dispatch_rows_grad(drows.data_ptr(), code, slots.data_ptr(), out.data_ptr(), T, k, G * cap, H, ld,
                                      ldo, _stream_handle(stream)))
    return out


def moe_combine(rows, slots, weights=None, out=None, *, stream=None):
    """Bring the experts' rows back to their tokens:
    ``out[t] = sum_j weights[t, j] * rows[slots[t, j]]`` for groups x capacity
    x width ``rows`` (f32, f16 or bf16), f32 ``weights`` (tokens x topk; none:
    ones); summed in f32, returned in the rows' type."""
    import torch
    if out is None and stream is not None:
        return _on_stream(stream, moe_combine, rows, slots, weights)
    code = _elem_type(rows.dtype)
    T, k = _slots_of(slots)
    G, cap, H = rows.shape
    ld = _expert_pitch(rows, H, rows.dtype, "rows")
    w = _weights_ptr(weights, slots)
    if out is None:
        out = torch.empty((T, H), dtype=rows.dtype, device=rows.device)
        ldo = H
    else:
        ldo = _token_pitch(out, T, H, rows.dtype, "out")
    check(_lib.moe_combine_rows(rows.data_ptr(), code, slots.data_ptr(), w, out.data_ptr(), T, k, G * cap, H, ld, ldo,
                                _stream_handle(stream)))
    return out


def moe_combine_grad(dout, rows, slots, weights=None, drows=None, *, stream=None):
    """The gradients of ``moe_combine``: ``(drows, dweights)`` with
    ``drows[slots[t, j]] = weights[t, j] * dout[t]`` (rows no slot names keep
    their contents, zeros when ``drows`` is not given) and ``dweights[t, j] =
    <dout[t], rows[slots[t, j]]>`` (f32, 0 for a dropped choice)."""
    import torch
    if stream is not None:
        return _on_stream(stream, moe_combine_grad, dout, rows, slots, weights, drows)
    code = _elem_type(dout.dtype)
    T, k = _slots_of(slots)
    G, cap, H = rows.shape
    ldd = _token_pitch(dout, T, H, dout.dtype, "dout")
    ld = _expert_pitch(rows, H, dout.dtype, "rows")
    w = _weights_ptr(weights, slots)
    if drows is None:
        drows = torch.zeros(rows.shape, dtype=rows.dtype, device=rows.device)
    if drows.shape != rows.shape:
        raise ValueError("drows must have the rows' shape")
    ldr = _expert_pitch(drows, H, dout.dtype, "drows")
    dweights = torch.empty((T, k), dtype=torch.float32, device=dout.device)
    check(_lib.moe_combine_rows_grad(dout.data_ptr(), rows.data_ptr(), code, slots.data_ptr(), w, drows.data_ptr(),
                                     dweights.data_ptr(), T, k, G * cap, H, ldd, ld, ldr, _stream_handle(stream)))
    return drows, dweights


# 8-bit integers.

def quantize_rows(X, group_rows=None, q=None, scales=None, *, stream=None):
    """Quantise the rows of an M x K (or batch x M x K) CUDA tensor (f32, f16
    or bf16) to int8: ``(q, scales)`` with ``scales = max|row| / 127`` and
    ``q = round(X / scales)``.

    ``q``'s rows are allocated with a pitch of a multiple of 16 bytes, as the
    products want.  ``group_rows`` (int32, one count per matrix) limits the
    rows that are read and written."""
    import torch
    if stream is not None and (q is None or scales is None):
        return _on_stream(stream, quantize_rows, X, group_rows, q, scales)
    code = _elem_type(X.dtype)
    shape = X.shape
    three = len(shape) == 3
    if three:
        batch, M, K = shape
        sX, ldx, unit = X.stride()
    elif len(shape) == 2:
        batch, (M, K), sX = 1, shape, 0
        ldx, unit = X.stride()
    if len(shape) not in (2, 3) or not X.is_cuda or (unit != 1 and K > 1 and X.numel()):
        raise ValueError("X must be a 2-D or 3-D CUDA tensor with a unit last stride")
    if q is None:
        ldq = K + -K % 16
        sQ = M * ldq if three else 0
        q = torch.empty_strided(shape, (sQ, ldq, 1) if three else (ldq, 1), dtype=torch.int8, device=X.device)
    else:
        if q.shape != shape or q.dtype != torch.int8 or (K > 1 and q.numel() and q.stride(-1) != 1):
            raise ValueError("q must be an int8 tensor of X's shape with a unit last stride")
        ldq = q.stride(-2)
        sQ = q.stride(0) if three else 0
    if scales is None:
        sS = M if three else 0
        scales = torch.empty((batch, M) if three else M, dtype=torch.float32, device=X.device)
    else:
        if scales.shape != shape[:-1] or scales.dtype != torch.float32 or (M > 1 and scales.stride(-1) != 1):
            raise ValueError("scales must be a float32 tensor of one value per row")
        sS = scales.stride(0) if three else 0
    counts = 0
    if group_rows is not None:
        if group_rows.dtype != torch.int32 or not group_rows.is_cuda or group_rows.numel() != batch \
                or not group_rows.is_contiguous():
            raise ValueError("group_rows must be a contiguous CUDA int32 tensor of one count per matrix")
        counts = group_rows.data_ptr()
    if M <= 1:
        ldx = ldq = K
    check(_lib.quantize_rows_s8(X.data_ptr(), code, q.data_ptr(), scales.data_ptr(), counts, M, K, ldx, ldq, sX, sQ,
                                sS, batch, _stream_handle(stream)))
    return q, scales


def _s8_vector(t, n, batch, three, name):
    """(pointer, stride) of a vector of n values, or one per matrix."""
    import torch
    if t is None:
        return 0, 0
    shape = t.shape
    dim = len(shape)
    if t.dtype != torch.float32 or not t.is_cuda or dim < 1 or shape[-1] != n or dim > (2 if three else 1) \
            or (n > 1 and t.stride(-1) != 1) or (dim == 2 and shape[0] != batch):
        raise ValueError(f"{name} must be a CUDA float32 tensor of {n} values" + (f" (or {batch} x {n})" if three else ""))
    return t.data_ptr(), t.stride(0) if dim == 2 and batch > 1 else 0


def _s8_call(A, B, scale_a, scale_b, group_rows, out, alpha, bias, activation, slope, out_dtype, stream):
    import torch
    if out is None and stream is not None:
        return _on_stream(stream, _s8_call, A, B, scale_a, scale_b, group_rows, None, alpha, bias, activation, slope,
                          out_dtype, None)
    if A.dtype != torch.int8 or B.dtype != torch.int8:
        raise TypeError("A and B must be torch.int8")
    dim = A.dim()
    if dim != B.dim() or dim not in (2, 3):
        raise ValueError("A and B must both be 2-D or both 3-D")
    three = dim == 3
    if three:
        batch, M, K = A.shape
        batch_b, K2, N = B.shape
        sA, lda, uA = A.stride()
        sB, ldb, uB = B.stride()
        if batch_b != batch:
            raise ValueError("batch sizes differ")
        shape = (batch, M, N)
    else:
        batch, sA, sB = 1, 0, 0
        M, K = A.shape
        K2, N = B.shape
        lda, uA = A.stride()
        ldb, uB = B.stride()
        shape = (M, N)
    if K2 != K:
        raise ValueError(f"inner sizes differ: {K} vs {K2}")
    if out is None:
        make = torch.empty if group_rows is None else torch.zeros
        out = make(shape, dtype=out_dtype or torch.float32, device=A.device)
    if out.shape != shape:
        raise ValueError(f"out must be a {' x '.join(map(str, shape))} tensor")
    sC, ldc, uC = out.stride() if three else (0, *out.stride())
    for t, unit, n, name in ((A, uA, K, "A"), (B, uB, N, "B"), (out, uC, N, "out")):
        if not t.is_cuda or (unit != 1 and n > 1 and t.numel()):
            raise ValueError(f"{name} must be a CUDA tensor with a unit last stride")
    pa, sa = _s8_vector(scale_a, M, batch, three, "scale_a")
    pb, sb = _s8_vector(scale_b, N, batch, three, "scale_b")
    pbias, sbias = _s8_vector(bias, N, batch, three, "bias")
    code = _elem_type(out.dtype)
    epi = None  # (none: alpha 1, no bias or activation, f32)
    if code or pbias or alpha != 1 or activation != "none":
        epi = ctypes.byref(GemmEpilogue(alpha, pbias or None, sbias, ACTIVATIONS.get(activation, activation), slope,
                                        code))
    args = (M, N, K, lda if M > 1 else max(K, 1), ldb if K > 1 else max(N, 1), ldc if M > 1 else max(N, 1), sA, sB,
            sC, sa, sb)
    if group_rows is None:
        check(_lib.gemm_s8_scaled(A.data_ptr(), B.data_ptr(), out.data_ptr(), pa, pb, *args, batch, epi,
                                  _stream_handle(stream)))
    else:
        check(_lib.gemm_s8_grouped_scaled(A.data_ptr(), B.data_ptr(), out.data_ptr(), pa, pb, group_rows.data_ptr(),
                                          batch, *args, epi, _stream_handle(stream)))
    return out


def gemm_s8(A, B, scale_a=None, scale_b=None, out=None, *, alpha=1.0, bias=None, activation="none", slope=0.01,
            out_dtype=None, stream=None):
    """``out = activation(alpha * scale_a[:, None] * scale_b[None, :] * (A @ B) + bias)``
    for int8 CUDA tensors A (M x K) and B (K x N), or a batch of them; the sums
    are exact integers.  ``scale_a`` holds M and ``scale_b`` N f32 values (per
    matrix, or one vector for the batch; none: ones); ``out`` is f32 unless
    ``out_dtype`` (or the given ``out``) says torch.float16 / torch.bfloat16.
    Pitches that are multiples of 16 bytes are read in place; others cost a
    copy.  Returns ``out``."""
    return _s8_call(A, B, scale_a, scale_b, None, out, alpha, bias, activation, slope, out_dtype, stream)


def grouped_gemm_s8(A, B, scale_a, scale_b, group_rows, out=None, *, alpha=1.0, bias=None, activation="none",
                    slope=0.01, out_dtype=None, stream=None):
    """The grouped (Mixture-of-Experts) form of ``gemm_s8``: A is groups x M x
    K, B groups x K x N; of group g the first ``group_rows[g]`` rows are
    computed, the others keep the contents of ``out`` (zeros when not given)."""
    import torch
    if A.dim() != 3 or group_rows.dtype != torch.int32 or not group_rows.is_cuda \
            or group_rows.numel() != A.shape[0] or not group_rows.is_contiguous():
        raise ValueError("A must be 3-D and group_rows a contiguous CUDA int32 tensor of one count per group")
    return _s8_call(A, B, scale_a, scale_b, group_rows, out, alpha, bias, activation, slope, out_dtype, stream)


def gemm_host(A_host, B_host, C_host, dA, dB, dC, stream=None):
    """End-to-end call from host memory: copy A and B (pinned CPU f16
    tensors) into the device buffers dA and dB, run the GEMM into dC, copy dC
    back into C_host (pinned CPU f32).  All on one stream, asynchronously;
    synchronise the stream before reading C_host."""
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    with torch.cuda.stream(s):
        dA.copy_(A_host, non_blocking=True)
        dB.copy_(B_host, non_blocking=True)
        gemm(dA, dB, dC, stream=s)
        C_host.copy_(dC, non_blocking=True)
    return C_host


class HostPipeline:
    """C = A . B for a stream of host-resident problems of one shape.

    Each ``submit`` copies A and B (pinned CPU f16 tensors) to the device,
    runs the GEMM and copies C back into the given pinned CPU f32 tensor.
    ``depth`` device buffer sets and three CUDA streams (upload, GEMM,
    download) let the upload of one problem overlap the GEMM and the download
    of the previous ones; events order the three stages of each problem and
    keep a buffer set from being reused before its result has been read back.
    Torch provides the memory, streams and copies; the GEMM is this library's.
    Call ``synchronize`` before reading the last ``depth`` results."""

    def __init__(self, M, N, K, depth=2, device=None):
        import torch
        self.M, self.N, self.K, self.depth = M, N, K, depth
        dev = torch.device("cuda") if device is None else torch.device(device)
        self.dA = [torch.empty((M, K), dtype=torch.float16, device=dev) for _ in range(depth)]
        self.dB = [torch.empty((K, N), dtype=torch.float16, device=dev) for _ in range(depth)]
        ldc = max(4, -(-N // 4) * 4)
        self.dC = [torch.empty((M, ldc), dtype=torch.float32, device=dev)[:, :N]
                   for _ in range(depth)]
        self.s_in = torch.cuda.Stream(device=dev)
        self.s_gemm = torch.cuda.Stream(device=dev)
        self.s_out = torch.cuda.Stream(device=dev)
        self.in_done = [torch.cuda.Event() for _ in range(depth)]
        self.gemm_done = [torch.cuda.Event() for _ in range(depth)]
        self.out_done = [torch.cuda.Event() for _ in range(depth)]
        self.used = [False] * depth
        self.count = 0

    def submit(self, A_host, B_host, C_host):
        import torch
        i = self.count % self.depth
        self.count += 1
        if self.used[i]:
            self.s_in.wait_event(self.out_done[i])  # buffer set i is free again
        with torch.cuda.stream(self.s_in):
            self.dA[i].copy_(A_host, non_blocking=True)
            self.dB[i].copy_(B_host, non_blocking=True)
            self.in_done[i].record(self.s_in)
        self.s_gemm.wait_event(self.in_done[i])
        gemm(self.dA[i], self.dB[i], self.dC[i], stream=self.s_gemm)
        self.gemm_done[i].record(self.s_gemm)
        self.s_out.wait_event(self.gemm_done[i])
        with torch.cuda.stream(self.s_out):
            C_host.copy_(self.dC[i], non_blocking=True)
            self.out_done[i].record(self.s_out)
        self.used[i] = True
        return C_host

    def synchronize(self):
        self.s_out.synchronize()
