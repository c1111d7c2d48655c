// api_checks.h -- argument checks that the operators' host sides share.
#pragma once

#include "api_internal.h"

namespace tsm {

constexpr int64_t kInt32Max = 2147483647;
constexpr int64_t kMaxSize = int64_t(1) << 40;

inline bool misaligned(const void *p, int64_t bytes)
{
    return (reinterpret_cast<uintptr_t>(p) & uintptr_t(bytes - 1)) != 0;
}

inline int elem_bytes(int32_t t) { return t == GEMM_OUT_F32 ? 4 : 2; }

inline bool known_elem(int32_t t) { return t == GEMM_OUT_F32 || t == GEMM_OUT_F16 || t == GEMM_OUT_BF16; }

// The current device and its state.  (What makes the state, in the thread's first
// call, goes to no stream, so that call may be a captured one.)
inline gemm_status_t current(int *dev, DeviceState **ds)
{
    const cudaError_t e = cudaGetDevice(dev);
    if (e != cudaSuccess)
        return fail_cuda(e, "cudaGetDevice");
    thread_local int made = -1;  // the device of the last call
    if (made == *dev)
        return device_state(*dev, ds);
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaThreadExchangeStreamCaptureMode(&mode);
    const gemm_status_t st = device_state(*dev, ds);
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (st == GEMM_OK)
        made = *dev;
    return st;
}

// One buffer of a call: checked for its address and, once all are known, on
// the device.
struct Buffer {
    const void *p;
    int64_t bytes;
    const char *name;
    bool written;
};

// Every buffer non-null where it holds something, no written one overlapping
// another.
inline gemm_status_t check_buffers(const Buffer *b, int n)
{
    for (int i = 0; i < n; ++i)
        if (b[i].bytes > 0 && !b[i].p)
            return fail(GEMM_ERR_INVALID_VALUE, "%s is NULL", b[i].name);
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n; ++j)
            if ((b[i].written || b[j].written) && overlaps(b[i].p, b[i].bytes, b[j].p, b[j].bytes))
                return fail(GEMM_ERR_ALIAS, "%s overlaps %s", b[i].name, b[j].name);
    return GEMM_OK;
}

inline gemm_status_t check_on_device(const Buffer *b, int n, int dev)
{
    for (int i = 0; i < n; ++i)
        if (b[i].bytes > 0) {
            const gemm_status_t st = check_device_pointer(b[i].p, b[i].bytes, dev, b[i].name);
            if (st != GEMM_OK)
                return st;
        }
    return GEMM_OK;
}

// Bytes spanned by `batch` matrices `stride` elements apart of `rows` rows `ld`
// apart.  More than 64 bits hold come out as the most that they hold, which
// lies in no allocation.
inline int64_t reach(int64_t batch, int64_t stride, int64_t rows, int64_t ld, int64_t cols, int64_t elem)
{
    if (batch <= 0 || rows <= 0 || cols <= 0)
        return 0;
    const __int128 bytes = (__int128(batch - 1) * stride + __int128(rows - 1) * ld + cols) * elem;
    return bytes > INT64_MAX ? INT64_MAX : int64_t(bytes);
}

// Bytes of `rows` rows of `width` elements `ld` apart.
inline int64_t span(int64_t rows, int64_t width, int64_t ld, int64_t elem) { return reach(1, 0, rows, ld, width, elem); }

// Bytes of one access: 16 or 4 where every address, pitch and width in `all`
// (or-ed together, in bytes) is a multiple, else one element.
inline int access_bytes(uint64_t all, int64_t elem)
{
    return (all & 15u) == 0 ? 16 : (all & 3u) == 0 ? 4 : int(elem);
}

}  // namespace tsm
