// api_internal.h -- what the host sides of the C ABI share (gemm_api.cu defines
// it): error reporting, the per-device state, argument checks and tensor maps.
#pragma once

#include "../../include/tsm_gemm.h"
#include "gemm_internal.h"

#include <string>

namespace tsm {

// The message behind gemm_last_error_string (cleared at each entry point).
extern thread_local std::string g_last_error;

// A 64-bit value unique to each launch of this process, never 0.
uint64_t next_launch_epoch();

// Record a message and return the status.
gemm_status_t fail(gemm_status_t st, const char *fmt, ...);
gemm_status_t fail_cuda(cudaError_t e, const char *what);

struct DeviceState {
    bool ready = false;
    int sms = 0;
    int cc_major = 0, cc_minor = 0;
    int smem_optin = 0;
    bool attrs_set[46] = {};  // see attr_index
    cudaMemPool_t pool = nullptr;
    uint32_t *status = nullptr;
    // Clusters of 2 and of 4 CTAs of the cluster-sum kernel that fit at once.
    int caps2 = 0, caps4 = 0;
};

gemm_status_t device_state(int dev, DeviceState **out);

// Bytes spanned by `batch` matrices of `rows` x `cols` elements of `elem`
// bytes, row stride `ld`, batch stride `stride` (all in elements).
int64_t span_bytes(int64_t batch, int64_t stride, int64_t rows, int64_t ld, int64_t cols, int64_t elem);

bool overlaps(const void *p, int64_t pn, const void *q, int64_t qn);

// The pointer is device memory of `dev` and its allocation covers `bytes`.
gemm_status_t check_device_pointer(const void *p, int64_t bytes, int dev, const char *name);

// A rank-3 tensor map (columns, rows, matrices), strides in elements.
gemm_status_t encode_3d(CUtensorMap *map, CUtensorMapDataType dt, int elem, const void *base,
                        int64_t cols, int64_t rows, int64_t mats, int64_t ld, int64_t stride,
                        uint32_t box_cols, uint32_t box_rows, CUtensorMapL2promotion promo,
                        const char *name, uint32_t box_mats = 1,
                        CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

// The public epilogue description, checked, as the kernels' Epilogue.
gemm_status_t epilogue_of(const gemm_epilogue_t *e, Epilogue *out);

inline int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

}  // namespace tsm
