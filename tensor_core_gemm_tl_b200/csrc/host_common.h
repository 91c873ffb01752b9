// host_common.h -- host-side pieces shared by the library's translation units:
// per-device state (SM count, the stream-ordered memory pool, raised
// shared-memory limits), the tensor-map encoder and small helpers.  Defined in
// tl_gemm.cu unless said otherwise.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <unordered_map>

#include "tl_gemm.h"

namespace tl {

constexpr uint64_t kDefaultTimeoutNs = 10ull * 1000 * 1000 * 1000;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled, or null when the driver does not offer it
EncodeTiledFn encode_fn();

struct DeviceState {
    int num_sms = 0;
    int cc_major = 0;
    cudaMemPool_t pool = nullptr;
    std::unordered_map<const void *, bool> smem_set;  // kernels whose smem limit is raised
    std::unordered_map<const void *, int> max_clusters;  // resident clusters of two, per kernel
};

// The current device's state, made on its first use
tl_status device_state(DeviceState **out);

// The device's stream-ordered pool for temporaries
tl_status ensure_pool(DeviceState *d);

// Raise a kernel's dynamic shared-memory limit once per device
tl_status raise_smem_limit(DeviceState *d, const void *fn, int bytes);

// Whether raise_smem_limit has been through for the kernel on this device
bool smem_limit_raised(DeviceState *d, const void *fn);

// Read and clear the error word of the kernels of one translation unit (each
// has its own; defined there); false when a CUDA call failed
bool take_error_attention_ex(unsigned int *word);
bool take_error_attention_bwd(unsigned int *word);
bool take_error_tree_attention(unsigned int *word);

} // namespace tl
