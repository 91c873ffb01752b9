// device_common.cuh -- what every kernel of the library shares: the device
// error word and its bits, the checked build's index test, the bounded waits
// and the paired 16-bit conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "sm100.cuh"

namespace tl {

// Device error word: one per translation unit, all of them read and cleared by
// tl_check_device.
static __device__ unsigned int g_device_error = 0;

// Read this translation unit's error word and clear it; false when a CUDA
// call failed.
static inline bool take_device_error(unsigned int *word)
{
    unsigned int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(v)) != cudaSuccess)
        return false;
    if (v && cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero)) != cudaSuccess)
        return false;
    *word = v;
    return true;
}

enum : unsigned {
    ERR_PRODUCER = 1u,
    ERR_MMA_DATA = 2u,
    ERR_MMA_ACC = 4u,
    ERR_EPILOGUE = 8u,
    ERR_DRAIN = 16u,
    ERR_SPLIT = 32u,   // a part of a split tile could not record its arrival (C incomplete)
    ERR_CHECK = 128u,  // checked build only: an index invariant failed (the access was skipped)
};

// The checked build (compiled with -DTL_CHECKED, libtlgemm_checked.so) tests
// the kernel's index invariants at run time: a violation sets ERR_CHECK in the
// device error word and the access it guards is skipped, never a trap.  In
// the product build check_ok() is the constant true and costs nothing.
#ifdef TL_CHECKED
constexpr bool kCheckedBuild = true;
#else
constexpr bool kCheckedBuild = false;
#endif

__device__ __forceinline__ bool check_ok(bool cond)
{
    if (kCheckedBuild && !cond) {
        atomicOr(&g_device_error, ERR_CHECK);
        return false;
    }
    return true;
}

// Bounded wait.  Returns false when the abort flag is raised by another role
// (or by the peer CTA) or when this wait runs past timeout_ns; then it raises
// the flag itself, and the peer's too when `peer_abort` (a shared::cluster
// address) is non-zero.  CLUSTER_SCOPE acquires at cluster scope, for
// barriers the peer CTA arrives on.
template <bool CLUSTER_SCOPE = false>
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                             uint64_t timeout_ns, unsigned code, uint32_t peer_abort = 0)
{
    auto test = [&]() { return CLUSTER_SCOPE ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity); };
    if (test())
        return true;
    const uint64_t t0 = global_timer_ns();
    while (true) {
        if (test())
            return true;
        if (*abort_flag)
            return false;
        if (global_timer_ns() - t0 > timeout_ns) {
            *abort_flag = 1;
            if (peer_abort)
                st_shared_cluster_u32(peer_abort, 1u);
            atomicOr(&g_device_error, code);
            return false;
        }
    }
}

// Bounded wait that ignores the abort flag (used to let in-flight work land).
__device__ __forceinline__ bool wait_drain(uint32_t bar, uint32_t parity, uint64_t timeout_ns)
{
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > timeout_ns) {
            atomicOr(&g_device_error, ERR_DRAIN);
            return false;
        }
    }
    return true;
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (DT == 1) {
        __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&v);
    } else {
        __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&v);
    }
}

template <int DT>
__device__ __forceinline__ float to_float(uint16_t bits)
{
    if constexpr (DT == 1)
        return __uint_as_float(static_cast<uint32_t>(bits) << 16);
    else
        return __half2float(__ushort_as_half(bits));
}

} // namespace tl
