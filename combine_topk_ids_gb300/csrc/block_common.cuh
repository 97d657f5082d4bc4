// Device and host helpers of the operators around the expert layer (norm, router, 4-bit
// experts).  Header-only; every symbol has internal linkage in each translation unit.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/moe_block.h"
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr unsigned kAllLanes = 0xffffffffu;

inline bool is_aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t dtype_bytes(int32_t d) { return d == MOE_DTYPE_FP32 ? 4 : 2; }
inline bool bad_dtype(int32_t d) { return d != MOE_DTYPE_BF16 && d != MOE_DTYPE_FP32; }
inline int status_of(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

__device__ __forceinline__ float lo_f32(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f32(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// two floats rounded to a bf16 pair (a in the low half)
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// The next kernel of the call may be launched: it waits for this one before it touches what
// this one writes.
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAllLanes, v, o);
    return v;
}

}  // namespace
}  // namespace moe
