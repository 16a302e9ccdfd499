// Helpers shared by the model operators (embedding, gated FFN, distillation).
#pragma once

#include <cuda_bf16.h>
#include <math.h>

#include <atomic>

#include "fp8z1_ops.h"
#include "internal.h"
#include "update.cuh"

namespace fp8z1 {

constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int kSms = 152;  // of a GB300: rules that choose by size go by it (results do not)

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t align256(int64_t n) { return (n + 255) & ~(int64_t)255; }

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x)
{
    return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x)
{
    return __float2bfloat16_rn(x);
}

__device__ __forceinline__ float e4m3_value(uint8_t code) { return e4m3x2_decode(code).x; }

// Lets kKernel take up to `bytes` (always the same) of dynamic shared memory on the
// current device; asked once for each, as the question costs as much as a launch.
template <auto kKernel>
bool allow_smem(int bytes)
{
    static std::atomic<uint32_t> asked{0};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev < 32 && asked.load(std::memory_order_relaxed) >> dev & 1) return true;
    if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (dev < 32) asked.fetch_or(1u << dev, std::memory_order_relaxed);
    return true;
}

// The SM count of the current device (0 when it cannot be read).
inline int sm_count_here()
{
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return n;
}

}  // namespace fp8z1
