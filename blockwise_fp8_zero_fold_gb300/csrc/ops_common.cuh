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

// out[c] = sum over i < n of part[i, c], [n, cols] FP32, in a fixed order (rms_norm.cu).
int launch_column_sum(const float* part, int n, int64_t cols, float* out, cudaStream_t s);

// The memory of `n` rows of `bytes` each, `ld` bytes apart (p NULL: none).
struct Area {
    const void* p;
    int64_t n, bytes, ld;
};
inline Area dense(const void* p, int64_t bytes) { return Area{p, 1, bytes, bytes}; }

// Whether two share a byte.  Rows of one stride may lie between the other's rows, as columns of one buffer; of several
// strides they count as shared wherever one begins before the other's end.
inline bool overlap(Area a, Area b)
{
    if (!a.p || !b.p || a.n < 1 || b.n < 1 || a.bytes < 1 || b.bytes < 1) return false;
    const auto begin = [](const Area& x) { return (unsigned __int128)reinterpret_cast<uintptr_t>(x.p); };
    const auto end = [&](const Area& x) { return begin(x) + (unsigned __int128)(x.n - 1) * (unsigned __int128)x.ld + x.bytes; };
    if (end(a) <= begin(b) || end(b) <= begin(a)) return false;
    if (a.n == 1) a.ld = b.ld;
    if (b.n == 1) b.ld = a.ld;
    if (a.ld != b.ld || (a.n == 1 && b.n == 1)) return true;
    const int64_t to = (int64_t)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p)) % a.ld;
    const int64_t at = to < 0 ? to + a.ld : to;  // of b's rows, from the start of one of a's
    return at < a.bytes || at + b.bytes > a.ld;
}
// Whether b is a, or shares nothing with it.
inline bool same_or_apart(const Area& a, const Area& b)
{
    return (a.p == b.p && a.n == b.n && a.bytes == b.bytes && (a.ld == b.ld || a.n == 1)) || !overlap(a, b);
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
