// Distillation loss against a teacher's top logits, and its gradient.
#include "ops_common.cuh"

namespace {

using namespace fp8z1;

constexpr int kThreads = 256;

__device__ float block_sum(float v, float* tmp)
{
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    v = tmp[0];
    for (int i = 1; i < kThreads / 32; ++i) v += tmp[i];
    return v;
}

__device__ float block_max(float v, float* tmp)
{
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = v;
    __syncthreads();
    v = tmp[0];
    for (int i = 1; i < kThreads / 32; ++i) v = fmaxf(v, tmp[i]);
    return v;
}

// One CTA per row.
template <class T>
__global__ void distill_kernel(const T* logits, int64_t ld, int64_t vocab, const int32_t* ids, const float* teacher,
                               int top, float tau, const float* weight, float* loss, T* dlogits, int64_t ld_d)
{
    __shared__ float tmp[kThreads / 32];
    __shared__ int32_t id[FP8Z1_DISTILL_MAX_TOP];
    __shared__ float p[FP8Z1_DISTILL_MAX_TOP];
    const int64_t r = blockIdx.x;
    const T* z = logits + r * ld;
    T* dz = dlogits ? dlogits + r * ld_d : nullptr;
    const float w = weight ? weight[r] : 1.0f;
    float tmax = -INFINITY;
    int any = 0;
    for (int k = threadIdx.x; k < top; k += kThreads) {
        const int32_t j = ids[r * top + k];
        const float t = teacher[r * top + k];
        const bool there = j >= 0 && j < vocab && t != -INFINITY;
        id[k] = there ? j : -1;
        p[k] = there ? t / tau : -INFINITY;
        any |= there;
        tmax = fmaxf(tmax, p[k]);
    }
    any = __syncthreads_or(any);
    if (w == 0.0f || !any) {
        if (threadIdx.x == 0) loss[r] = 0.0f;
        if (dz)
            for (int64_t j = threadIdx.x; j < vocab; j += kThreads) dz[j] = from_float<T>(0.0f);
        return;
    }
    tmax = block_max(tmax, tmp);
    float mass = 0.0f;
    for (int k = threadIdx.x; k < top; k += kThreads) mass += id[k] < 0 ? 0.0f : expf(p[k] - tmax);
    mass = block_sum(mass, tmp);
    float zmax = -INFINITY;
    for (int64_t j = threadIdx.x; j < vocab; j += kThreads) zmax = fmaxf(zmax, to_float(z[j]));
    zmax = block_max(zmax, tmp);
    if (zmax == -INFINITY) zmax = 0.0f;
    float total = 0.0f;
    for (int64_t j = threadIdx.x; j < vocab; j += kThreads) total += expf((to_float(z[j]) - zmax) / tau);
    total = block_sum(total, tmp);
    float l = 0.0f;
    // a row of -inf alone has q = 0: its log q is z = -inf, not -inf - -inf
    const float log_total = total == 0.0f ? 0.0f : logf(total), log_mass = logf(mass);
    for (int k = threadIdx.x; k < top; k += kThreads) {
        if (id[k] < 0) continue;
        const float lp = p[k] - tmax - log_mass;
        const float pk = expf(lp);
        l += pk * (lp - ((to_float(z[id[k]]) - zmax) / tau - log_total));
        p[k] = pk;
    }
    l = block_sum(l, tmp);
    if (threadIdx.x == 0) loss[r] = tau * tau * l;
    if (!dz) return;
    const float inv = total > 0.0f ? 1.0f / total : (total == 0.0f ? 0.0f : total);
    for (int64_t j = threadIdx.x; j < vocab; j += kThreads) {
        float d = expf((to_float(z[j]) - zmax) / tau) * inv;
        for (int k = 0; k < top; ++k)
            if (id[k] == j) d -= p[k];
        dz[j] = from_float<T>(w * tau * d);
    }
}

}  // namespace

extern "C" int fp8z1_distill(const void* logits, int32_t type, int64_t ld, int64_t rows, int64_t vocab,
                             const int32_t* teacher_ids, const float* teacher_logits, int64_t top,
                             float temperature, const float* row_weight, float* loss, void* dlogits, int64_t ld_d,
                             void* stream)
{
    if (rows < 0 || rows > kMaxRows || vocab < 1 || vocab >= (int64_t)1 << 31 || top < 1 ||
        top > FP8Z1_DISTILL_MAX_TOP || (type != FP8Z1_F32 && type != FP8Z1_BF16) || ld < vocab ||
        (dlogits && ld_d < vocab) || (dlogits && dlogits == logits && ld_d != ld) || !isfinite(temperature) ||
        temperature <= 0.0f)
        return FP8Z1_EINVAL;
    if (rows > 0 && (!logits || !teacher_ids || !teacher_logits || !loss)) return FP8Z1_EINVAL;
    const int esz = type == FP8Z1_F32 ? 4 : 2;
    if (!aligned(logits, esz) || !aligned(dlogits, esz) || !aligned(teacher_ids, 4) || !aligned(teacher_logits, 4) ||
        !aligned(row_weight, 4) || !aligned(loss, 4))
        return FP8Z1_EALIGN;
    if (rows == 0) return FP8Z1_OK;
    NvtxRange r("fp8z1_distill");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    count_launch();
    if (type == FP8Z1_F32)
        distill_kernel<float><<<(unsigned)rows, kThreads, 0, s>>>(
            static_cast<const float*>(logits), ld, vocab, teacher_ids, teacher_logits, (int)top, temperature,
            row_weight, loss, static_cast<float*>(dlogits), ld_d);
    else
        distill_kernel<__nv_bfloat16><<<(unsigned)rows, kThreads, 0, s>>>(
            static_cast<const __nv_bfloat16*>(logits), ld, vocab, teacher_ids, teacher_logits, (int)top, temperature,
            row_weight, loss, static_cast<__nv_bfloat16*>(dlogits), ld_d);
    return launch_status();
}
