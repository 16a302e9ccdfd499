// Embedding lookup from an FP8 table, and the table's gradient.
#include "ops_common.cuh"

namespace {

using namespace fp8z1;

struct Ids {
    const void* p;
    int32_t bytes;
    __device__ __forceinline__ int64_t at(int64_t t) const
    {
        return bytes == 8 ? static_cast<const int64_t*>(p)[t] : static_cast<const int32_t*>(p)[t];
    }
};

template <class T>
__global__ void embed_kernel(int64_t vocab, int64_t dim, const uint8_t* codes, const float* scales, Ids ids,
                             float alpha, T* out, int64_t ld)
{
    const int64_t t = blockIdx.x, id = ids.at(t);
    const bool there = id >= 0 && id < vocab;
    const int64_t sc = (dim + 127) / 128;
    for (int64_t d = threadIdx.x; d < dim; d += blockDim.x)
        out[t * ld + d] = from_float<T>(
            there ? alpha * (e4m3_value(codes[id * dim + d]) * scales[id / 128 * sc + d / 128]) : 0.0f);
}

// One CTA per table row; its threads walk the tokens in order.
template <class T>
__global__ void embed_grad_kernel(int64_t dim, Ids ids, int64_t tokens, float alpha, const T* dy, int64_t ld,
                                  float* d_table)
{
    __shared__ int32_t list[1024];
    __shared__ int32_t warp_count[8];
    const int64_t v = blockIdx.x;
    for (int64_t d0 = 0; d0 < dim; d0 += blockDim.x) {
        const int64_t d = d0 + threadIdx.x;
        float acc = 0.0f;
        for (int64_t t0 = 0; t0 < tokens; t0 += blockDim.x) {
            const int64_t t = t0 + threadIdx.x;
            const bool hit = t < tokens && ids.at(t) == v;
            if (!__syncthreads_or(hit)) continue;
            const unsigned m = __ballot_sync(0xffffffffu, hit);
            const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
            if (lane == 0) warp_count[w] = __popc(m);
            __syncthreads();
            int base = 0, n = 0;
            for (int i = 0; i < (int)blockDim.x / 32; ++i) {
                if (i < w) base += warp_count[i];
                n += warp_count[i];
            }
            if (hit) list[base + __popc(m & ((1u << lane) - 1))] = (int32_t)t;
            __syncthreads();
            if (d < dim)
                for (int i = 0; i < n; ++i) acc += to_float(dy[list[i] * ld + d]);
            __syncthreads();
        }
        if (d < dim) d_table[v * dim + d] = alpha * acc;
    }
}

int check_ids(int64_t vocab, int64_t dim, const void* ids, int32_t id_bytes, int64_t tokens, float alpha,
              const void* rows, int32_t type, int64_t ld)
{
    if (vocab < 1 || vocab >= (int64_t)1 << 31 || dim < 1 || dim >= (int64_t)1 << 31 || tokens < 0 ||
        tokens > kMaxRows || (id_bytes != 4 && id_bytes != 8) || (type != FP8Z1_F32 && type != FP8Z1_BF16) ||
        ld < dim || !isfinite(alpha))
        return FP8Z1_EINVAL;
    if (tokens > 0 && (!ids || !rows)) return FP8Z1_EINVAL;
    if (!aligned(ids, id_bytes) || !aligned(rows, type == FP8Z1_F32 ? 4 : 2)) return FP8Z1_EALIGN;
    return FP8Z1_OK;
}

}  // namespace

extern "C" int fp8z1_embed(int64_t vocab, int64_t dim, const uint8_t* codes, const float* scales, const void* ids,
                           int32_t id_bytes, int64_t tokens, float alpha, void* out, int32_t out_type,
                           int64_t ld_out, void* stream)
{
    if (!codes || !scales) return FP8Z1_EINVAL;
    const int st = check_ids(vocab, dim, ids, id_bytes, tokens, alpha, out, out_type, ld_out);
    if (st != FP8Z1_OK) return st;
    if (!aligned(scales, 4)) return FP8Z1_EALIGN;
    if (tokens == 0) return FP8Z1_OK;
    NvtxRange r("fp8z1_embed");
    const Ids i{ids, id_bytes};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    count_launch();
    if (out_type == FP8Z1_F32)
        embed_kernel<<<(unsigned)tokens, 256, 0, s>>>(vocab, dim, codes, scales, i, alpha, static_cast<float*>(out), ld_out);
    else
        embed_kernel<<<(unsigned)tokens, 256, 0, s>>>(vocab, dim, codes, scales, i, alpha,
                                                      static_cast<__nv_bfloat16*>(out), ld_out);
    return launch_status();
}

extern "C" int fp8z1_embed_grad_workspace(int64_t vocab, int64_t dim, int64_t tokens, int64_t* bytes)
{
    if (!bytes || vocab < 1 || vocab >= (int64_t)1 << 31 || dim < 1 || dim >= (int64_t)1 << 31 || tokens < 0 ||
        tokens > kMaxRows)
        return FP8Z1_EINVAL;
    *bytes = 256;
    return FP8Z1_OK;
}

extern "C" int fp8z1_embed_grad(int64_t vocab, int64_t dim, const void* ids, int32_t id_bytes, int64_t tokens,
                                float alpha, const void* dy, int32_t dy_type, int64_t ld_dy, float* d_table,
                                void* workspace, void* stream)
{
    if (!d_table || !workspace) return FP8Z1_EINVAL;
    const int st = check_ids(vocab, dim, ids, id_bytes, tokens, alpha, dy, dy_type, ld_dy);
    if (st != FP8Z1_OK) return st;
    if (!aligned(d_table, 4) || !aligned(workspace, 256)) return FP8Z1_EALIGN;
    NvtxRange r("fp8z1_embed_grad");
    const Ids i{ids, id_bytes};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    count_launch();
    if (dy_type == FP8Z1_F32)
        embed_grad_kernel<<<(unsigned)vocab, 256, 0, s>>>(dim, i, tokens, alpha, static_cast<const float*>(dy), ld_dy, d_table);
    else
        embed_grad_kernel<<<(unsigned)vocab, 256, 0, s>>>(dim, i, tokens, alpha, static_cast<const __nv_bfloat16*>(dy),
                                                          ld_dy, d_table);
    return launch_status();
}
