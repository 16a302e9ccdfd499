// Tokens sorted by expert, and back.
//
// A choice (t, j) of expert ids[t, j] gets a row: rows are grouped by expert, a group
// in the order of the choices.  offsets[e] is the first row of expert e, place[t, j]
// the choice's row (-1: no expert).
//
//   dispatch   rows[place[t, j]] = x[t], rows behind the last 0
//   combine    y[t] = r[t] + sum_j w[t, j] rows[place[t, j]]     (with w = 1 dispatch's gradient)
//   gradient   d_rows[place[t, j]] = w[t, j] dy[t],   d_w[t, j] = dy[t] . rows[place[t, j]]
//
// Sums are FP32 in the order of j (over columns: of the threads), without atomics.
// All four are bound by the rows moved: a token's row is read once for all its choices.
#include <cooperative_groups.h>

#include <algorithm>

#include "ops_common.cuh"

namespace fp8z1 {
namespace {

using bf16 = __nv_bfloat16;
namespace cg = cooperative_groups;

constexpr int kMostExperts = 1024, kMostTop = 64;

// ---- the sort -----------------------------------------------------------------------
//
// A cluster of CTAs, each warp a run of the choices, twice over: counts of every
// expert in shared memory by warp, their sums over warps, CTAs and experts, then every
// choice's row is its warp's next one of that expert.  Choices of one expert inside
// 32 are ranked by a match of the lanes.

struct SortArgs {
    const void* ids;
    int64_t n;
    int32_t experts;
    int32_t per_warp;  // choices of a warp, a multiple of 32
    int32_t *offsets, *place;
};

template <class Id>
__device__ __forceinline__ int expert_of(const Id* ids, int64_t i, int64_t n, int experts)
{
    if (i >= n) return -1;
    const Id e = ids[i];
    return e >= 0 && e < (Id)experts ? (int)e : -1;
}

template <class Id>
__global__ void __launch_bounds__(1024) sort_kernel(const SortArgs a)
{
    extern __shared__ int32_t counts[];  // [warps][experts], then [experts] of the CTA
    __shared__ int32_t scan[32];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.experts;
    int32_t* mine = counts + warp * E;
    int32_t* total = counts + warps * E;
    const Id* ids = static_cast<const Id*>(a.ids);
    const int64_t i0 = ((int64_t)rank * warps + warp) * a.per_warp, i1 = min(i0 + a.per_warp, a.n);
    for (int e = lane; e < E; e += 32) mine[e] = 0;
    __syncwarp();
    for (int64_t i = i0; i < i1; i += 32) {
        const int e = expert_of(ids, i + lane, a.n, E);
        const unsigned same = __match_any_sync(0xffffffffu, e);
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        int32_t sum = 0;
        for (int w = 0; w < warps; ++w) {
            const int32_t n = counts[w * E + e];
            counts[w * E + e] = sum;
            sum += n;
        }
        total[e] = sum;
    }
    if (ctas > 1)
        cluster.sync();
    else
        __syncthreads();
    // 32 neighbouring experts a warp: what lies before each of them
    int32_t before = 0;  // of all experts up to this round's first
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        int32_t all = 0, ahead = 0;
        if (e < E)
            for (int c = 0; c < ctas; ++c) {
                const int32_t n = ctas > 1 ? cluster.map_shared_rank(total, c)[e] : total[e];
                if (c < rank) ahead += n;
                all += n;
            }
        int32_t sum = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t n = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += n;
        }
        if (lane == 31) scan[warp] = sum;
        __syncthreads();
        int32_t start = before + sum - all, last = before;
        for (int w = 0; w < warps; ++w) {
            if (w < warp) start += scan[w];
            last += scan[w];
        }
        before = last;
        if (e < E) {
            for (int w = 0; w < warps; ++w) counts[w * E + e] += start + ahead;
            if (rank == 0) a.offsets[e] = start;
            if (rank == 0 && e == E - 1) a.offsets[E] = start + all;
        }
        __syncthreads();
    }
    for (int64_t i = i0; i < i1; i += 32) {
        const int e = expert_of(ids, i + lane, a.n, E);
        const unsigned same = __match_any_sync(0xffffffffu, e);
        const int32_t at = e < 0 ? -1 : mine[e] + __popc(same & ((1u << lane) - 1));
        if (i + lane < a.n) a.place[i + lane] = at;
        __syncwarp();
        if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
        __syncwarp();
    }
    if (ctas > 1) cluster.sync();  // no CTA leaves before its counts are read
}

// ---- rows ----------------------------------------------------------------------------

struct RowArgs {
    int64_t tokens, n;  // n: tokens * top
    int32_t top, experts;
    int64_t cols;       // of the element type, or of V
    const int32_t *offsets, *place;
    const float* weight;
    const void *x, *rows;
    void *y, *out;
    int64_t ld_x, ld_rows, ld_y, ld_out;
    float* d_weight;
};

// Rows behind the last expert's, cleared by the CTAs in turn.
template <class V>
__device__ __forceinline__ void clear_rest(const RowArgs& a, V* out, int64_t ld, int64_t cols)
{
    const int64_t last = min(max((int64_t)a.offsets[a.experts], (int64_t)0), a.n);
    for (int64_t r = last + blockIdx.x; r < a.n; r += gridDim.x)
        for (int64_t c = threadIdx.x; c < cols; c += blockDim.x) out[r * ld + c] = V{};
}

// A choice's row, or -1
__device__ __forceinline__ int64_t row_of(const RowArgs& a, int64_t choice)
{
    const int32_t p = __ldg(a.place + choice);
    return p >= 0 && p < a.n ? p : -1;
}

// A CTA a token; V: as many bytes of a row as its alignment lets be moved at a time.
template <class V>
__global__ void __launch_bounds__(256) dispatch_kernel(const RowArgs a)
{
    V* out = static_cast<V*>(a.out);
    const V* x = static_cast<const V*>(a.x) + (int64_t)blockIdx.x * a.ld_x;
    const int64_t first = (int64_t)blockIdx.x * a.top;
    for (int64_t c0 = 0; c0 < a.cols; c0 += 4 * blockDim.x) {
        V v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = c0 + i * blockDim.x + threadIdx.x;
            if (c < a.cols) v[i] = x[c];
        }
        for (int j = 0; j < a.top; ++j) {
            const int64_t r = row_of(a, first + j);
            if (r < 0) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t c = c0 + i * blockDim.x + threadIdx.x;
                if (c < a.cols) out[r * a.ld_out + c] = v[i];
            }
        }
    }
    clear_rest(a, out, a.ld_out, a.cols);
}

// kN neighbouring elements
template <class T, int kN>
__device__ __forceinline__ void load(const T* p, float (&v)[kN])
{
    if constexpr (kN == 1) {
        v[0] = to_float(*p);
    } else if constexpr (sizeof(T) == 4) {
        static_assert(kN == 4, "16 bytes");
        const float4 f = *reinterpret_cast<const float4*>(p);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
        static_assert(kN == 8, "16 bytes");
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
template <class T, int kN>
__device__ __forceinline__ void store(T* p, const float (&v)[kN])
{
    if constexpr (kN == 1) {
        *p = from_float<T>(v[0]);
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&two);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// kN columns of a token a thread, the rows of kTogether choices on their way at once.
constexpr int kTogether = 8;
template <class T, int kN>
__global__ void __launch_bounds__(256) combine_kernel(const RowArgs a)
{
    const int64_t t = blockIdx.x, c = ((int64_t)blockIdx.y * blockDim.x + threadIdx.x) * kN;
    if (c >= a.cols) return;
    const T* rows = static_cast<const T*>(a.rows) + c;
    float sum[kN] = {};
    if (a.x) load<T, kN>(static_cast<const T*>(a.x) + t * a.ld_x + c, sum);
    float add[kN] = {};  // the residual joins last
#pragma unroll
    for (int i = 0; i < kN; ++i) add[i] = sum[i], sum[i] = 0.0f;
    for (int j0 = 0; j0 < a.top; j0 += kTogether) {
        float v[kTogether][kN], w[kTogether];
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
            w[j] = 0.0f;
#pragma unroll
            for (int i = 0; i < kN; ++i) v[j][i] = 0.0f;
            if (j0 + j >= a.top) continue;
            const int64_t r = row_of(a, t * a.top + j0 + j);
            if (r < 0) continue;
            w[j] = a.weight ? __ldg(a.weight + t * a.top + j0 + j) : 1.0f;
            load<T, kN>(rows + r * a.ld_rows, v[j]);
        }
#pragma unroll
        for (int j = 0; j < kTogether; ++j)
#pragma unroll
            for (int i = 0; i < kN; ++i) sum[i] = __fmaf_rn(w[j], v[j][i], sum[i]);
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) sum[i] += add[i];
    store<T, kN>(static_cast<T*>(a.y) + t * a.ld_y + c, sum);
}

// A CTA a token, kTogether choices at a time.
template <class T, int kN>
__global__ void __launch_bounds__(256) combine_grad_kernel(const RowArgs a)
{
    __shared__ float sums[8][kTogether];
    const int64_t t = blockIdx.x;
    const T* dy = static_cast<const T*>(a.y) + t * a.ld_y;
    const T* rows = static_cast<const T*>(a.rows);
    T* out = static_cast<T*>(a.out);
    for (int j0 = 0; j0 < a.top; j0 += kTogether) {
        float dot[kTogether] = {}, w[kTogether];
        int64_t r[kTogether];
#pragma unroll
        for (int j = 0; j < kTogether; ++j) {
            r[j] = j0 + j < a.top ? row_of(a, t * a.top + j0 + j) : -1;
            w[j] = r[j] >= 0 ? __ldg(a.weight + t * a.top + j0 + j) : 0.0f;
        }
        for (int64_t c = (int64_t)threadIdx.x * kN; c < a.cols; c += (int64_t)blockDim.x * kN) {
            float d[kN], v[kTogether][kN];
            load<T, kN>(dy + c, d);
#pragma unroll
            for (int j = 0; j < kTogether; ++j) {
                if (r[j] >= 0) {
                    load<T, kN>(rows + r[j] * a.ld_rows + c, v[j]);
                } else {
#pragma unroll
                    for (int i = 0; i < kN; ++i) v[j][i] = 0.0f;
                }
            }
#pragma unroll
            for (int j = 0; j < kTogether; ++j) {
                if (r[j] < 0) continue;
                float g[kN];
#pragma unroll
                for (int i = 0; i < kN; ++i) {
                    dot[j] = __fmaf_rn(d[i], v[j][i], dot[j]);
                    g[i] = w[j] * d[i];
                }
                store<T, kN>(out + r[j] * a.ld_out + c, g);
            }
        }
#pragma unroll
        for (int j = 0; j < kTogether; ++j)
#pragma unroll
            for (int o = 16; o; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
        __syncthreads();
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int j = 0; j < kTogether; ++j) sums[threadIdx.x >> 5][j] = dot[j];
        __syncthreads();
        if (threadIdx.x < kTogether && j0 + threadIdx.x < a.top) {
            float s = 0.0f;
            for (int q = 0; q < (int)(blockDim.x >> 5); ++q) s += sums[q][threadIdx.x];
            a.d_weight[t * a.top + j0 + threadIdx.x] = s;
        }
    }
    clear_rest(a, out, a.ld_out, a.cols);
}

int check(int64_t tokens, int64_t top, int64_t experts)
{
    if (tokens < 0 || top < 1 || top > kMostTop || experts < 1 || experts > kMostExperts || tokens > kMaxRows / top)
        return FP8Z1_EINVAL;
    return FP8Z1_OK;
}
int check(int64_t tokens, int64_t top, int64_t experts, int64_t dim, int32_t type)
{
    if (dim < 1 || dim > (int64_t)1 << 23 || (type != FP8Z1_F32 && type != FP8Z1_BF16)) return FP8Z1_EINVAL;
    return check(tokens, top, experts);
}

unsigned threads_for(int64_t vectors) { return (unsigned)std::min<int64_t>(256, std::max<int64_t>(1, ceil_div(vectors, 32)) * 32); }

template <class V>
int launch_dispatch(RowArgs a, int64_t bytes, int64_t size, cudaStream_t s)
{
    const int64_t n = (int64_t)sizeof(V);
    a.cols = bytes / n;
    a.ld_x = a.ld_x * size / n;
    a.ld_out = a.ld_out * size / n;
    count_launch();
    dispatch_kernel<V><<<(unsigned)a.tokens, threads_for(ceil_div(a.cols, 4)), 0, s>>>(a);
    return launch_status();
}

template <class T, int kN>
int launch_combine(const RowArgs& a, cudaStream_t s)
{
    const unsigned threads = threads_for(ceil_div(a.cols, kN));
    count_launch();
    combine_kernel<T, kN><<<dim3((unsigned)a.tokens, (unsigned)ceil_div(ceil_div(a.cols, kN), threads)), threads, 0, s>>>(a);
    return launch_status();
}

template <class T, int kN>
int launch_combine_grad(const RowArgs& a, cudaStream_t s)
{
    count_launch();
    combine_grad_kernel<T, kN><<<(unsigned)a.tokens, threads_for(ceil_div(a.cols, kN)), 0, s>>>(a);
    return launch_status();
}

bool fits(const void* p, int64_t ld, int64_t size, int64_t bytes) { return !p || (aligned(p, bytes) && ld * size % bytes == 0); }

}  // namespace
}  // namespace fp8z1

using namespace fp8z1;

extern "C" int fp8z1_route(const void* ids, int32_t id_bytes, int64_t tokens, int64_t top, int64_t experts,
                           int32_t* offsets, int32_t* place, void* stream)
{
    int st = check(tokens, top, experts);
    if (st != FP8Z1_OK) return st;
    const int64_t n = tokens * top;
    if (!offsets || (n && (!ids || !place)) || (id_bytes != 4 && id_bytes != 8)) return FP8Z1_EINVAL;
    if (!aligned(ids, id_bytes) || !aligned(offsets, 4) || !aligned(place, 4)) return FP8Z1_EALIGN;
    NvtxRange range("fp8z1_route");
    // one CTA up to 8192 choices, then up to 8 CTAs of 32 warps
    const int ctas = (int)std::min<int64_t>(8, std::max<int64_t>(1, ceil_div(n, 8192)));
    const int warps = ctas > 1 ? 32 : (int)std::min<int64_t>(32, std::max<int64_t>(4, ceil_div(n, 64)));
    SortArgs a = {ids, n, (int32_t)experts, 0, offsets, place};
    a.per_warp = (int32_t)(ceil_div(ceil_div(n, (int64_t)ctas * warps), 32) * 32);
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at[1] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    c.gridDim = dim3((unsigned)ctas);
    c.blockDim = dim3((unsigned)warps * 32);
    c.dynamicSmemBytes = (size_t)(warps + 1) * experts * 4;
    c.stream = static_cast<cudaStream_t>(stream);
    c.attrs = at;
    c.numAttrs = 1;
    constexpr int kMostSmem = 33 * kMostExperts * 4;
    if (!(id_bytes == 4 ? allow_smem<sort_kernel<int32_t>>(kMostSmem) : allow_smem<sort_kernel<int64_t>>(kMostSmem)))
        return FP8Z1_ECUDA;
    count_launch();
    if ((id_bytes == 4 ? cudaLaunchKernelEx(&c, sort_kernel<int32_t>, a) : cudaLaunchKernelEx(&c, sort_kernel<int64_t>, a)) !=
        cudaSuccess) {
        cudaGetLastError();
        return FP8Z1_ECUDA;
    }
    return launch_status();
}

extern "C" int fp8z1_dispatch(int64_t tokens, int64_t top, int64_t experts, int64_t dim, const void* x, int32_t type,
                              int64_t ld_x, const int32_t* offsets, const int32_t* place, void* rows, int64_t ld_rows,
                              void* stream)
{
    int st = check(tokens, top, experts, dim, type);
    if (st != FP8Z1_OK) return st;
    if (tokens == 0) return FP8Z1_OK;
    if (!x || !offsets || !place || !rows || ld_x < dim || ld_rows < dim) return FP8Z1_EINVAL;
    const int64_t size = type == FP8Z1_F32 ? 4 : 2, bytes = dim * size;
    if (!aligned(x, size) || !aligned(rows, size) || !aligned(offsets, 4) || !aligned(place, 4)) return FP8Z1_EALIGN;
    NvtxRange range("fp8z1_dispatch");
    RowArgs a = {};
    a.tokens = tokens;
    a.n = tokens * top;
    a.top = (int32_t)top;
    a.experts = (int32_t)experts;
    a.offsets = offsets;
    a.place = place;
    a.x = x;
    a.ld_x = ld_x;
    a.out = rows;
    a.ld_out = ld_rows;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto all = [&](int64_t b) { return bytes % b == 0 && fits(x, ld_x, size, b) && fits(rows, ld_rows, size, b); };
    if (all(16)) return launch_dispatch<uint4>(a, bytes, size, s);
    if (all(4)) return launch_dispatch<uint32_t>(a, bytes, size, s);
    return launch_dispatch<uint16_t>(a, bytes, size, s);
}

extern "C" int fp8z1_combine(int64_t tokens, int64_t top, int64_t dim, const void* rows, int32_t type, int64_t ld_rows,
                             const int32_t* place, const float* weight, const void* residual, int64_t ld_residual,
                             void* y, int64_t ld_y, void* stream)
{
    int st = check(tokens, top, 1, dim, type);
    if (st != FP8Z1_OK) return st;
    if (tokens == 0) return FP8Z1_OK;
    if (!rows || !place || !y || ld_rows < dim || (residual && ld_residual < dim) || ld_y < dim) return FP8Z1_EINVAL;
    const int64_t size = type == FP8Z1_F32 ? 4 : 2;
    if (!aligned(rows, size) || !aligned(residual, size) || !aligned(y, size) || !aligned(place, 4) || !aligned(weight, 4))
        return FP8Z1_EALIGN;
    NvtxRange range("fp8z1_combine");
    RowArgs a = {};
    a.tokens = tokens;
    a.n = tokens * top;
    a.top = (int32_t)top;
    a.cols = dim;
    a.place = place;
    a.weight = weight;
    a.x = residual;
    a.ld_x = ld_residual;
    a.rows = rows;
    a.ld_rows = ld_rows;
    a.y = y;
    a.ld_y = ld_y;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec = dim * size % 16 == 0 && fits(rows, ld_rows, size, 16) && fits(residual, ld_residual, size, 16) &&
                     fits(y, ld_y, size, 16);
    if (type == FP8Z1_F32) return vec ? launch_combine<float, 4>(a, s) : launch_combine<float, 1>(a, s);
    return vec ? launch_combine<bf16, 8>(a, s) : launch_combine<bf16, 1>(a, s);
}

extern "C" int fp8z1_combine_grad(int64_t tokens, int64_t top, int64_t experts, int64_t dim, const void* dy, int32_t type,
                                  int64_t ld_dy, const void* rows, int64_t ld_rows, const int32_t* offsets,
                                  const int32_t* place, const float* weight, void* d_rows, int64_t ld_d, float* d_weight,
                                  void* stream)
{
    int st = check(tokens, top, experts, dim, type);
    if (st != FP8Z1_OK) return st;
    if (tokens == 0) return FP8Z1_OK;
    if (!dy || !rows || !offsets || !place || !weight || !d_rows || !d_weight || ld_dy < dim || ld_rows < dim || ld_d < dim)
        return FP8Z1_EINVAL;
    const int64_t size = type == FP8Z1_F32 ? 4 : 2;
    if (!aligned(dy, size) || !aligned(rows, size) || !aligned(d_rows, size) || !aligned(offsets, 4) || !aligned(place, 4) ||
        !aligned(weight, 4) || !aligned(d_weight, 4))
        return FP8Z1_EALIGN;
    NvtxRange range("fp8z1_combine_grad");
    RowArgs a = {};
    a.tokens = tokens;
    a.n = tokens * top;
    a.top = (int32_t)top;
    a.experts = (int32_t)experts;
    a.cols = dim;
    a.offsets = offsets;
    a.place = place;
    a.weight = weight;
    a.rows = rows;
    a.ld_rows = ld_rows;
    a.y = const_cast<void*>(dy);
    a.ld_y = ld_dy;
    a.out = d_rows;
    a.ld_out = ld_d;
    a.d_weight = d_weight;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec = dim * size % 16 == 0 && fits(dy, ld_dy, size, 16) && fits(rows, ld_rows, size, 16) &&
                     fits(d_rows, ld_d, size, 16);
    if (type == FP8Z1_F32) return vec ? launch_combine_grad<float, 4>(a, s) : launch_combine_grad<float, 1>(a, s);
    return vec ? launch_combine_grad<bf16, 8>(a, s) : launch_combine_grad<bf16, 1>(a, s);
}
