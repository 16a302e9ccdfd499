// Root-mean-square norm of rows, the residual added first, and its gradient.
//
//   s = x + r,   rstd = (mean_j s_j^2 + eps)^-1/2,   y = s rstd w
//   in 8 bits: for 128 neighbouring columns  c = max |y| / 448 (1 if that is 0),  code = e4m3(y / c)
//   g = dy w,   h = s rstd,   dx = rstd (g - h mean_j(g_j h_j)) + d_total,   dw = sum over rows of dy h
//
// s is rounded to the rows' type, as the residual stream keeps it, and the norm is
// that of the rounded row; sums, rstd, y before its one rounding and dw are FP32.
//
// A row is held in registers from its one read on: a warp's (8 rows a CTA) up to 1024
// columns, a CTA's beyond.  Few rows are spread over more threads (8 elements each
// for 32), as latency counts there.
#include <algorithm>

#include "ops_common.cuh"

namespace fp8z1 {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kMostDim = 16384;

// Element j of a thread's kE.  Vectors: 8 neighbours, a warp's 256 in a row; 16 lanes
// hold 128 columns.  Single elements: 128 columns are a warp's elements 4i .. 4i + 3.
template <bool kVec>
__device__ __forceinline__ int column(int j, int tid, int threads)
{
    if (kVec) return ((j >> 3) * threads + tid) * 8 + (j & 7);
    return ((j >> 2) * (threads >> 5) + (tid >> 5)) * 128 + (j & 3) * 32 + (tid & 31);
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8])
{
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void load8(const bf16* p, float (&v)[8])
{
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float* v)
{
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(bf16* p, const float* v)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&two);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// A thread's elements of a row (0 past its end), and back.
template <int kE, bool kVec, class T>
__device__ __forceinline__ void load_row(const T* p, int dim, int tid, int threads, float (&v)[kE])
{
    if constexpr (kVec) {
#pragma unroll
        for (int j = 0; j < kE; j += 8) {
            const int c = column<true>(j, tid, threads);
            float t[8] = {};
            if (c < dim) load8(p + c, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[j + i] = t[i];
        }
    } else {
#pragma unroll
        for (int j = 0; j < kE; ++j) {
            const int c = column<false>(j, tid, threads);
            v[j] = c < dim ? to_float(p[c]) : 0.0f;
        }
    }
}
template <int kE, bool kVec, class T>
__device__ __forceinline__ void store_row(T* p, int dim, int tid, int threads, const float (&v)[kE])
{
#pragma unroll
    for (int j = 0; j < kE; j += kVec ? 8 : 1) {
        const int c = column<kVec>(j, tid, threads);
        if (c >= dim) continue;
        if constexpr (kVec)
            store8(p + c, &v[j]);
        else
            p[c] = from_float<T>(v[j]);
    }
}

// The sums of a and b over a row's threads, in a fixed order; every thread gets them.
// `part`: two floats for each warp; a CTA's next use of it is a barrier away.
template <bool kWarpRow>
__device__ __forceinline__ float2 row_sum(float a, float b, float2* part)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (kWarpRow) return make_float2(a, b);
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) part[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const float2 mine = lane < warps ? part[lane] : make_float2(0.0f, 0.0f);
    a = mine.x, b = mine.y;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    return make_float2(a, b);
}

// The squares of numbers beyond 2^60 or so leave FP32 in a sum of 16384.  Such a row is
// summed again 2^-80 times as large (eps, at most 2^66 by then, is nothing beside it).
constexpr float kHuge = 1.0e37f, kShrink = 0x1p-80f;

struct Args {
    int64_t rows;
    int dim;
    float eps, inv_dim;
    int64_t ld_x, ld_r, ld_t, ld_y;
    const void *x, *r;
    const float* weight;
    void *total, *y;
    uint8_t* codes;
    float* scales;
    int groups;  // of 128 columns
};

template <class T, int kE, bool kVec, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 256 : kE == 8 ? 1024 : 512) norm_kernel(const Args a)
{
    __shared__ float2 part[32];
    const int threads = kWarpRow ? 32 : blockDim.x, tid = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = kWarpRow ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    if (kWarpRow && row >= a.rows) return;
    float v[kE];
    load_row<kE, kVec>(static_cast<const T*>(a.x) + row * a.ld_x, a.dim, tid, threads, v);
    if (a.r) {
        float r[kE];
        load_row<kE, kVec>(static_cast<const T*>(a.r) + row * a.ld_r, a.dim, tid, threads, r);
#pragma unroll
        for (int j = 0; j < kE; ++j) v[j] = to_float(from_float<T>(v[j] + r[j]));
        store_row<kE, kVec>(static_cast<T*>(a.total) + row * a.ld_t, a.dim, tid, threads, v);
    }
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kE; ++j) sum = __fmaf_rn(v[j], v[j], sum);
    sum = row_sum<kWarpRow>(sum, 0.0f, part).x;
    float rstd = __frsqrt_rn(__fmaf_rn(sum, a.inv_dim, a.eps));
    if (sum > kHuge) {
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < kE; ++j) {
            const float t = v[j] * kShrink;
            sum = __fmaf_rn(t, t, sum);
        }
        rstd = __frsqrt_rn(row_sum<kWarpRow>(sum, 0.0f, part).x * a.inv_dim) * kShrink;
    }
    {
        float w[kE];
        load_row<kE, kVec>(a.weight, a.dim, tid, threads, w);
#pragma unroll
        for (int j = 0; j < kE; ++j) v[j] = v[j] * rstd * w[j];
    }
    if (a.y) store_row<kE, kVec>(static_cast<T*>(a.y) + row * a.ld_y, a.dim, tid, threads, v);
    if (!a.codes) return;
    uint8_t* codes = a.codes + row * a.dim;
    float* scales = a.scales + row * a.groups;
    constexpr int kPart = kVec ? 8 : 4;
#pragma unroll
    for (int j = 0; j < kE; j += kPart) {
        const int c = column<kVec>(j, tid, threads);
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < kPart; ++i) amax = fmaxf(amax, fabsf(v[j + i]));
#pragma unroll
        for (int o = kVec ? 8 : 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        float scale = __fdiv_rn(amax, 448.0f);
        if (scale == 0.0f) scale = 1.0f;
        if constexpr (kVec) {
            if (c >= a.dim) continue;
            if ((tid & 15) == 0) scales[c >> 7] = scale;
            uint32_t two[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                two[i] = e4m3x2(__fdiv_rn(v[j + 2 * i], scale), __fdiv_rn(v[j + 2 * i + 1], scale));
            *reinterpret_cast<uint2*>(codes + c) = make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
        } else {
            if ((tid & 31) == 0 && c < a.dim) scales[c >> 7] = scale;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + 32 * i < a.dim) codes[c + 32 * i] = (uint8_t)e4m3x2(__fdiv_rn(v[j + i], scale), 0.0f);
        }
    }
}

struct GradArgs {
    int64_t rows;
    int dim;
    float eps, inv_dim;
    int64_t ld_dy, ld_s, ld_t, ld_dx;
    const void *dy, *s, *d_total;
    const float* weight;
    void* dx;
    float* part;  // [CTAs, dim]
};

// dx of rows blockIdx.x, + gridDim.x, ...; the columns' sums of dy h over them stay in
// registers and are written at the end (of 8 warps' rows in their order).
template <class T, int kE, bool kVec, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 256 : 512) norm_grad_kernel(const GradArgs a)
{
    __shared__ float2 part[32];
    __shared__ float columns[kWarpRow ? 32 * kE : 1];
    const int threads = kWarpRow ? 32 : blockDim.x, tid = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
    const int64_t first = kWarpRow ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    const int64_t step = (int64_t)gridDim.x * (kWarpRow ? 8 : 1);
    float dw[kE];
#pragma unroll
    for (int j = 0; j < kE; ++j) dw[j] = 0.0f;
    for (int64_t row = first; row < a.rows; row += step) {
        float v[kE], d[kE], w[kE];
        load_row<kE, kVec>(static_cast<const T*>(a.s) + row * a.ld_s, a.dim, tid, threads, v);
        load_row<kE, kVec>(static_cast<const T*>(a.dy) + row * a.ld_dy, a.dim, tid, threads, d);
        load_row<kE, kVec>(a.weight, a.dim, tid, threads, w);
        float sum = 0.0f, dot = 0.0f;
#pragma unroll
        for (int j = 0; j < kE; ++j) {
            sum = __fmaf_rn(v[j], v[j], sum);
            dot = __fmaf_rn(d[j] * w[j], v[j], dot);
        }
        const float2 both = row_sum<kWarpRow>(sum, dot, part);
        float rstd = __frsqrt_rn(__fmaf_rn(both.x, a.inv_dim, a.eps)), mean = both.y * rstd * a.inv_dim;
        if (both.x > kHuge) {  // as the norm's
            sum = dot = 0.0f;
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                const float t = v[j] * kShrink;
                sum = __fmaf_rn(t, t, sum);
                dot = __fmaf_rn(d[j] * w[j], t, dot);
            }
            const float2 again = row_sum<kWarpRow>(sum, dot, part);
            const float r = __frsqrt_rn(again.x * a.inv_dim);
            rstd = r * kShrink;
            mean = again.y * r * a.inv_dim;
        }
#pragma unroll
        for (int j = 0; j < kE; ++j) {
            const float h = v[j] * rstd;
            dw[j] = __fmaf_rn(d[j], h, dw[j]);
            v[j] = rstd * __fmaf_rn(-h, mean, d[j] * w[j]);
        }
        if (a.d_total) {
            load_row<kE, kVec>(static_cast<const T*>(a.d_total) + row * a.ld_t, a.dim, tid, threads, d);
#pragma unroll
            for (int j = 0; j < kE; ++j) v[j] += d[j];
        }
        store_row<kE, kVec>(static_cast<T*>(a.dx) + row * a.ld_dx, a.dim, tid, threads, v);
    }
    float* out = a.part + (int64_t)blockIdx.x * a.dim;
    if constexpr (kWarpRow) {
        for (int q = 0; q < 8; ++q) {
            if (threadIdx.x >> 5 == q)
#pragma unroll
                for (int j = 0; j < kE; ++j) {
                    const int c = column<kVec>(j, tid, 32);
                    columns[c] = q ? columns[c] + dw[j] : dw[j];
                }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.dim; c += 256) out[c] = columns[c];
    } else {
        store_row<kE, kVec>(out, a.dim, tid, threads, dw);
    }
}

// The sums of `n` rows of partial sums: 32 columns a CTA, 32 threads a column, in a fixed order.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part, int n, int64_t dim, float* out)
{
    __shared__ float sums[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t c0 = (int64_t)blockIdx.x * 32, c = c0 + x;
    float s = 0.0f;
    if (c < dim)
#pragma unroll 8
        for (int i = y; i < n; i += 32) s += part[i * dim + c];
    sums[y][x] = s;
    __syncthreads();
    s = sums[x][y];  // the warp's column
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (x == 0 && c0 + y < dim) out[c0 + y] = s;
}

int check(int64_t rows, int64_t dim, int32_t type, float eps)
{
    if (rows < 0 || rows > kMaxRows || dim < 1 || dim > kMostDim || (type != FP8Z1_F32 && type != FP8Z1_BF16) ||
        !(eps >= 1e-20f && eps <= 1e20f))
        return FP8Z1_EINVAL;
    return FP8Z1_OK;
}

// Whether a buffer's rows can be taken 8 elements at a time.
bool fits(const void* p, int64_t ld, int size) { return !p || (aligned(p, 16) && ld * size % 16 == 0); }

// Threads of a row with 8 or 32 elements each.
int threads_of(int64_t dim, int each)
{
    int t = 32;
    while ((int64_t)t * each < dim) t *= 2;
    return t;
}

template <template <class, int, bool, bool> class F, class... A>
int by_shape(int32_t type, bool vec, int each, bool warp, const A&... args)
{
#define FP8Z1_CASE(T, E, V, W) \
    if (each == E && vec == V && warp == W) return F<T, E, V, W>::run(args...);
#define FP8Z1_CASES(T) \
    FP8Z1_CASE(T, 8, true, true) FP8Z1_CASE(T, 8, true, false) FP8Z1_CASE(T, 8, false, true) \
    FP8Z1_CASE(T, 8, false, false) FP8Z1_CASE(T, 32, true, true) FP8Z1_CASE(T, 32, true, false) \
    FP8Z1_CASE(T, 32, false, true) FP8Z1_CASE(T, 32, false, false)
    if (type == FP8Z1_F32) {
        FP8Z1_CASES(float)
    } else {
        FP8Z1_CASES(bf16)
    }
#undef FP8Z1_CASES
#undef FP8Z1_CASE
    return FP8Z1_EINVAL;
}

template <class T, int kE, bool kVec, bool kWarpRow>
struct Norm {
    static int run(const Args& a, int threads, cudaStream_t s)
    {
        count_launch();
        if (kWarpRow)
            norm_kernel<T, kE, kVec, true><<<(unsigned)ceil_div(a.rows, 8), 256, 0, s>>>(a);
        else
            norm_kernel<T, kE, kVec, false><<<(unsigned)a.rows, threads, 0, s>>>(a);
        return launch_status();
    }
};

template <class T, int kE, bool kVec, bool kWarpRow>
struct Grad {
    static int run(const GradArgs& a, int threads, unsigned ctas, cudaStream_t s)
    {
        count_launch();
        if constexpr (!kWarpRow && kE == 8)
            return FP8Z1_EINVAL;  // not called: the gradient takes 32 elements a thread beyond a warp's
        else
            norm_grad_kernel<T, kE, kVec, kWarpRow><<<ctas, kWarpRow ? 256 : threads, 0, s>>>(a);
        return launch_status();
    }
};

// CTAs of the gradient: as many as run at once, each with a row at least.
int64_t grad_ctas(int64_t rows, int64_t dim)
{
    const int threads = threads_of(dim, 32);
    const int64_t most = (int64_t)kSms * (threads == 32 ? 2 : std::max(1, 512 / threads));
    return std::max<int64_t>(1, std::min(most, threads == 32 ? ceil_div(rows, 8) : rows));
}

}  // namespace

int launch_column_sum(const float* part, int n, int64_t cols, float* out, cudaStream_t s)
{
    count_launch();
    column_sum_kernel<<<(unsigned)ceil_div(cols, 32), 1024, 0, s>>>(part, n, cols, out);
    return launch_status();
}

}  // namespace fp8z1

using namespace fp8z1;

extern "C" int fp8z1_rms_norm(int64_t rows, int64_t dim, const void* x, int32_t type, int64_t ld_x,
                              const void* residual, int64_t ld_r, const float* weight, float eps, void* total,
                              int64_t ld_total, void* y, int64_t ld_y, uint8_t* codes, float* scales, void* stream)
{
    int st = check(rows, dim, type, eps);
    if (st != FP8Z1_OK) return st;
    if (rows == 0) return FP8Z1_OK;
    if (!x || !weight || (!y && !codes) || !codes != !scales || !residual != !total || ld_x < dim ||
        (residual && (ld_r < dim || ld_total < dim)) || (y && ld_y < dim))
        return FP8Z1_EINVAL;
    const int size = type == FP8Z1_F32 ? 4 : 2;
    if (!aligned(x, size) || !aligned(residual, size) || !aligned(total, size) || !aligned(y, size) ||
        !aligned(weight, 4) || !aligned(scales, 4))
        return FP8Z1_EALIGN;
    NvtxRange range("fp8z1_rms_norm");
    const bool vec = dim % 8 == 0 && fits(x, ld_x, size) && fits(residual, ld_r, size) && fits(total, ld_total, size) &&
                     fits(y, ld_y, size) && aligned(weight, 16) && aligned(codes, 8);
    int each = 32, threads = threads_of(dim, 32);
    if (dim <= 8192 && rows * threads < kSms * 512) each = 8, threads = threads_of(dim, 8);
    const Args a = {rows, (int)dim, eps, 1.0f / (float)dim, ld_x, ld_r, ld_total, ld_y, x, residual, weight, total, y,
                    codes, scales, (int)ceil_div(dim, 128)};
    return by_shape<Norm>(type, vec, each, threads == 32, a, threads, static_cast<cudaStream_t>(stream));
}

extern "C" int fp8z1_rms_norm_grad_workspace(int64_t rows, int64_t dim, int64_t* bytes)
{
    if (!bytes || check(rows, dim, FP8Z1_F32, 1.0f) != FP8Z1_OK) return FP8Z1_EINVAL;
    *bytes = grad_ctas(rows, dim) * dim * 4;
    return FP8Z1_OK;
}

extern "C" int fp8z1_rms_norm_grad(int64_t rows, int64_t dim, const void* dy, int32_t type, int64_t ld_dy,
                                   const void* total, int64_t ld_total, const float* weight, float eps,
                                   const void* d_total, int64_t ld_dt, void* dx, int64_t ld_dx, float* d_weight,
                                   void* workspace, void* stream)
{
    int st = check(rows, dim, type, eps);
    if (st != FP8Z1_OK) return st;
    if (!d_weight) return FP8Z1_EINVAL;
    if (!aligned(d_weight, 4)) return FP8Z1_EALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (rows == 0) return cudaMemsetAsync(d_weight, 0, (size_t)dim * 4, s) == cudaSuccess ? FP8Z1_OK : FP8Z1_ECUDA;
    if (!dy || !total || !weight || !dx || !workspace || ld_dy < dim || ld_total < dim || ld_dx < dim ||
        (d_total && ld_dt < dim))
        return FP8Z1_EINVAL;
    const int size = type == FP8Z1_F32 ? 4 : 2;
    if (!aligned(dy, size) || !aligned(total, size) || !aligned(d_total, size) || !aligned(dx, size) ||
        !aligned(weight, 4) || !aligned(workspace, 256))
        return FP8Z1_EALIGN;
    NvtxRange range("fp8z1_rms_norm_grad");
    const bool vec = dim % 8 == 0 && fits(dy, ld_dy, size) && fits(total, ld_total, size) && fits(d_total, ld_dt, size) &&
                     fits(dx, ld_dx, size) && aligned(weight, 16);
    const int threads = threads_of(dim, 32);
    const int each = dim <= 256 ? 8 : 32;
    const unsigned ctas = (unsigned)grad_ctas(rows, dim);
    const GradArgs a = {rows, (int)dim, eps, 1.0f / (float)dim, ld_dy, ld_total, ld_dt, ld_dx, dy, total, d_total, weight,
                        dx, static_cast<float*>(workspace)};
    if ((st = by_shape<Grad>(type, vec, each, threads == 32, a, threads, ctas, s)) != FP8Z1_OK) return st;
    return launch_column_sum(a.part, (int)ctas, dim, d_weight, s);
}
