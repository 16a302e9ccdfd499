// Root-mean-square norm of rows, the residual added first, and its gradient.
//
//   s = x + r,   rstd = (mean_j s_j^2 + eps)^-1/2,   y = s rstd w
//   in 8 bits: for 128 neighbouring columns  c = max |y| / 448 (1 if that is 0),  code = e4m3(y / c)
//   g = dy w,   h = s rstd,   dx = rstd (g - h mean_j(g_j h_j)) + d_total,   dw = sum over rows of dy h
//
// s is rounded to the rows' type, as the residual stream keeps it, and the norm is
// that of the rounded row; sums, rstd, y before its one rounding and dw are FP32.
//
// A row is held in registers from its one read on, by a warp (8 rows a CTA) or by a CTA.  All
// is bound by memory but for the smallest calls, which latency bounds.  The gradient of longer
// rows: persistent CTAs whose rows come to shared memory as bulk copies ahead of their use, as
// registers alone hold too few bytes under way (159 us for 8192 rows of 7168).
//
// With rows of 7168 BF16: 16384 with a residual to 8 bits 133 us, 6.2 TB/s; 8192 forward 66 us, 7.1 TB/s,
// their gradient 91 us, 5.2 TB/s, and 4 us for the columns' sums.  32 rows 3 us from a captured graph.  2003 rows of
// 4097 FP32, single elements: 15 and 26 us, the gradient at 3.8 TB/s, bound by its instructions.
#include <algorithm>
#include <mutex>

#include "ops_common.cuh"
#include "tc.cuh"

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

// A thread's elements of a row as they were read.
template <class T, int kE>
struct Held;
template <int kE>
struct Held<float, kE> {
    float raw[kE];
    __device__ __forceinline__ float get(int j) const { return raw[j]; }
    __device__ __forceinline__ void set(int j, float v) { raw[j] = v; }
    __device__ __forceinline__ void set8(int j, const float* p)
    {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        raw[j] = a.x, raw[j + 1] = a.y, raw[j + 2] = a.z, raw[j + 3] = a.w;
        raw[j + 4] = b.x, raw[j + 5] = b.y, raw[j + 6] = b.z, raw[j + 7] = b.w;
    }
};
template <int kE>
struct Held<bf16, kE> {
    uint32_t raw[kE / 2] = {};
    __device__ __forceinline__ float get(int j) const { return __uint_as_float(j & 1 ? raw[j / 2] & 0xffff0000u : raw[j / 2] << 16); }
    __device__ __forceinline__ void set(int j, bf16 v)
    {
        const uint32_t b = *reinterpret_cast<const unsigned short*>(&v);
        raw[j / 2] = j & 1 ? (raw[j / 2] & 0xffffu) | b << 16 : (raw[j / 2] & 0xffff0000u) | b;
    }
    __device__ __forceinline__ void set8(int j, const bf16* p)
    {
        const uint4 a = *reinterpret_cast<const uint4*>(p);
        raw[j / 2] = a.x, raw[j / 2 + 1] = a.y, raw[j / 2 + 2] = a.z, raw[j / 2 + 3] = a.w;
    }
};

// A thread's elements of a row, zeros past the end: all from p, or those of [lo, hi) from `here` in shared memory.
template <int kE, bool kVec, bool kStaged, class T>
__device__ __forceinline__ void hold(Held<T, kE>& v, const T* p, const T* here, int lo, int hi, int dim, int tid, int threads)
{
#pragma unroll
    for (int j = 0; j < kE; j += kVec ? 8 : 4) {
        const int c = column<kVec>(j, tid, threads);
        if constexpr (kVec) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v.set(j + i, from_float<T>(0.0f));
            if (c < dim) v.set8(j, (kStaged ? here : p) + c);
        } else if (kStaged && (c & ~31) >= lo && (c | 31) + 96 < hi) {  // the warp's 128
#pragma unroll
            for (int i = 0; i < 4; ++i) v.set(j + i, here[c + 32 * i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int d = c + 32 * i;
                T e = from_float<T>(0.0f);
                if (kStaged && d >= lo && d < hi)
                    e = here[d];
                else if (d < dim)
                    e = p[d];
                v.set(j + i, e);
            }
        }
    }
}

// kN neighbours (kVec: 8) or elements 32 apart from column c on, zeros past the end; and back.
template <bool kVec>
constexpr int kPiece = kVec ? 8 : 4;
template <bool kVec, class T>
__device__ __forceinline__ void load_piece(const T* p, int c, int dim, float (&v)[kPiece<kVec>])
{
    if constexpr (kVec) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        if (c < dim) load8(p + c, v);
    } else if ((c | 31) + 96 < dim) {  // the warp's 128
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = to_float(p[c + 32 * i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = c + 32 * i < dim ? to_float(p[c + 32 * i]) : 0.0f;
    }
}
template <bool kVec, class T>
__device__ __forceinline__ void store_piece(T* p, int c, int dim, const float (&v)[kPiece<kVec>])
{
    if constexpr (kVec) {
        if (c < dim) store8(p + c, v);
    } else if ((c | 31) + 96 < dim) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[c + 32 * i] = from_float<T>(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + 32 * i < dim) p[c + 32 * i] = from_float<T>(v[i]);
    }
}

// The sum of a over a row's threads, in a fixed order; every thread gets it.  `part`: a float
// for each warp of the CTA.
__device__ __forceinline__ float2 warp_sum(float2 a)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a.x += __shfl_xor_sync(0xffffffffu, a.x, o);
        a.y += __shfl_xor_sync(0xffffffffu, a.y, o);
    }
    return a;
}
template <bool kWarpRow>
__device__ __forceinline__ float row_sum(float a, float* part)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if constexpr (kWarpRow) return a;
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = a;
    __syncthreads();
    a = part[0];
    for (int w = 1; w < (int)(blockDim.x >> 5); ++w) a += part[w];
    return a;
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

// A row by a warp, or by a CTA.
template <class T, int kE, bool kVec, bool kWarpRow>
__global__ void __launch_bounds__(kWarpRow ? 256 : 1024) norm_kernel(const Args a)
{
    constexpr int kP = kPiece<kVec>;
    __shared__ float part[2][32];
    const int threads = kWarpRow ? 32 : blockDim.x, tid = kWarpRow ? threadIdx.x & 31 : threadIdx.x;
    const int64_t row = kWarpRow ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    if (kWarpRow && row >= a.rows) return;
    Held<T, kE> s;
    hold<kE, kVec, false, T>(s, static_cast<const T*>(a.x) + row * a.ld_x, nullptr, 0, 0, a.dim, tid, threads);
    if (a.r) {
        Held<T, kE> r;
        hold<kE, kVec, false, T>(r, static_cast<const T*>(a.r) + row * a.ld_r, nullptr, 0, 0, a.dim, tid, threads);
#pragma unroll
        for (int j = 0; j < kE; j += kP) {
            float v[kP];
#pragma unroll
            for (int i = 0; i < kP; ++i) s.set(j + i, from_float<T>(s.get(j + i) + r.get(j + i))), v[i] = s.get(j + i);
            store_piece<kVec>(static_cast<T*>(a.total) + row * a.ld_t, column<kVec>(j, tid, threads), a.dim, v);
        }
    }
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < kE; ++j) sum = __fmaf_rn(s.get(j), s.get(j), sum);
    sum = row_sum<kWarpRow>(sum, part[0]);
    float rstd = __frsqrt_rn(__fmaf_rn(sum, a.inv_dim, a.eps));
    if (sum > kHuge) {
        sum = 0.0f;
#pragma unroll
        for (int j = 0; j < kE; ++j) {
            const float t = s.get(j) * kShrink;
            sum = __fmaf_rn(t, t, sum);
        }
        rstd = __frsqrt_rn(row_sum<kWarpRow>(sum, part[1]) * a.inv_dim) * kShrink;
    }
    T* y = static_cast<T*>(a.y) + row * a.ld_y;
    uint8_t* codes = a.codes + row * a.dim;
    float* scales = a.scales + row * a.groups;
#pragma unroll
    for (int j = 0; j < kE; j += kP) {
        const int c = column<kVec>(j, tid, threads);
        float v[kP];
        load_piece<kVec>(a.weight, c, a.dim, v);
#pragma unroll
        for (int i = 0; i < kP; ++i) v[i] = s.get(j + i) * rstd * v[i];
        if (a.y) store_piece<kVec>(y, c, a.dim, v);
        if (!a.codes) continue;
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < kP; ++i) amax = fmaxf(amax, fabsf(v[i]));
        // of non-negative numbers, as integers: 16 lanes hold 128 columns, or all
        const uint32_t lanes = kVec ? tid & 16 ? 0xffff0000u : 0xffffu : 0xffffffffu;
        amax = __uint_as_float(__reduce_max_sync(lanes, __float_as_uint(amax)));
        // one division for the 128: an element a rounding away from the middle of two codes may take the other.
        // Below 2^-117 the reciprocal would leave FP32: such a group is 0.
        const float scale = amax >= 0x1p-117f ? __fdiv_rn(amax, 448.0f) : 1.0f, up = __frcp_rn(scale);
        if constexpr (kVec) {
            if (c >= a.dim) continue;
            if ((tid & 15) == 0) scales[c >> 7] = scale;
            uint32_t two[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) two[i] = e4m3x2(v[2 * i] * up, v[2 * i + 1] * up);
            *reinterpret_cast<uint2*>(codes + c) = make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
        } else {
            if ((tid & 31) == 0 && c < a.dim) scales[c >> 7] = scale;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c + 32 * i < a.dim) codes[c + 32 * i] = (uint8_t)e4m3x2(v[i] * up, 0.0f);
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

// dx of a row, and its part of d_weight, from what a thread holds of the normed row and dy; `w` the weight, `sums`
// adds two numbers over the row's threads, `more` d_total's elements from a column on.
template <class T, int kE, bool kVec, class F, class G>
__device__ __forceinline__ void grad_row(const GradArgs& a, int64_t row, int tid, int threads, const Held<T, kE>& s, const Held<T, kE>& d,
                                         const float* w, float (&dw)[kE], F sums, G more)
{
    constexpr int kP = kPiece<kVec>;
    auto add = [&](float by) {
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < kE; j += kP) {
            float wj[kP];
            load_piece<kVec>(w, column<kVec>(j, tid, threads), a.dim, wj);
#pragma unroll
            for (int i = 0; i < kP; ++i) {
                const float v = s.get(j + i) * by;
                sum.x = __fmaf_rn(v, v, sum.x);
                sum.y = __fmaf_rn(d.get(j + i) * wj[i], v, sum.y);
            }
        }
        return sum;
    };
    float2 sum = sums(add(1.0f), 0);
    float rstd = __frsqrt_rn(__fmaf_rn(sum.x, a.inv_dim, a.eps)), mean = sum.y * rstd * a.inv_dim;
    if (sum.x > kHuge) {  // as the norm's
        sum = sums(add(kShrink), 2);
        const float r = __frsqrt_rn(sum.x * a.inv_dim);
        rstd = r * kShrink;
        mean = sum.y * r * a.inv_dim;
    }
    T* dx = static_cast<T*>(a.dx) + row * a.ld_dx;
#pragma unroll
    for (int j = 0; j < kE; j += kP) {
        const int c = column<kVec>(j, tid, threads);
        float v[kP];
        load_piece<kVec>(w, c, a.dim, v);
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            const float h = s.get(j + i) * rstd;
            dw[j + i] = __fmaf_rn(d.get(j + i), h, dw[j + i]);
            v[i] = rstd * __fmaf_rn(-h, mean, d.get(j + i) * v[i]);
        }
        if (a.d_total) more(c, v);
        store_piece<kVec>(dx, c, a.dim, v);
    }
}

// Rows of a warp each, 8 a CTA, + 8 gridDim.x ...: the columns' sums of dy h over them stay in
// registers and are added at the end, in the order of the warps.
template <class T, int kE, bool kVec>
__global__ void __launch_bounds__(256) norm_grad_kernel(const GradArgs a)
{
    __shared__ float columns[32 * kE];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float dw[kE];
#pragma unroll
    for (int j = 0; j < kE; ++j) dw[j] = 0.0f;
    for (int64_t row = (int64_t)blockIdx.x * 8 + warp; row < a.rows; row += (int64_t)gridDim.x * 8) {
        Held<T, kE> s, d;
        hold<kE, kVec, false, T>(s, static_cast<const T*>(a.s) + row * a.ld_s, nullptr, 0, 0, a.dim, lane, 32);
        hold<kE, kVec, false, T>(d, static_cast<const T*>(a.dy) + row * a.ld_dy, nullptr, 0, 0, a.dim, lane, 32);
        grad_row<T, kE, kVec>(
            a, row, lane, 32, s, d, a.weight, dw, [](float2 v, int) { return warp_sum(v); },
            [&](int c, float(&v)[kPiece<kVec>]) {
                float t[kPiece<kVec>];
                load_piece<kVec>(static_cast<const T*>(a.d_total) + row * a.ld_t, c, a.dim, t);
#pragma unroll
                for (int i = 0; i < kPiece<kVec>; ++i) v[i] += t[i];
            });
    }
    for (int q = 0; q < 8; ++q) {
        if (warp == q)
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                const int c = column<kVec>(j, lane, 32);
                columns[c] = q ? columns[c] + dw[j] : dw[j];
            }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < a.dim; c += 256) a.part[(int64_t)blockIdx.x * a.dim + c] = columns[c];
}

// ---- longer rows: on their way through shared memory ---------------------------------------
//
// A CTA's last warp copies its rows, a row of each input a stage, as soon as a stage has been read;
// groups of the other warps take them in turn.  Bulk copies move whole 16 bytes on 16-byte
// boundaries; what a row has before its first and behind its last such boundary is read where it lies.

//
// A stage is always the same group's.  Copies come in any order: a group that took over another's stage could look
// for its second row there before the first has come, and a barrier that is a phase behind passes for filled.
//
// A wait that runs out ends its group's use of the ring: no stage is given back whose copies did not come, so
// that no barrier is filled twice; the group's dx from that row on and d_weight are NaN.  The copying thread
// leaves when all that it sent has come.

__device__ unsigned g_timeouts;
#if FP8Z1_CHECKED
__device__ unsigned g_stall;  // of the first CTA's first row, bit 0: it is never copied, 1: a warp does not give it back
#endif

constexpr int kMostStages = 16, kMostGroups = 8;
constexpr int kBarriers = 16 * kMostStages;  // bytes: full, empty [kMostStages]

struct Ring {
    const void* in[3];
    int64_t ld[3];
    int n;              // inputs
    int stages, pitch;  // pitch: bytes of a row's place; no stages: rows too long for two are read where they lie
    int groups, threads;  // threads of a group
};

template <class T>
struct Span {  // of a row's elements in whole 16 bytes
    int lo, hi;
    __device__ __forceinline__ Span(const T* p, int dim)
    {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        lo = (int)((-at & 15) / sizeof(T));
        hi = (int)((((at + dim * sizeof(T)) & ~(uintptr_t)15) - at) / sizeof(T));
        if (hi < lo) hi = lo = 0;
    }
};

// By one thread: the copies of a row's inputs to a stage, counted on its barrier.
template <class T>
__device__ __forceinline__ void fetch(const Ring& r, int64_t row, int dim, uint32_t stage, uint32_t bar)
{
    uint32_t bytes = 0;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (k >= r.n) break;
        const Span<T> s(static_cast<const T*>(r.in[k]) + row * r.ld[k], dim);
        bytes += (uint32_t)(s.hi - s.lo) * sizeof(T);
    }
    tc::bar_expect(bar, bytes);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        if (k >= r.n) break;
        const T* p = static_cast<const T*>(r.in[k]) + row * r.ld[k];
        const Span<T> s(p, dim);
        if (s.hi == s.lo) continue;
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                         stage + k * r.pitch + (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15) + (uint32_t)(s.lo * sizeof(T))),
                     "l"(p + s.lo), "r"((uint32_t)(s.hi - s.lo) * (uint32_t)sizeof(T)), "r"(bar)
                     : "memory");
    }
}

// What a thread takes of input k of the row in a stage.
template <int kE, bool kVec, class T>
__device__ __forceinline__ void take(Held<T, kE>& v, const Ring& r, const void* in, int64_t ld, int k, int64_t row, int dim,
                                     const uint8_t* stage, int tid)
{
    const T* p = static_cast<const T*>(in) + row * ld;
    const Span<T> s(p, dim);
    if (r.stages)
        hold<kE, kVec, true, T>(v, p, reinterpret_cast<const T*>(stage + k * r.pitch + (reinterpret_cast<uintptr_t>(p) & 15)), s.lo, s.hi,
                                dim, tid, r.threads);
    else
        hold<kE, kVec, false, T>(v, p, nullptr, 0, 0, dim, tid, r.threads);
}

template <class T, int kE, bool kVec, int kThreads>
__global__ void __launch_bounds__(kThreads, 1) norm_grad_ring_kernel(const GradArgs a, const Ring r)
{
    extern __shared__ __align__(128) uint8_t smem[];  // barriers, the weight, stages
    __shared__ float2 part[kMostGroups][3][32];  // 6144 bytes
    const uint32_t bar_full = tc::smem_addr(smem), bar_empty = bar_full + 8 * kMostStages;
    float* weight = reinterpret_cast<float*>(smem + kBarriers);
    uint8_t* stages = smem + kBarriers + (a.dim + 3) / 4 * 16;
    const int stage_bytes = r.n * r.pitch, warps = r.threads >> 5;
    const int group = threadIdx.x / r.threads, tid = threadIdx.x - group * r.threads;
    if (threadIdx.x == 0) {
        for (int i = 0; i < r.stages; ++i) {
            tc::bar_init(bar_full + 8 * i, 1);
            tc::bar_init(bar_empty + 8 * i, warps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    for (int c = threadIdx.x; c < a.dim; c += blockDim.x) weight[c] = a.weight[c];
    __syncthreads();
    if (group == r.groups) {
        if (tid != 0) return;
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true, again = false;  // whether every stage has been filled
        for (int64_t row = blockIdx.x; r.stages && row < a.rows; row += gridDim.x) {
            ok = tc::bar_wait(bar_empty + 8 * slot, phase ^ 1);
            if (!ok) break;  // the readers' waits run out too
#if FP8Z1_CHECKED
            if (!(g_stall & 1 && row == 0))
#endif
                fetch<T>(r, row, a.dim, tc::smem_addr(stages) + slot * stage_bytes, bar_full + 8 * slot);
            if (++slot == r.stages) slot = 0, phase ^= 1, again = true;
        }
        // the copies in flight end before the CTA does, whatever became of the readers
        for (int i = 0; i < (again ? r.stages : slot); ++i) ok &= tc::bar_wait(bar_full + 8 * i, i < slot ? phase : phase ^ 1);
        if (!ok) atomicAdd(&g_timeouts, 1u);
        return;
    }
    float dw[kE];
#pragma unroll
    for (int j = 0; j < kE; ++j) dw[j] = 0.0f;
    int slot = group, odd = 0;
    uint32_t phase = 0;
    bool lost = false;  // a wait of the group ran out
    const int rows = (int)a.rows;  // and a step more, within 2^31
    int row = blockIdx.x + group * gridDim.x;
    for (; row < rows && !lost; row += r.groups * gridDim.x) {
        const bool ok = r.stages == 0 || tc::bar_wait_warp(bar_full + 8 * slot, phase);
        if (!ok && (tid & 31) == 0) atomicAdd(&g_timeouts, 1u);
        const uint8_t* stage = stages + slot * stage_bytes;
        Held<T, kE> s, d;
        take<kE, kVec, T>(s, r, a.s, a.ld_s, 0, row, a.dim, stage, tid);
        take<kE, kVec, T>(d, r, a.dy, a.ld_dy, 1, row, a.dim, stage, tid);
        float squares = 0.0f;
        auto sums = [&](float2 v, int again) {
            v = warp_sum(v);
            if (!ok) v.x = -INFINITY;  // a copy that never came: the row becomes NaN, and no squares have this sum
            // two rows' sums lie side by side: one barrier a row
            float2* mine = part[group][again ? 2 : odd];
            if ((tid & 31) == 0) mine[tid >> 5] = v;
            asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "r"(r.threads) : "memory");
            v = mine[0];
            for (int w = 1; w < warps; ++w) v.x += mine[w].x, v.y += mine[w].y;
            squares = v.x;
            return v;
        };
        const T* more = static_cast<const T*>(a.d_total) + (int64_t)row * a.ld_t;
        const Span<T> span(more, a.dim);
        const T* here = reinterpret_cast<const T*>(stage + 2 * r.pitch + (reinterpret_cast<uintptr_t>(more) & 15));
        grad_row<T, kE, kVec>(a, row, tid, r.threads, s, d, weight, dw, sums, [&](int c, float(&v)[kPiece<kVec>]) {
            float t[kPiece<kVec>];
            if (!r.stages) {
                load_piece<kVec>(more, c, a.dim, t);
            } else if constexpr (kVec) {
                load_piece<true>(here, c, a.dim, t);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = c + 32 * i;
                    t[i] = 0.0f;
                    if (e >= span.lo && e < span.hi)
                        t[i] = to_float(here[e]);
                    else if (e < a.dim)
                        t[i] = to_float(more[e]);
                }
            }
#pragma unroll
            for (int i = 0; i < kPiece<kVec>; ++i) v[i] += t[i];
        });
        if (!(squares >= 0.0f)) {  // or the row's own NaN
            for (int w = 0; w < warps; ++w) lost |= part[group][odd][w].x < 0.0f;
            if (lost) continue;  // with the whole group, to the end
        }
        __syncwarp();
#if FP8Z1_CHECKED
        if (!(g_stall & 2 && row == 0 && tid == 0))
#endif
            if (r.stages && (tid & 31) == 0) tc::bar_arrive(bar_empty + 8 * slot);
        odd ^= 1;
        slot += r.groups;
        if (slot >= r.stages) slot -= r.stages, phase ^= 1;
    }
    for (; row < rows; row += r.groups * gridDim.x)  // what a lost group did not come to
        for (int c = tid; c < a.dim; c += r.threads) static_cast<T*>(a.dx)[(int64_t)row * a.ld_dx + c] = from_float<T>(NAN);
#pragma unroll
    for (int j = 0; j < kE; ++j) {
        const int c = column<kVec>(j, tid, r.threads);
        if (c < a.dim) a.part[((int64_t)blockIdx.x * r.groups + group) * a.dim + c] = dw[j];
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

constexpr int kWarpDim = 1024;  // up to here a warp has a row

// Threads of a CTA's row with so many elements each.
int threads_of(int64_t dim, int each) { return (int)ceil_div(dim, each * 32) * 32; }
// The gradient's ring: a CTA an SM, of 15 warps and the one that copies, for 128 registers a thread; as many elements a
// thread as they hold of three inputs and the weight's sums (groups of 28 warps at 8 elements took 120 us for 8192 rows
// of 7168 BF16, two of 14 at 16 with spilled registers 189, this 91).  Single elements 16, as 32 spill some 80 registers:
// 8192 rows of 7169 BF16 329 us, at 16 150; beyond 7680, where 15 warps no longer hold a row at 16, they take 32 all the
// same (4096 rows of 7681 BF16 189 us, of 16383 215).  19 warps and 96 registers where they hold two rows and 15 one, from
// 3585 to 4608: 2003 rows of 4097 FP32 32 us for 38, 8192 of BF16 86 for 132; single FP32 elements spill 13 registers
// there, other widths more (7169 FP32 187 for 128), or gain nothing.
constexpr int kRingSmem = 224 * 1024;
int ring_each(int64_t dim, int size, bool vec) { return dim > 7680 || (size == 2 && vec) ? 32 : 16; }
int ring_groups(int64_t dim, int each)
{
    const int threads = threads_of(dim, each);
    if (each == 16 && 480 / threads == 1 && 608 / threads == 2) return 2;
    return std::min(kMostGroups, std::max(1, 480 / threads));
}
int shape_ring(Ring& r, int64_t dim, int size, int each)  // bytes of shared memory
{
    r.threads = threads_of(dim, each);
    r.groups = ring_groups(dim, each);
    r.pitch = (int)ceil_div(dim * size + 16, 16) * 16;
    const int fixed = kBarriers + (int)ceil_div(dim, 4) * 16, stage = r.n * r.pitch;
    r.stages = std::min(kMostStages, (kRingSmem - fixed - 6144) / stage);
    r.stages -= r.stages % r.groups;  // every stage is one group's: see above
    if (r.stages < 2 || r.threads > 480) r.stages = 0;
    return fixed + r.stages * stage;
}

// Calls f.template run<T, kE, kVec>() for the types and sizes of a call.
template <int kLittle, int kMuch, class F>
int by_shape(int32_t type, bool vec, int each, F f)
{
    if (type == FP8Z1_F32)
        return each == kLittle ? (vec ? f.template run<float, kLittle, true>() : f.template run<float, kLittle, false>())
                               : (vec ? f.template run<float, kMuch, true>() : f.template run<float, kMuch, false>());
    return each == kLittle ? (vec ? f.template run<bf16, kLittle, true>() : f.template run<bf16, kLittle, false>())
                           : (vec ? f.template run<bf16, kMuch, true>() : f.template run<bf16, kMuch, false>());
}

struct WarpRows {
    const Args& a;
    cudaStream_t s;
    template <class T, int kE, bool kVec>
    int run() const
    {
        norm_kernel<T, kE, kVec, true><<<(unsigned)ceil_div(a.rows, 8), 256, 0, s>>>(a);
        return launch_status();
    }
};
struct CtaRows {
    const Args& a;
    int threads;
    cudaStream_t s;
    template <class T, int kE, bool kVec>
    int run() const
    {
        norm_kernel<T, kE, kVec, false><<<(unsigned)a.rows, threads, 0, s>>>(a);
        return launch_status();
    }
};
struct GradWarpRows {
    const GradArgs& a;
    unsigned ctas;
    cudaStream_t s;
    template <class T, int kE, bool kVec>
    int run() const
    {
        norm_grad_kernel<T, kE, kVec><<<ctas, 256, 0, s>>>(a);
        return launch_status();
    }
};
struct GradRingRows {
    const GradArgs& a;
    const Ring& r;
    int smem;
    unsigned ctas;
    cudaStream_t s;
    template <class T, int kE, bool kVec, int kThreads>
    int launch() const
    {
        if (!allow_smem<norm_grad_ring_kernel<T, kE, kVec, kThreads>>(kRingSmem - 6144)) return FP8Z1_ECUDA;
        norm_grad_ring_kernel<T, kE, kVec, kThreads><<<ctas, r.groups * r.threads + (r.stages ? 32 : 0), smem, s>>>(a, r);
        return launch_status();
    }
    template <class T, int kE, bool kVec>
    int run() const
    {
        if constexpr (kE == 16 && kVec && sizeof(T) == 2) return FP8Z1_EINVAL;  // 32 of these
        else if constexpr (kE == 16) return r.groups * r.threads > 480 ? launch<T, kE, kVec, 640>() : launch<T, kE, kVec, 512>();
        else return launch<T, kE, kVec, 512>();
    }
};

// CTAs of the gradient: as many as run at once, each with a row at least; and the rows of partial sums, at most.
int64_t grad_ctas(int64_t rows, int64_t dim)
{
    if (dim <= kWarpDim) return std::max<int64_t>(1, std::min<int64_t>(2 * kSms, ceil_div(rows, 8)));
    return std::max<int64_t>(1, std::min<int64_t>(kSms, rows));
}
int64_t grad_parts(int64_t rows, int64_t dim) { return grad_ctas(rows, dim) * (dim <= kWarpDim ? 1 : std::max(ring_groups(dim, 16), ring_groups(dim, 32))); }

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
        (residual && (ld_r < dim || ld_total < dim)) || (y && (ld_y < dim || y == total)))
        return FP8Z1_EINVAL;
    const int size = type == FP8Z1_F32 ? 4 : 2;
    if (!aligned(x, size) || !aligned(residual, size) || !aligned(total, size) || !aligned(y, size) ||
        !aligned(weight, 4) || !aligned(scales, 4))
        return FP8Z1_EALIGN;
    {
        const Area in[] = {{x, rows, dim * size, ld_x * size}, {residual, rows, dim * size, ld_r * size}};
        const Area out[] = {{total, rows, dim * size, ld_total * size}, {y, rows, dim * size, ld_y * size}};
        const Area bits[] = {dense(codes, rows * dim), dense(scales, rows * ceil_div(dim, 128) * 4)}, w = dense(weight, dim * 4);
        if (overlap(out[0], out[1]) || overlap(bits[0], bits[1])) return FP8Z1_EINVAL;
        // a row is whole in registers before its results leave, others are not
        for (int i = 0; i < 2; ++i)
            for (int j = 0; j < 2; ++j)
                if (!same_or_apart(out[i], in[j]) || overlap(bits[i], in[j]) || overlap(bits[i], out[j])) return FP8Z1_EINVAL;
        for (int i = 0; i < 2; ++i)
            if (overlap(out[i], w) || overlap(bits[i], w)) return FP8Z1_EINVAL;
    }
    NvtxRange range("fp8z1_rms_norm");
    const bool vec = dim % 8 == 0 && fits(x, ld_x, size) && fits(residual, ld_r, size) && fits(total, ld_total, size) &&
                     fits(y, ld_y, size) && aligned(weight, 16) && aligned(codes, 8);
    const Args a = {rows, (int)dim, eps, 1.0f / (float)dim, ld_x, ld_r, ld_total, ld_y, x, residual, weight, total, y,
                    codes, scales, (int)ceil_div(dim, 128)};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    count_launch();
    if (dim <= 256) return by_shape<8, 8>(type, vec, 8, WarpRows{a, s});
    // 8 elements a thread while the SMs hold all rows' threads at once, 32 beyond: us at 7168 columns, BF16 to 8 bits, 304
    // rows 4.7 (5.3 with 32), 608 7.8 (6.2), 4864 53 (42); at 1024 columns 2432 rows 4.7 (4.8), 4864 7.7 (6.5)
    if (dim <= 8192 && rows * threads_of(dim, 8) <= 2048 * kSms) return by_shape<8, 8>(type, vec, 8, CtaRows{a, threads_of(dim, 8), s});
    if (dim <= kWarpDim) return by_shape<32, 32>(type, vec, 32, WarpRows{a, s});
    return by_shape<32, 32>(type, vec, 32, CtaRows{a, threads_of(dim, 32), s});
}

extern "C" int fp8z1_rms_norm_grad_workspace(int64_t rows, int64_t dim, int64_t* bytes)
{
    if (!bytes || check(rows, dim, FP8Z1_F32, 1.0f) != FP8Z1_OK) return FP8Z1_EINVAL;
    *bytes = grad_parts(rows, dim) * dim * 4;
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
    const Area to = {dx, rows, dim * size, ld_dx * size};
    if (overlap(to, dense(weight, dim * 4)) || overlap(to, dense(d_weight, dim * 4)) ||
        !same_or_apart(to, Area{dy, rows, dim * size, ld_dy * size}) || !same_or_apart(to, Area{total, rows, dim * size, ld_total * size}) ||
        !same_or_apart(to, Area{d_total, rows, dim * size, ld_dt * size}))
        return FP8Z1_EINVAL;
    NvtxRange range("fp8z1_rms_norm_grad");
    const bool vec = dim % 8 == 0 && fits(dy, ld_dy, size) && fits(total, ld_total, size) && fits(d_total, ld_dt, size) &&
                     fits(dx, ld_dx, size) && aligned(weight, 16);
    const unsigned ctas = (unsigned)grad_ctas(rows, dim);
    const GradArgs a = {rows, (int)dim, eps, 1.0f / (float)dim, ld_dy, ld_total, ld_dt, ld_dx, dy, total, d_total, weight,
                        dx, static_cast<float*>(workspace)};
    int parts = (int)ctas;
    count_launch();
    if (dim <= kWarpDim) {
        st = by_shape<8, 32>(type, vec, dim <= 256 ? 8 : 32, GradWarpRows{a, ctas, s});
    } else {
        Ring r = {};
        r.in[0] = total;
        r.ld[0] = ld_total;
        r.in[1] = dy;
        r.ld[1] = ld_dy;
        r.in[2] = d_total;
        r.ld[2] = ld_dt;
        r.n = d_total ? 3 : 2;
        const int each = ring_each(dim, size, vec), smem = shape_ring(r, dim, size, each);
        parts *= r.groups;
        st = by_shape<16, 32>(type, vec, each, GradRingRows{a, r, smem, ctas, s});
    }
    if (st != FP8Z1_OK) return st;
    return launch_column_sum(a.part, parts, dim, d_weight, s);
}

extern "C" int fp8z1_rms_norm_timeouts(uint32_t* count)
{
    if (!count) return FP8Z1_EINVAL;
    // the devices' counters only grow, so that no count is lost between a read and a reset
    static std::mutex lock;
    static uint32_t seen[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return FP8Z1_ECUDA;
    std::lock_guard<std::mutex> hold(lock);
    unsigned n = 0;
    if (cudaMemcpyFromSymbol(&n, g_timeouts, 4) != cudaSuccess) {
        cudaGetLastError();
        return FP8Z1_ECUDA;
    }
    *count = n - seen[dev];
    seen[dev] = n;
    return FP8Z1_OK;
}

extern "C" int fp8z1_checked_rms_norm_stall(uint32_t kernels)
{
#if FP8Z1_CHECKED
    return cudaMemcpyToSymbol(g_stall, &kernels, 4) == cudaSuccess ? FP8Z1_OK : FP8Z1_ECUDA;
#else
    (void)kernels;
    return FP8Z1_EINVAL;
#endif
}
