// Matrix product with an FP8 weight: entry points, and the kernels that bring rows to the
// tensor cores' types (linear_gemm.cu: the products; linear_wgrad.cu: the weight's gradient).
//
// Forward:  pairs of BF16 rows (8-bit rows go as they are), product.
// Backward: dz = dy act'(z) to pairs, its columns' sums; dx, a product with the weight turned;
//           d_weight, of dy and x as they lie when dz is dy in BF16, else of FP16 terms.
//
// 2051 rows of 4096 to 14336 with a bias, GELU and z saved: pairs 9 us and product 202; dz 96, dx 161, x's FP16 terms
// (24 for 2048 rows of 7168; they start when dx has ended), d_weight 306, the bias's gradient 4.
#include <cooperative_groups.h>

#include <mutex>

#include "linear.cuh"

namespace fp8z1 {
namespace linear {
namespace {

namespace cg = cooperative_groups;
using ffn::after_previous;
using ffn::ColumnScale;
using ffn::Cut;
using ffn::next_may_start;
using ffn::pair_encode;
using ffn::pair_scale;
using ffn::PairScale;

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t half_pair(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// kN neighbours of a row from column c on, zeros past its end.
template <int kN>
__device__ __forceinline__ void load_some(const bf16* p, int64_t c, int64_t cols, bool vec, float (&v)[kN])
{
    if (vec && c + kN <= cols) {
        uint32_t w[kN / 2];
        if constexpr (kN == 8) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(p + c));
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
        } else {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(p + c));
            w[0] = u.x, w[1] = u.y;
        }
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kN; ++i) v[i] = c + i < cols ? to_float(p[c + i]) : 0.0f;
    }
}
__device__ __forceinline__ void load_some(const float* p, int64_t c, int64_t cols, bool vec, float (&v)[4])
{
    if (vec && c + 4 <= cols) {
        const float4 u = __ldg(reinterpret_cast<const float4*>(p + c));
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = c + i < cols ? p[c + i] : 0.0f;
    }
}

// Rows of BF16 to FP8 pairs, a warp 1024 columns of a row, all of its loads on their way
// before the first is needed; 16 lanes have a block of 128.
constexpr int kRowColumns = 1024;
__global__ void __launch_bounds__(256) split_kernel(const bf16* x, int64_t ld, int64_t T, int64_t cols, int64_t pitch, bool vec,
                                                    uint8_t* hi, uint8_t* lo, float* scale)
{
    next_may_start();
    const int lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (row >= T) return;
    const bf16* src = x + row * ld;
    constexpr int kLoads = kRowColumns / 256;
    float v[kLoads][8];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int64_t c = (int64_t)blockIdx.y * kRowColumns + i * 256 + lane * 8;
        load_some<8>(src, c, cols, vec, v[i]);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int64_t c = (int64_t)blockIdx.y * kRowColumns + i * 256 + lane * 8;
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[i][j]));
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (c >= pitch) continue;
        const PairScale ps = pair_scale(amax);
        uint32_t h[4], l[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) pair_encode<Lo::kE5M2>(v[i][2 * j], v[i][2 * j + 1], ps.up, h[j], l[j]);
        *reinterpret_cast<uint2*>(hi + row * pitch + c) = make_uint2(h[0] | h[1] << 16, h[2] | h[3] << 16);
        *reinterpret_cast<uint2*>(lo + row * pitch + c) = make_uint2(l[0] | l[1] << 16, l[2] | l[3] << 16);
        if ((lane & 15) == 0) scale[c / kBlock * T + row] = ps.down;
    }
}

struct DzArgs {
    const void *dy;
    const float* pre;
    int64_t ld, T, N, Np;
    int32_t act;
    bool vec_dy, vec_pre;
    Backward b;  // what is not wanted is NULL
};

// dz of 128 rows x 128 columns, a warp 8 rows and a lane 4 columns of each, in registers
// from its one read on: pairs for dx (a row's 128 share a scale), FP16 terms for d_weight
// (a column's 256 do: two CTAs tell each other their largest), the columns' sums.  The terms: a
// column's largest number is brought to 2^14, so that columns of small numbers keep their 22
// bits beside large ones.  2051 rows of 14336 with an activation take 96 us, 3.6 TB/s (256 rows by a CTA of 1024
// threads, which loads and stores by turns, 123); its 64 registers spill 15 of BF16 dy's.
constexpr int kDzRows = kTall / 2;
template <class D, bool kAct, bool kTerms>
__global__ void __launch_bounds__(512, 2) dz_kernel(const DzArgs a)
{
    constexpr bool kExact = !kTerms;  // BF16 values
    __shared__ uint32_t peaks[2][128];  // of this CTA's rows, of the other's
    __shared__ float sums[16][128];
    next_may_start();
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r0 = (int64_t)blockIdx.x * kDzRows + warp * 8, c = (int64_t)blockIdx.y * 128 + lane * 4;
    const bool terms = kTerms && a.b.dz_hi;
    if (terms) {
        if (threadIdx.x < 128) peaks[0][threadIdx.x] = 0;
        cluster.barrier_arrive();  // this CTA has started: the other may write to it
    }
    float v[8][4];
    if (kAct && sizeof(D) == 2 && a.vec_dy && a.vec_pre) {
        // dy waits in its own 16 bits, so that the registers hold all rows' loads at once
        uint2 d[8];
        const bool in = c < a.N;  // rows of whole fours
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const bool here = in && r0 + r < a.T;
            d[r] = here ? __ldg(reinterpret_cast<const uint2*>(static_cast<const bf16*>(a.dy) + (r0 + r) * a.ld + c)) : make_uint2(0, 0);
            const float4 z = here ? __ldg(reinterpret_cast<const float4*>(a.pre + (r0 + r) * a.N + c)) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            v[r][0] = z.x, v[r][1] = z.y, v[r][2] = z.z, v[r][3] = z.w;
        }
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            v[r][0] = __uint_as_float(d[r].x << 16) * slope(v[r][0], a.act);
            v[r][1] = __uint_as_float(d[r].x & 0xffff0000u) * slope(v[r][1], a.act);
            v[r][2] = __uint_as_float(d[r].y << 16) * slope(v[r][2], a.act);
            v[r][3] = __uint_as_float(d[r].y & 0xffff0000u) * slope(v[r][3], a.act);
        }
    } else {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[r][j] = 0.0f;
            if (r0 + r < a.T) load_some(static_cast<const D*>(a.dy) + (r0 + r) * a.ld, c, a.N, a.vec_dy, v[r]);
        }
        if (kAct)
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                float z[4] = {};
                if (r0 + r < a.T) load_some(a.pre + (r0 + r) * a.N, c, a.N, a.vec_pre, z);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[r][j] *= slope(z[j], a.act);
            }
    }
    if (a.b.hi)
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (r0 + r >= a.T) break;
            const float amax = fmaxf(fmaxf(fabsf(v[r][0]), fabsf(v[r][1])), fmaxf(fabsf(v[r][2]), fabsf(v[r][3])));
            // FP32 dz in two E4M3 terms: 9 bits, one more than a BF16 gradient would hand to dx's product, and dx is off by
            // 1.8e-3 of its norm (its own rounding 1.66e-3).  A third term would make that product half as long again.
            const PairScale ps = pair_scale(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax))));
            uint32_t h0, l0, h1, l1;
            pair_encode<kExact ? Lo::kE5M2 : Lo::kE4M3>(v[r][0], v[r][1], ps.up, h0, l0);
            pair_encode<kExact ? Lo::kE5M2 : Lo::kE4M3>(v[r][2], v[r][3], ps.up, h1, l1);
            *reinterpret_cast<uint32_t*>(a.b.hi + (r0 + r) * a.Np + c) = h0 | h1 << 16;
            *reinterpret_cast<uint32_t*>(a.b.lo + (r0 + r) * a.Np + c) = l0 | l1 << 16;
            if (lane == 0) a.b.scale[(int64_t)blockIdx.y * a.T + r0 + r] = ps.down;
        }
    if (a.b.part) {
        float s[4] = {};
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += v[r][j];
        *reinterpret_cast<float4*>(&sums[warp][lane * 4]) = make_float4(s[0], s[1], s[2], s[3]);
    }
    if (terms) {
        __syncwarp();
        cluster.barrier_wait();
        uint32_t p[4] = {};
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = max(p[j], abs_bits(v[r][j]));
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) atomicMax(&peaks[0][lane * 4 + j], p[j]);  // the order leaves the largest as it is
    }
    __syncthreads();
    if (terms && threadIdx.x < 128) cluster.map_shared_rank(&peaks[1][0], (int)cluster.block_rank() ^ 1)[threadIdx.x] = peaks[0][threadIdx.x];
    if (a.b.part && threadIdx.x < 128) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 16; ++w) s += sums[w][threadIdx.x];
        const int64_t col = (int64_t)blockIdx.y * 128 + threadIdx.x;
        if (col < a.N) a.b.part[(int64_t)blockIdx.x * a.N + col] = s;
    }
    if (!terms) return;
    __syncwarp();
    cluster.sync();
    float up[4], down[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const ColumnScale s = ffn::column_scale(max(peaks[0][lane * 4 + j], peaks[1][lane * 4 + j]) >> 23);
        up[j] = s.up, down[j] = s.down;
    }
    if (warp == 0 && !(blockIdx.x & 1))
        *reinterpret_cast<float4*>(a.b.dz_factor + (int64_t)(blockIdx.x >> 1) * a.Np + c) = make_float4(down[0], down[1], down[2], down[3]);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        if (r0 + r >= a.T) break;
        const int64_t at = (r0 + r) * a.Np + c;
        const float f0 = v[r][0] * up[0], f1 = v[r][1] * up[1], f2 = v[r][2] * up[2], f3 = v[r][3] * up[3];
        const __half2 h0 = __floats2half2_rn(f0, f1), h1 = __floats2half2_rn(f2, f3);
        const float2 g0 = __half22float2(h0), g1 = __half22float2(h1);
        *reinterpret_cast<uint2*>(a.b.dz_hi + at) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
        *reinterpret_cast<uint2*>(a.b.dz_lo + at) = make_uint2(half_pair(f0 - g0.x, f1 - g0.y), half_pair(f2 - g1.x, f3 - g1.y));
    }
}

// x of 256 rows x 128 columns to FP16, the largest finite number of them brought to 2^14: a BF16
// number is held whole down to 2^-31 of it.
__global__ void __launch_bounds__(1024) x16_kernel(const bf16* x, int64_t ld, int64_t T, int64_t cols, int64_t pitch, bool vec,
                                                   __half* out, float* factor)
{
    __shared__ uint32_t peak;
    next_may_start();
    after_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r0 = (int64_t)blockIdx.x * kTall + warp * 8, c = (int64_t)blockIdx.y * 128 + lane * 4;
    if (threadIdx.x == 0) peak = 0;
    float v[8][4];
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[r][j] = 0.0f;
        if (r0 + r < T) load_some<4>(x + (r0 + r) * ld, c, cols, vec, v[r]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t b = abs_bits(v[r][j]);
            if (b < 0x7f800000u) top = max(top, b);
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    __syncthreads();
    if (lane == 0) atomicMax(&peak, top);
    __syncthreads();
    const int e = ffn::peak_exponent(peak);
    const ffn::Pow2 up = ffn::pow2(14 - e);
    if (threadIdx.x == 0) factor[(int64_t)blockIdx.x * (pitch / 128) + blockIdx.y] = ffn::peak_factor(peak);
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        if (r0 + r >= T) break;
        *reinterpret_cast<uint2*>(out + (r0 + r) * pitch + c) =
            make_uint2(half_pair(up.times(v[r][0]), up.times(v[r][1])), half_pair(up.times(v[r][2]), up.times(v[r][3])));
    }
}

// Rows to ones that lie on 16 bytes.
__global__ void __launch_bounds__(256) copy_kernel(const bf16* from, int64_t ld, int64_t cols, bf16* to, int64_t pitch)
{
    next_may_start();
    after_previous();
    for (int64_t c = threadIdx.x; c < pitch; c += 256)
        to[blockIdx.x * pitch + c] = c < cols ? from[blockIdx.x * ld + c] : __float2bfloat16_rn(0.0f);
}

struct Dims {
    int64_t T, R, C;
    bool k_major;  // the weight is [N, K]
    int32_t act, x_type, y_type;
    int64_t K() const { return k_major ? C : R; }
    int64_t N() const { return k_major ? R : C; }
    int64_t Kp() const { return ceil_div(K(), 128) * 128; }
    int64_t Np() const { return ceil_div(N(), 128) * 128; }
    bool exact() const { return act == FP8Z1_ACT_NONE && y_type == FP8Z1_BF16; }  // dz is dy in BF16
};

struct Forward {
    uint8_t *hi, *lo;
    float* scale;
    void cut(Cut& c, const Dims& d)
    {
        if (d.x_type != FP8Z1_BF16) return;
        hi = c.take<uint8_t>(d.T * d.Kp());
        lo = c.take<uint8_t>(d.T * d.Kp());
        scale = c.take<float>(d.T * (d.Kp() / 128));
    }
};

void cut(Backward& b, Cut& c, const Dims& d)
{
    const int64_t tall = ceil_div(d.T, kTall), Np = d.Np(), Kp = d.Kp();
    b = Backward{};
    b.hi = c.take<uint8_t>(d.T * Np);
    b.lo = c.take<uint8_t>(d.T * Np);
    b.scale = c.take<float>(d.T * (Np / 128));
    b.part = c.take<float>(2 * tall * d.N());
    if (d.exact()) {
        b.x_copy = c.take<bf16>(d.T * Kp);
        b.dy_copy = c.take<bf16>(d.T * Np);
    } else {
        b.dz_hi = c.take<__half>(d.T * Np);
        b.dz_lo = c.take<__half>(d.T * Np);
        b.dz_factor = c.take<float>(tall * Np);
        b.x16 = c.take<__half>(d.T * Kp);
        b.x_factor = c.take<float>(tall * (Kp / 128));
    }
}

int check(const fp8z1_linear_dims* p, Dims& d)
{
    if (!p || p->tokens < 0 || p->tokens > kMaxRows || p->rows < 1 || p->rows > (int64_t)1 << 22 || p->cols < 16 ||
        p->cols % 16 || p->cols > (int64_t)1 << 22 || (p->transposed != 0 && p->transposed != 1) ||
        p->activation < FP8Z1_ACT_NONE || p->activation > FP8Z1_ACT_GELU_TANH ||
        (p->x_type != FP8Z1_BF16 && p->x_type != FP8Z1_E4M3) || (p->y_type != FP8Z1_F32 && p->y_type != FP8Z1_BF16))
        return FP8Z1_EINVAL;
    d = Dims{p->tokens, p->rows, p->cols, p->transposed == 1, p->activation, p->x_type, p->y_type};
    return FP8Z1_OK;
}

// The first kernel of its pass, in clusters of two.
int launch_dz(void (*kernel)(DzArgs), dim3 grid, cudaStream_t s, const DzArgs& a)
{
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at[1] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    c.gridDim = grid;
    c.blockDim = dim3(512);
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 1;
    count_launch();
    if (cudaLaunchKernelEx(&c, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return FP8Z1_ECUDA;
    }
    return launch_status();
}

bool on16(const void* p, int64_t ld, int size) { return aligned(p, 16) && ld * size % 16 == 0; }

}  // namespace
}  // namespace linear
}  // namespace fp8z1

using namespace fp8z1;
using namespace fp8z1::linear;

extern "C" int fp8z1_linear_sizes(const fp8z1_linear_dims* dims, int64_t* forward_bytes, int64_t* backward_bytes)
{
    Dims d;
    const int st = check(dims, d);
    if (st != FP8Z1_OK) return st;
    if (!forward_bytes || !backward_bytes) return FP8Z1_EINVAL;
    Cut f(nullptr), b(nullptr);
    Forward().cut(f, d);
    Backward back;
    cut(back, b, d);
    *forward_bytes = f.at;
    *backward_bytes = b.at;
    return FP8Z1_OK;
}

extern "C" int fp8z1_linear(const fp8z1_linear_dims* dims, const void* x, int64_t ld_x, const float* x_scale,
                            const uint8_t* codes, const float* scales, const float* bias, const void* residual,
                            int64_t ld_residual, void* y, int64_t ld_y, float* pre, void* workspace, void* stream)
{
    Dims d;
    int st = check(dims, d);
    if (st != FP8Z1_OK) return st;
    if (d.T == 0) return FP8Z1_OK;
    const int64_t K = d.K(), N = d.N();
    const bool fp8 = d.x_type == FP8Z1_E4M3;
    const int y_size = d.y_type == FP8Z1_F32 ? 4 : 2;
    if (!x || !codes || !scales || !y || ld_x < K || ld_y < N || (residual && ld_residual < N) || (fp8 ? !x_scale : !workspace))
        return FP8Z1_EINVAL;
    if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(bias, 4) || !aligned(residual, 2) || !aligned(y, y_size) ||
        !aligned(pre, 4) || (fp8 ? !aligned(x, 16) || ld_x % 16 || !aligned(x_scale, 4) : !aligned(x, 2) || !aligned(workspace, 256)))
        return FP8Z1_EALIGN;
    {
        const Area out = {y, d.T, N * y_size, ld_y * y_size}, z = dense(pre, d.T * N * 4), r = {residual, d.T, N * 2, ld_residual * 2};
        const Area read[] = {dense(codes, d.R * d.C), dense(scales, ceil_div(d.R, 128) * ceil_div(d.C, 128) * 4), dense(bias, N * 4),
                             {fp8 ? x : nullptr, d.T, K, ld_x}, dense(fp8 ? x_scale : nullptr, d.T * ceil_div(K, 128) * 4)};
        for (const Area& a : read)
            if (overlap(out, a) || overlap(z, a)) return FP8Z1_EINVAL;
        // a tile's residual is read when others' results may be there
        if (overlap(out, z) || overlap(z, r) || (d.y_type == FP8Z1_BF16 ? !same_or_apart(out, r) : overlap(out, r))) return FP8Z1_EINVAL;
    }
    NvtxRange range("fp8z1_linear");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Rows rows = {};
    rows.T = d.T;
    if (fp8) {
        rows.hi = static_cast<const uint8_t*>(x);
        rows.pitch = ld_x;
        rows.scale = x_scale;
        rows.scale_row = ceil_div(K, 128);
        rows.scale_block = 1;
    } else {
        Forward f;
        Cut c(workspace);
        f.cut(c, d);
        const bf16* xb = static_cast<const bf16*>(x);
        count_launch();
        split_kernel<<<dim3((unsigned)ceil_div(d.T, 8), (unsigned)ceil_div(d.Kp(), kRowColumns)), 256, 0, s>>>(
            xb, ld_x, d.T, K, d.Kp(), on16(x, ld_x, 2), f.hi, f.lo, f.scale);
        if ((st = launch_status()) != FP8Z1_OK) return st;
        rows.hi = f.hi;
        rows.lo = f.lo;
        rows.lo_format = Lo::kE5M2;
        rows.pitch = d.Kp();
        rows.scale = f.scale;
        rows.scale_row = 1;
        rows.scale_block = d.T;
    }
    Out o = {};
    o.T = d.T;
    o.N = N;
    o.bias = bias;
    o.act = d.act;
    o.residual = static_cast<const bf16*>(residual);
    o.ld_r = ld_residual;
    o.y = y;
    o.ld_y = ld_y;
    o.pre = pre;
    o.f32 = d.y_type == FP8Z1_F32;
    o.vec_y = on16(y, ld_y, y_size);
    o.vec_r = on16(residual, ld_residual, 2);
    o.vec_pre = on16(pre, N, 4);
    o.vec_bias = aligned(bias, 16);
    return launch_product(rows, Weight{codes, scales, d.R, d.C, d.k_major}, o, s);
}

extern "C" int fp8z1_linear_grad(const fp8z1_linear_dims* dims, const void* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                                 const uint8_t* codes, const float* scales, const float* pre, void* dx, int64_t ld_dx,
                                 float* d_weight, float* d_bias, void* workspace, void* stream)
{
    Dims d;
    int st = check(dims, d);
    if (st != FP8Z1_OK) return st;
    if (d.x_type != FP8Z1_BF16 || (!dx && !d_weight && !d_bias)) return FP8Z1_EINVAL;
    if (!aligned(d_weight, 16) || !aligned(d_bias, 4)) return FP8Z1_EALIGN;
    const int64_t K = d.K(), N = d.N();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (d.T == 0) {
        if ((d_weight && cudaMemsetAsync(d_weight, 0, (size_t)(d.R * d.C) * 4, s) != cudaSuccess) ||
            (d_bias && cudaMemsetAsync(d_bias, 0, (size_t)N * 4, s) != cudaSuccess))
            return FP8Z1_ECUDA;
        return FP8Z1_OK;
    }
    const int dy_size = d.y_type == FP8Z1_F32 ? 4 : 2;
    if (!dy || ld_dy < N || !workspace || (d_weight && (!x || ld_x < K)) || (dx && (!codes || !scales || ld_dx < K)) ||
        (d.act != FP8Z1_ACT_NONE && !pre))
        return FP8Z1_EINVAL;
    if (!aligned(dy, dy_size) || (d_weight && !aligned(x, 2)) || (dx && (!aligned(dx, 2) || !aligned(codes, 16) || !aligned(scales, 4))) ||
        !aligned(pre, 4) || !aligned(workspace, 256))
        return FP8Z1_EALIGN;
    {
        const Area to_x = {dx, d.T, K * 2, ld_dx * 2}, to_w = dense(d_weight, d.R * d.C * 4), to_b = dense(d_bias, N * 4);
        const Area xs = {x, d.T, K * 2, ld_x * 2}, dys = {dy, d.T, N * dy_size, ld_dy * dy_size};
        if (overlap(to_x, to_w) || overlap(to_x, to_b) || overlap(to_w, to_b) || overlap(to_x, dense(codes, d.R * d.C)) ||
            overlap(to_x, dense(scales, ceil_div(d.R, 128) * ceil_div(d.C, 128) * 4)))
            return FP8Z1_EINVAL;
        // d_weight comes after dx, of x and (where dz is dy itself) of dy
        if (d_weight && (overlap(to_x, xs) || (d.exact() && (overlap(to_x, dys) || overlap(to_w, xs) || overlap(to_w, dys)))))
            return FP8Z1_EINVAL;
    }
    NvtxRange range("fp8z1_linear_grad");
    Backward b;
    Cut c(workspace);
    cut(b, c, d);
    const dim3 tall((unsigned)ceil_div(d.T, kTall), (unsigned)(d.Kp() / 128));
    DzArgs z = {};
    z.dy = dy;
    z.pre = pre;
    z.ld = ld_dy;
    z.T = d.T;
    z.N = N;
    z.Np = d.Np();
    z.act = d.act;
    z.vec_dy = aligned(dy, 4 * dy_size) && ld_dy % 4 == 0;
    z.vec_pre = aligned(pre, 16) && N % 4 == 0;
    z.b = b;
    if (!dx) z.b.hi = z.b.lo = nullptr;
    if (!d_bias) z.b.part = nullptr;
    if (!d_weight) z.b.dz_hi = z.b.dz_lo = nullptr;
    if (dx || d_bias || !d.exact()) {
        const dim3 tiles(2 * tall.x, (unsigned)(d.Np() / 128));
        if (d.exact())
            st = launch_dz(dz_kernel<bf16, false, false>, tiles, s, z);
        else if (d.y_type == FP8Z1_F32)
            st = d.act ? launch_dz(dz_kernel<float, true, true>, tiles, s, z) : launch_dz(dz_kernel<float, false, true>, tiles, s, z);
        else
            st = launch_dz(dz_kernel<bf16, true, true>, tiles, s, z);
        if (st != FP8Z1_OK) return st;
    }
    if (dx) {
        Rows rows = {};
        rows.hi = b.hi;
        rows.lo = b.lo;
        rows.lo_format = d.exact() ? Lo::kE5M2 : Lo::kE4M3;
        rows.T = d.T;
        rows.pitch = d.Np();
        rows.scale = b.scale;
        rows.scale_row = 1;
        rows.scale_block = d.T;
        Out o = {};
        o.T = d.T;
        o.N = K;
        o.y = dx;
        o.ld_y = ld_dx;
        o.vec_y = on16(dx, ld_dx, 2);
        if ((st = launch_product(rows, Weight{codes, scales, d.R, d.C, d.k_major}.transposed(), o, s)) != FP8Z1_OK) return st;
    }
    if (d_weight) {
        Wgrad g = {};
        g.T = d.T;
        g.N = N;
        g.K = K;
        g.Np = d.Np();
        g.Kp = d.Kp();
        g.k_major = d.k_major;
        g.exact = d.exact();
        g.b = b;
        g.out = d_weight;
        const bf16* xb = static_cast<const bf16*>(x);
        if (g.exact) {
            g.x = xb;
            g.ld_x = ld_x;
            g.dz = static_cast<const bf16*>(dy);
            g.ld_dz = ld_dy;
            if (!on16(x, ld_x, 2)) {
                if ((st = ffn::launch_after(copy_kernel, dim3((unsigned)d.T), 256, 0, s, xb, ld_x, K, b.x_copy, d.Kp())) != FP8Z1_OK)
                    return st;
                g.x = b.x_copy;
                g.ld_x = d.Kp();
            }
            if (!on16(dy, ld_dy, 2)) {
                if ((st = ffn::launch_after(copy_kernel, dim3((unsigned)d.T), 256, 0, s, static_cast<const bf16*>(dy), ld_dy, N,
                                            b.dy_copy, d.Np())) != FP8Z1_OK)
                    return st;
                g.dz = b.dy_copy;
                g.ld_dz = d.Np();
            }
        } else if ((st = ffn::launch_after(x16_kernel, tall, 1024, 0, s, xb, ld_x, d.T, K,
                                           d.Kp(), aligned(x, 8) && ld_x % 4 == 0, b.x16, b.x_factor)) != FP8Z1_OK) {
            return st;
        }
        if ((st = launch_wgrad(g, s)) != FP8Z1_OK) return st;
    }
    return d_bias ? launch_column_sum(b.part, 2 * (int)tall.x, N, d_bias, s) : FP8Z1_OK;
}

extern "C" int fp8z1_linear_timeouts(uint32_t* count)
{
    if (!count) return FP8Z1_EINVAL;
    // the devices' counters only grow, so that no count is lost between a read and a reset
    static std::mutex lock;
    static uint32_t seen[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return FP8Z1_ECUDA;
    std::lock_guard<std::mutex> hold(lock);
    unsigned a = 0, b = 0;
    int st = read_timeouts_product(&a);
    if (st == FP8Z1_OK) st = read_timeouts_wgrad(&b);
    if (st != FP8Z1_OK) {
        cudaGetLastError();
        return st;
    }
    *count = a + b - seen[dev];
    seen[dev] = a + b;
    return FP8Z1_OK;
}

extern "C" int fp8z1_checked_linear_stall(uint32_t kernels)
{
#if FP8Z1_CHECKED
    const int st = stall_product(kernels);
    return st == FP8Z1_OK ? stall_wgrad(kernels >> 2 & 3) : st;
#else
    (void)kernels;
    return FP8Z1_EINVAL;
#endif
}
