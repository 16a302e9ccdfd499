// The gated feed-forward block of a few tokens: matrix-vector products that
// stream the FP8 codes once.
//
//   h = silu(x Wg) * (x Wu)   (FP32),   y = h Wd   (rounded to BF16 once)
//
// Bound by the codes read and by their decoding, neither alone: one token of 4096 x
// 14336 takes 43 us, 26 at the rate of a copy, with half the issue slots decoding and DRAM
// at 53 % in the first product and 38 % in the second, whose start overlaps.  A cluster of up to 8
// CTAs has 128 or 64 columns of a product (gate_up: gate columns and the up columns
// beside them), each CTA a part of K; a thread has 16 neighbouring columns (16 bytes
// of a row), three or four rows on their way while as many are multiplied, and FP32
// sums of up to 4 tokens.  Scale blocks are 128 x 128, so a row's 16 columns share
// their scale: it goes to the vector's element.  Sums are added over a CTA's threads
// and the cluster's CTAs in a fixed order.  The second product's codes are on their
// way before h is there.
#include <cooperative_groups.h>

#include <climits>
#include <type_traits>

#include "ffn.cuh"

namespace fp8z1 {
namespace ffn {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kMostSplit = 8, kTokens = 4;  // kernels for 1 token and for up to 4
constexpr int kMostSlice = 8192;  // of K, a CTA's
// CTAs of an SM, for which a token's 16 sums a thread leave registers, and rows on
// their way.  (One token of 4096 x 14336: 48 us with 3 CTAs and 4 rows, 44 with 4
// and 3, 48 with 5 and 2.)
__host__ __device__ constexpr int resident(int tokens) { return tokens == 1 ? 4 : 2; }
__host__ __device__ constexpr int hold(int tokens) { return tokens == 1 ? 3 : 4; }

struct Args {
    Runs runs;
    int64_t K, N;      // rows and columns of the product (kGateUp: N = F)
    int64_t C;         // columns of the weight
    const uint8_t* w;
    const float* scale;
    int32_t sr, sc;    // the scale grid of an expert
    int32_t split;     // CTAs of a cluster
    int32_t slice;     // rows of each, a multiple of 128
    const bf16* x;     // kGateUp
    int64_t ld_x;
    float* h;          // [tokens, F]
    bf16* y;           // down
    int64_t ld_y;
};

// kHold rows' codes of a thread's columns.
template <int kStep, int kHold>
__device__ __forceinline__ void load_rows(uint4 (&c)[kHold], const uint8_t* w, int64_t C, int k, int n)
{
#pragma unroll
    for (int i = 0; i < kHold; ++i)
        if (k + i * kStep < n) c[i] = __ldcs(reinterpret_cast<const uint4*>(w + (int64_t)(k + i * kStep) * C));
}

// kOut columns of the result, kMost tokens.  kGateUp: threads of the first half of
// a row's have gate columns, those of the other half the up columns.
template <bool kGateUp, int kOut, int kMost>
__global__ void __launch_bounds__(kThreads, resident(kMost)) gemv_kernel(const Args a)
{
    using T = std::conditional_t<kGateUp, bf16, float>;  // the vectors' type
    constexpr int kHalf = kOut / 16, kAcross = kGateUp ? 2 * kHalf : kHalf, kDeep = kThreads / kAcross;
    constexpr int kCols = kAcross * 16, kWarps = kThreads / 32, kHold = hold(kMost);
    extern __shared__ __align__(16) uint8_t smem[];  // scales [2][slice / 128], then vectors [kMost][slice]
    __shared__ float sums[kWarps][kMost][kCols];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t n0 = (int64_t)(blockIdx.x / a.split) * kOut;
    int64_t e = blockIdx.y;
    if (a.runs.experts > a.runs.tokens) {  // blockIdx.y is a token: the expert whose run begins there, if one does
        __shared__ int found;
        if (tid == 0) found = INT_MAX;
        __syncthreads();
        for (int i = tid; i < a.runs.experts; i += kThreads) {
            int64_t lo, hi;
            a.runs.get(i, lo, hi);
            if (lo == blockIdx.y && hi > lo) atomicMin(&found, i);
        }
        __syncthreads();
        e = found;
    }
    const int deep = tid / kAcross, across = tid % kAcross, half = across / kHalf;
    // this CTA's rows, this thread's first column in the weight
    const int64_t k0 = (int64_t)rank * a.slice;
    const int rows = (int)max(min((int64_t)a.slice, a.K - k0), (int64_t)0);
    const int64_t col = n0 + across % kHalf * 16;
    const bool there = col < a.N;
    int64_t lo = 0, hi = 0;
    if (e < a.runs.experts) a.runs.get(e, lo, hi);
    const uint8_t* w = a.w + (e * a.K + k0) * a.C + col + (half ? a.N : 0);
    uint4 x[kHold], y[kHold];
    if (there && hi > lo) load_rows<kDeep, kHold>(x, w, a.C, deep, rows);
    // the down product's CTAs may start beside the last of gate_up's: its first codes are on their way when h is there
    if (kGateUp)
        next_may_start();
    else
        after_previous();
    if (!kGateUp && blockIdx.y == 0 && rank == 0) {  // rows of no expert
        int64_t l, h;
        a.runs.get(a.runs.experts - 1, l, h);
        for (; h < a.runs.tokens; ++h)
            if (tid < kOut && n0 + tid < a.N) a.y[h * a.ld_y + n0 + tid] = __float2bfloat16_rn(0.0f);
    }
    if (hi == lo) return;  // the same in every CTA of the cluster
    const int blocks = a.slice / 128;
    float* scales = reinterpret_cast<float*>(smem);
    T* v = reinterpret_cast<T*>(scales + (2 * blocks + 3) / 4 * 4);
    // a CTA's columns lie in one scale block (gate_up: one each)
    for (int i = tid; i < 2 * blocks; i += kThreads) {
        const int64_t b = k0 / 128 + i % blocks;
        const int64_t c = (n0 + (i >= blocks && kGateUp ? a.N : 0)) / 128;
        scales[i] = b < a.sr ? __ldg(a.scale + (e * a.sr + b) * a.sc + c) : 0.0f;
    }
    const float* my_scales = scales + half * blocks;

    const int n_tokens = (int)min((int64_t)kMost, hi - lo);
    for (int t = 0; t < n_tokens; ++t)
        for (int k = tid * 8; k < rows; k += kThreads * 8) {  // rows and strides are multiples of 8 elements
            if constexpr (kGateUp) {
                *reinterpret_cast<uint4*>(v + t * a.slice + k) =
                    __ldg(reinterpret_cast<const uint4*>(a.x + (lo + t) * a.ld_x + k0 + k));
            } else {
                const float4* p = reinterpret_cast<const float4*>(a.h + (lo + t) * a.K + k0 + k);
                float4* o = reinterpret_cast<float4*>(v + t * a.slice + k);
                o[0] = p[0];
                o[1] = p[1];
            }
        }
    __syncthreads();
    uint64_t acc[kMost][8];
#pragma unroll
    for (int t = 0; t < kMost; ++t)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[t][j] = 0;
    auto multiply = [&](const uint4(&c)[kHold], int k) {
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
            const int at = k + i * kDeep;
            if (at >= rows) break;
            const float s = my_scales[at >> 7];
            const uint32_t words[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
            uint64_t two[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 f = e4m3x2_decode(words[j >> 1] >> (16 * (j & 1)) & 0xffffu);
                two[j] = tc::pair(f.x, f.y);
            }
#pragma unroll
            for (int t = 0; t < kMost; ++t) {
                if (t >= n_tokens) break;
                const float xs = to_float(v[t * a.slice + at]) * s;
                const uint64_t x2 = tc::pair(xs, xs);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[t][j] = tc::fma_pair(two[j], x2, acc[t][j]);
            }
        }
    };
    if (there)
        for (int k = deep; k < rows; k += 2 * kHold * kDeep) {
            load_rows<kDeep, kHold>(y, w, a.C, k + kHold * kDeep, rows);
            multiply(x, k);
            load_rows<kDeep, kHold>(x, w, a.C, k + 2 * kHold * kDeep, rows);
            multiply(y, k + kHold * kDeep);
        }
    // over the warp's rows, the CTA's warps, the cluster's CTAs
#pragma unroll
    for (int t = 0; t < kMost; ++t) {
        if (t >= n_tokens) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float2 f = tc::unpair(acc[t][j]);
#pragma unroll
            for (int o = kAcross; o < 32; o <<= 1) {
                f.x += __shfl_xor_sync(0xffffffffu, f.x, o);
                f.y += __shfl_xor_sync(0xffffffffu, f.y, o);
            }
            if (lane < kAcross) *reinterpret_cast<float2*>(&sums[warp][t][lane * 16 + j * 2]) = f;
        }
    }
    __syncthreads();
    for (int i = tid; i < n_tokens * kCols; i += kThreads) {  // to the first warp's
        const int t = i / kCols, n = i % kCols;
        float f = sums[0][t][n];
#pragma unroll
        for (int q = 1; q < kWarps; ++q) f += sums[q][t][n];
        sums[0][t][n] = f;
    }
    cluster.sync();
    // each CTA finishes its share of the columns
    for (int i = rank * kThreads + tid; i < kOut * n_tokens; i += a.split * kThreads) {
        const int n = i % kOut, t = i / kOut;
        if (n0 + n >= a.N) continue;
        float f = 0.0f, u = 0.0f;
        for (int q = 0; q < a.split; ++q) {
            const float* p = cluster.map_shared_rank(&sums[0][t][0], q);
            f += p[n];
            if (kGateUp) u += p[kOut + n];
        }
        if (kGateUp)
            a.h[(lo + t) * a.N + n0 + n] = f / (1.0f + expf(-f)) * u;
        else
            a.y[(lo + t) * a.ld_y + n0 + n] = __float2bfloat16_rn(f);
    }
    cluster.sync();  // no CTA leaves before its sums are read
}

// The time of a launch by its rounds of CTAs, in rows of 64 columns; a CTA's fixed
// steps are worth 1024 rows.
struct Shape {
    double time;
    int32_t split, slice;
};
Shape shape(int64_t K, int64_t N, int64_t runs, int out, int resident)
{
    const int64_t groups = ceil_div(N, out) * runs;
    Shape best = {1e30, 1, 0};
    for (int n = 1; n <= kMostSplit; ++n) {
        const int64_t slice = ceil_div(ceil_div(K, n), 128) * 128;
        if (slice > kMostSlice || (n > 1 && slice < 256)) continue;
        const double t = (double)ceil_div(groups * n, kSms * resident) * (double)((slice + 1024) * out / 64);
        if (t < best.time) best = {t, n, (int32_t)slice};
    }
    return best;
}

template <bool kGateUp, int kOut, int kMost>
int launch(Args a, const Shape& shape, int64_t runs, cudaStream_t s)
{
    using T = std::conditional_t<kGateUp, bf16, float>;
    const auto kernel = gemv_kernel<kGateUp, kOut, kMost>;
    a.split = shape.split;
    a.slice = shape.slice;
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)a.split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    c.gridDim = dim3((unsigned)(ceil_div(a.N, kOut) * a.split), (unsigned)runs);
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = (size_t)((2 * (a.slice / 128) + 3) / 4 * 16 + (int64_t)a.slice * kMost * sizeof(T));
    c.stream = s;
    c.attrs = at;
    c.numAttrs = kGateUp ? 1 : 2;
    if (!allow_smem<gemv_kernel<kGateUp, kOut, kMost>>(kMostSlice * (kMost * (int)sizeof(T) + 1))) return FP8Z1_ECUDA;
    count_launch();
    if (cudaLaunchKernelEx(&c, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return FP8Z1_ECUDA;
    }
    return launch_status();
}

template <bool kGateUp>
int launch(const Args& a, cudaStream_t s)
{
    const int64_t runs = a.runs.experts < a.runs.tokens ? a.runs.experts : a.runs.tokens;
    const bool one = a.runs.tokens == 1;
    const Shape wide = shape(a.K, a.N, runs, 128, resident(one ? 1 : kTokens)), narrow = shape(a.K, a.N, runs, 64, resident(one ? 1 : kTokens));
    if (wide.time <= narrow.time)
        return one ? launch<kGateUp, 128, 1>(a, wide, runs, s) : launch<kGateUp, 128, kTokens>(a, wide, runs, s);
    return one ? launch<kGateUp, 64, 1>(a, narrow, runs, s) : launch<kGateUp, 64, kTokens>(a, narrow, runs, s);
}

}  // namespace

bool few_tokens(const Dims& d)
{
    // The slices of the vectors have to fit shared memory.  One token's products are read; more tokens multiply every
    // decoded code again, which the tensor cores do not notice.  Here and there, us, by the multiplications: 264 M (three
    // tokens of 7168 x 4096) 40 and 41, 277 M (four of 4096 x 5632) 38 and 40, 302 M (three of 4096 x 8192) 42 and 43,
    // 352 M (four of 7168 x 4096, of 2048 x 14336; two of 4096 x 14336) 46 and 41, 46 and 44, 60 and 60, 705 M (four of
    // 4096 x 14336) 79 and 60.  One token of 4096 x 14336 44 and 59, of 7168 x 18432 80 and 94; four over 32 experts of
    // 7168 x 2048, mostly one each, 51 and 55.
    return d.T <= kTokens && (d.H > d.F ? d.H : d.F) <= kMostSplit * kMostSlice &&
           (d.T == 1 || d.T * 3 * d.H * d.F <= (int64_t)5 << 26);
}

int launch_gemv(const Dims& d, const Runs& runs, const bf16* x, int64_t ld_x, const Weight& wgu, const Weight& wd, float* h,
                bf16* y, int64_t ld_y, cudaStream_t s)
{
    Args a = {};
    a.runs = runs;
    a.K = d.H;
    a.N = d.F;
    a.C = 2 * d.F;
    a.w = wgu.codes;
    a.scale = wgu.scale;
    a.sr = (int32_t)ceil_div(d.H, 128);
    a.sc = (int32_t)(d.F / 64);
    a.x = x;
    a.ld_x = ld_x;
    a.h = h;
    const int st = launch<true>(a, s);
    if (st != FP8Z1_OK) return st;
    a.K = d.F;
    a.N = a.C = d.H;
    a.w = wd.codes;
    a.scale = wd.scale;
    a.sr = (int32_t)(d.F / 128);
    a.sc = (int32_t)ceil_div(d.H, 128);
    a.y = y;
    a.ld_y = ld_y;
    return launch<false>(a, s);
}

}  // namespace ffn
}  // namespace fp8z1
