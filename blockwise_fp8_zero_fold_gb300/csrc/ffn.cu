// Gated feed-forward block on FP8 weights, forward and backward.
#include "ops_common.cuh"

namespace {

using namespace fp8z1;

constexpr int kTile = 64, kStep = 16;

// An FP8 weight [E, R, C] and its block scales.
struct Weight {
    const uint8_t* codes;
    const float* scale;
    int64_t R, C;
    __device__ __forceinline__ float at(int64_t e, int64_t r, int64_t c) const
    {
        const int64_t sr = (R + 127) / 128, sc = (C + 127) / 128;
        return e4m3_value(codes[(e * R + r) * C + c]) * scale[(e * sr + r / 128) * sc + c / 128];
    }
};

struct Runs {
    const int32_t* offsets;  // NULL: one expert with every row
    int64_t tokens, experts;
    // rows [lo, hi) of expert e, inside [0, tokens] whatever the table holds
    __device__ __forceinline__ void get(int64_t e, int64_t& lo, int64_t& hi) const
    {
        lo = offsets ? min(max((int64_t)offsets[e], (int64_t)0), tokens) : 0;
        hi = offsets ? min(max((int64_t)offsets[e + 1], lo), tokens) : tokens;
    }
};

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

// D[m, n] = sum_k A(m, k) B(k, n) over a 64 x 64 tile; 256 threads, 4 x 4 each.
template <class A, class B, class Out>
__device__ __forceinline__ void product(int64_t m0, int64_t M, int64_t n0, int64_t N, int64_t K, const A& a,
                                        const B& b, const Out& out)
{
    __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += kStep) {
        for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
            const int k = i % kStep, m = i / kStep;
            sa[k][m] = m0 + m < M && k0 + k < K ? a(m0 + m, k0 + k) : 0.0f;
            const int n = i % kTile, kk = i / kTile;
            sb[kk][n] = n0 + n < N && k0 + kk < K ? b(k0 + kk, n0 + n) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStep; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < M && n < N) out(m, n, acc[i][j]);
        }
}

using bf16 = __nv_bfloat16;

// rows [lo, hi) x columns: gu = x gate_up
__global__ void gate_up_kernel(Runs runs, const bf16* x, int64_t ld, Weight w, float* gu)
{
    int64_t lo, hi;
    runs.get(blockIdx.z, lo, hi);
    const int64_t m0 = (int64_t)blockIdx.y * kTile, e = blockIdx.z;
    if (m0 >= hi - lo) return;
    product(m0, hi - lo, (int64_t)blockIdx.x * kTile, w.C, w.R,
            [&](int64_t m, int64_t k) { return to_float(x[(lo + m) * ld + k]); },
            [&](int64_t k, int64_t n) { return w.at(e, k, n); },
            [&](int64_t m, int64_t n, float v) { gu[(lo + m) * w.C + n] = v; });
}

// y = (silu(g) * u) down; rows of no expert get zeros from expert 0's CTAs
__global__ void down_kernel(Runs runs, const float* gu, Weight w, bf16* y, int64_t ld)
{
    int64_t lo, hi;
    runs.get(blockIdx.z, lo, hi);
    const int64_t m0 = (int64_t)blockIdx.y * kTile, e = blockIdx.z, F = w.R;
    if (m0 >= hi - lo) return;
    product(m0, hi - lo, (int64_t)blockIdx.x * kTile, w.C, F,
            [&](int64_t m, int64_t k) {
                const float* p = gu + (lo + m) * 2 * F;
                return silu(p[k]) * p[F + k];
            },
            [&](int64_t k, int64_t n) { return w.at(e, k, n); },
            [&](int64_t m, int64_t n, float v) { y[(lo + m) * ld + n] = __float2bfloat16_rn(v); });
}

__global__ void zero_rest_kernel(Runs runs, bf16* y, int64_t ld, int64_t cols)
{
    int64_t lo, hi;
    runs.get(runs.experts - 1, lo, hi);
    for (int64_t r = hi + blockIdx.x; r < runs.tokens; r += gridDim.x)
        for (int64_t c = threadIdx.x; c < cols; c += blockDim.x) y[r * ld + c] = __float2bfloat16_rn(0.0f);
}

// dgu = [dg | du] from dh = dy down^T
__global__ void dgu_kernel(Runs runs, const bf16* dy, int64_t ld, Weight w, const float* gu, float* dgu)
{
    int64_t lo, hi;
    runs.get(blockIdx.z, lo, hi);
    const int64_t m0 = (int64_t)blockIdx.y * kTile, e = blockIdx.z, F = w.R;
    if (m0 >= hi - lo) return;
    product(m0, hi - lo, (int64_t)blockIdx.x * kTile, F, w.C,
            [&](int64_t m, int64_t k) { return to_float(dy[(lo + m) * ld + k]); },
            [&](int64_t k, int64_t n) { return w.at(e, n, k); },
            [&](int64_t m, int64_t n, float dh) {
                const int64_t at = (lo + m) * 2 * F + n;
                const float g = gu[at], u = gu[at + F], s = 1.0f / (1.0f + expf(-g));
                dgu[at] = dh * u * s * (1.0f + g * (1.0f - s));
                dgu[at + F] = dh * (g * s);
            });
}

__global__ void dx_kernel(Runs runs, const float* dgu, Weight w, bf16* dx, int64_t ld)
{
    int64_t lo, hi;
    runs.get(blockIdx.z, lo, hi);
    const int64_t m0 = (int64_t)blockIdx.y * kTile, e = blockIdx.z;
    if (m0 >= hi - lo) return;
    product(m0, hi - lo, (int64_t)blockIdx.x * kTile, w.R, w.C,
            [&](int64_t m, int64_t k) { return dgu[(lo + m) * w.C + k]; },
            [&](int64_t k, int64_t n) { return w.at(e, n, k); },
            [&](int64_t m, int64_t n, float v) { dx[(lo + m) * ld + n] = __float2bfloat16_rn(v); });
}

__global__ void d_gate_up_kernel(Runs runs, const bf16* x, int64_t ld, const float* dgu, float* out, int64_t H,
                                 int64_t F2)
{
    int64_t lo, hi;
    runs.get(blockIdx.z, lo, hi);
    float* o = out + blockIdx.z * H * F2;
    product((int64_t)blockIdx.y * kTile, H, (int64_t)blockIdx.x * kTile, F2, hi - lo,
            [&](int64_t m, int64_t k) { return to_float(x[(lo + k) * ld + m]); },
            [&](int64_t k, int64_t n) { return dgu[(lo + k) * F2 + n]; },
            [&](int64_t m, int64_t n, float v) { o[m * F2 + n] = v; });
}

__global__ void d_down_kernel(Runs runs, const float* gu, const bf16* dy, int64_t ld, float* out, int64_t F,
                              int64_t H)
{
    int64_t lo, hi;
    runs.get(blockIdx.z, lo, hi);
    float* o = out + blockIdx.z * F * H;
    product((int64_t)blockIdx.y * kTile, F, (int64_t)blockIdx.x * kTile, H, hi - lo,
            [&](int64_t m, int64_t k) {
                const float* p = gu + (lo + k) * 2 * F;
                return silu(p[m]) * p[F + m];
            },
            [&](int64_t k, int64_t n) { return to_float(dy[(lo + k) * ld + n]); },
            [&](int64_t m, int64_t n, float v) { o[m * H + n] = v; });
}

int check_dims(const fp8z1_ffn_dims* d)
{
    if (!d || d->tokens < 0 || d->tokens > kMaxRows || d->hidden < 16 || d->hidden % 16 ||
        d->hidden >= (int64_t)1 << 24 || d->inner < 128 || d->inner % 128 || d->inner >= (int64_t)1 << 24 ||
        d->experts < 1 || d->experts > 1024)
        return FP8Z1_EINVAL;
    return FP8Z1_OK;
}

int check_rows(const void* p, int64_t ld, int64_t cols)
{
    if (!p || ld < cols) return FP8Z1_EINVAL;
    return aligned(p, 16) && ld % 8 == 0 ? FP8Z1_OK : FP8Z1_EALIGN;
}

int check_weights(const fp8z1_ffn_dims* d, const int32_t* off, const uint8_t* gu, const float* gus, const uint8_t* dn,
                  const float* dns)
{
    if (!gu || !gus || !dn || !dns || (!off && d->experts != 1)) return FP8Z1_EINVAL;
    return aligned(gu, 16) && aligned(dn, 16) && aligned(gus, 4) && aligned(dns, 4) && aligned(off, 4)
               ? FP8Z1_OK
               : FP8Z1_EALIGN;
}

unsigned tiles(int64_t n) { return (unsigned)ceil_div(n, kTile); }

}  // namespace

extern "C" int fp8z1_ffn_sizes(const fp8z1_ffn_dims* d, int64_t* saved_bytes, int64_t* forward_bytes,
                               int64_t* backward_bytes)
{
    const int st = check_dims(d);
    if (st != FP8Z1_OK) return st;
    if (!saved_bytes || !forward_bytes || !backward_bytes) return FP8Z1_EINVAL;
    *saved_bytes = *forward_bytes = *backward_bytes = align256(d->tokens * 2 * d->inner * 4) + 256;
    return FP8Z1_OK;
}

extern "C" int fp8z1_ffn_forward(const fp8z1_ffn_dims* d, const void* x, int64_t ld_x, const int32_t* d_offsets,
                                 const uint8_t* gate_up, const float* gate_up_scale, const uint8_t* down,
                                 const float* down_scale, void* y, int64_t ld_y, void* saved, void* workspace,
                                 void* stream)
{
    int st = check_dims(d);
    if (st != FP8Z1_OK) return st;
    if (d->tokens == 0) return FP8Z1_OK;
    if ((st = check_weights(d, d_offsets, gate_up, gate_up_scale, down, down_scale)) != FP8Z1_OK) return st;
    if ((st = check_rows(x, ld_x, d->hidden)) != FP8Z1_OK || (st = check_rows(y, ld_y, d->hidden)) != FP8Z1_OK) return st;
    if (!workspace) return FP8Z1_EINVAL;
    if (!aligned(saved, 256) || !aligned(workspace, 256)) return FP8Z1_EALIGN;
    NvtxRange r("fp8z1_ffn_forward");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Runs runs{d_offsets, d->tokens, d->experts};
    const Weight wgu{gate_up, gate_up_scale, d->hidden, 2 * d->inner}, wd{down, down_scale, d->inner, d->hidden};
    float* gu = static_cast<float*>(saved ? saved : workspace);
    const unsigned E = (unsigned)d->experts, mt = tiles(d->tokens);
    count_launch();
    gate_up_kernel<<<dim3(tiles(wgu.C), mt, E), 256, 0, s>>>(runs, static_cast<const bf16*>(x), ld_x, wgu, gu);
    count_launch();
    down_kernel<<<dim3(tiles(wd.C), mt, E), 256, 0, s>>>(runs, gu, wd, static_cast<bf16*>(y), ld_y);
    count_launch();
    zero_rest_kernel<<<64, 256, 0, s>>>(runs, static_cast<bf16*>(y), ld_y, d->hidden);
    return launch_status();
}

extern "C" int fp8z1_ffn_backward(const fp8z1_ffn_dims* d, const void* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                                  const int32_t* d_offsets, const uint8_t* gate_up, const float* gate_up_scale,
                                  const uint8_t* down, const float* down_scale, const void* saved, void* dx,
                                  int64_t ld_dx, float* d_gate_up, float* d_down, void* workspace, void* stream)
{
    int st = check_dims(d);
    if (st != FP8Z1_OK) return st;
    if ((st = check_weights(d, d_offsets, gate_up, gate_up_scale, down, down_scale)) != FP8Z1_OK) return st;
    if (!d_gate_up || !d_down) return FP8Z1_EINVAL;
    if (!aligned(d_gate_up, 16) || !aligned(d_down, 16)) return FP8Z1_EALIGN;
    if (d->tokens > 0) {
        if ((st = check_rows(x, ld_x, d->hidden)) != FP8Z1_OK || (st = check_rows(dy, ld_dy, d->hidden)) != FP8Z1_OK ||
            (dx && (st = check_rows(dx, ld_dx, d->hidden)) != FP8Z1_OK))
            return st;
        if (!saved || !workspace) return FP8Z1_EINVAL;
        if (!aligned(saved, 256) || !aligned(workspace, 256)) return FP8Z1_EALIGN;
    }
    NvtxRange r("fp8z1_ffn_backward");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Runs runs{d_offsets, d->tokens, d->experts};
    const Weight wgu{gate_up, gate_up_scale, d->hidden, 2 * d->inner}, wd{down, down_scale, d->inner, d->hidden};
    const float* gu = static_cast<const float*>(saved);
    float* dgu = static_cast<float*>(workspace);
    const bf16 *xb = static_cast<const bf16*>(x), *dyb = static_cast<const bf16*>(dy);
    const unsigned E = (unsigned)d->experts, mt = tiles(d->tokens);
    if (d->tokens > 0) {
        count_launch();
        dgu_kernel<<<dim3(tiles(d->inner), mt, E), 256, 0, s>>>(runs, dyb, ld_dy, wd, gu, dgu);
        if (dx) {
            count_launch();
            dx_kernel<<<dim3(tiles(d->hidden), mt, E), 256, 0, s>>>(runs, dgu, wgu, static_cast<bf16*>(dx), ld_dx);
            count_launch();
            zero_rest_kernel<<<64, 256, 0, s>>>(runs, static_cast<bf16*>(dx), ld_dx, d->hidden);
        }
    }
    count_launch();
    d_gate_up_kernel<<<dim3(tiles(wgu.C), tiles(wgu.R), E), 256, 0, s>>>(runs, xb, ld_x, dgu, d_gate_up, wgu.R, wgu.C);
    count_launch();
    d_down_kernel<<<dim3(tiles(wd.C), tiles(wd.R), E), 256, 0, s>>>(runs, gu, dyb, ld_dy, d_down, wd.R, wd.C);
    return launch_status();
}
