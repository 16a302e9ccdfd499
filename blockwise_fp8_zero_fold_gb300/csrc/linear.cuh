// The matrix product with an FP8 weight: what its translation units share.
#pragma once

#include "ffn.cuh"

namespace fp8z1 {
namespace linear {

using ffn::bf16;
using ffn::kBlock;
using ffn::Lo;

// y [T, N] = x [T, K] w: the weight is [K, N] row-major, or with `k_major` its transpose [N, K].
struct Weight {
    const uint8_t* codes;
    const float* scale;
    int64_t R, C;  // as it lies
    bool k_major;
    int64_t K() const { return k_major ? C : R; }
    int64_t N() const { return k_major ? R : C; }
    Weight transposed() const { return Weight{codes, scale, R, C, !k_major}; }
};

// Rows of FP8 numbers, value = (hi + lo) * scale[k / 128][row]; lo NULL: hi alone
struct Rows {
    const uint8_t *hi, *lo;
    Lo lo_format;
    int64_t T, pitch;                 // rows, bytes of one
    const float* scale;
    int64_t scale_row, scale_block;  // strides of `scale`
};

// What becomes of a sum z: y = act(z + bias) + residual.
struct Out {
    int64_t T, N;
    const float* bias;     // [N] or NULL
    int32_t act;           // FP8Z1_ACT_*
    const bf16* residual;  // or NULL
    int64_t ld_r;
    void* y;
    int64_t ld_y;
    float* pre;            // z + bias, [T, N], or NULL
    bool f32;              // y's type
    bool vec_y, vec_r, vec_pre, vec_bias;  // whole 16 bytes on 16-byte boundaries
};

// z's factor in its activation, a sigmoid of c(z), by t = exp(-|c|) <= 1: nothing overflows.
constexpr float kGelu = 1.5957691216057308f, kCubic = 0.044715f;  // gelu_tanh: c = kGelu (z + kCubic z^3)
__device__ __forceinline__ float gate_argument(float z, int act)
{
    return act == FP8Z1_ACT_SILU ? z : kGelu * __fmaf_rn(kCubic * z * z, z, z);
}
// By expf, off by a unit in the last place: __expf is off by more the larger |c| is (some 100 at 80), which an FP32 result
// would show.  One for BF16 results too: it costs them 2 % (2051 rows of 4096 x 14336 with GELU 195 -> 198 us), and two of
// them in a tile's end 4 to 9 % in rows of odd widths.
__device__ __forceinline__ float activate(float z, int act)
{
    if (act == FP8Z1_ACT_NONE) return z;
    const float c = gate_argument(z, act), t = expf(-fabsf(c));
    return z * __fdividef(c < 0.0f ? t : 1.0f, 1.0f + t);
}
// The activation's derivative: s + z s (1 - s) c', the second term 0 where t is.
__device__ __forceinline__ float slope(float z, int act)
{
    const float c = gate_argument(z, act), t = expf(-fabsf(c)), big = __fdividef(1.0f, 1.0f + t), small = t * big;
    const float s = c < 0.0f ? small : big;
    const float dc = act == FP8Z1_ACT_SILU ? 1.0f : kGelu * __fmaf_rn(3.0f * kCubic * z, z, 1.0f);
    return t > 0.0f ? __fmaf_rn(z * (small * big), dc, s) : s;
}

// FP16 numbers of the weight's gradient: two terms of dz, one of x, 256 rows at a time at powers of two.
constexpr int kTall = 256;

struct Backward {
    uint8_t *hi, *lo;      // dz, [T, Np]
    float* scale;          // [Np / 128, T]
    __half *dz_hi, *dz_lo; // [T, Np]
    float* dz_factor;      // [T / 256, Np]
    __half* x16;           // [T, Kp]
    float* x_factor;       // [T / 256, Kp / 128]
    float* part;           // [T / 128, N] sums of dz's columns
    bf16 *x_copy, *dy_copy;  // [T, Kp], [T, Np]: where theirs do not lie on 16 bytes
};

// ---- launches (each returns a status) --------------------------------------------

// y of the product; see linear_gemm.cu.
int launch_product(const Rows& x, const Weight& w, const Out& o, cudaStream_t s);
// d_weight [R, C]: sums over the T rows of dz and x; see linear_wgrad.cu.  `exact`: dz and x
// are BF16 rows; else FP16 terms.
struct Wgrad {
    int64_t T, N, K;
    bool k_major;
    bool exact;
    const bf16 *dz, *x;
    int64_t ld_dz, ld_x;
    Backward b;
    int64_t Np, Kp;
    float* out;
};
int launch_wgrad(const Wgrad& g, cudaStream_t s);

int read_timeouts_product(unsigned* n);
int read_timeouts_wgrad(unsigned* n);
#if FP8Z1_CHECKED
int stall_product(unsigned kernels);
int stall_wgrad(unsigned kernels);
#endif

}  // namespace linear
}  // namespace fp8z1
