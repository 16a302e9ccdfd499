// The gated feed-forward block's buffers, shared by its translation units.
//
// Token rows are regrouped so that every expert starts a tile of 128 rows:
// tile t of the launch holds rows [token0, token0 + rows) of its expert, and row
// r of it is row 128 t + r of every internal buffer.  Rows of a tile past its
// own are multiplied like the others and stored nowhere; in the operands of the
// weight gradients they are zeros.
#pragma once

#include <algorithm>
#include <cuda_fp16.h>

#include "ops_common.cuh"
#include "tc.cuh"

namespace fp8z1 {
namespace ffn {

constexpr int kRows = 128;      // token rows of a tile
constexpr int kBlock = 128;     // the scale blocks' side, and a K step of the FP8 products

struct Tile {
    int32_t expert, token0, rows, pad;
};

// Per expert: the bits of the largest finite magnitudes (as non-negative floats), in a
// sector of its own (every warp of the row kernels adds to them: with four experts in a
// sector 8192 rows of 7168 took 54 us for 41).
struct Peaks {
    uint32_t x, dy;
    uint32_t pad[6];
};

// Which rows belong to whom; written by the plan kernel.
struct Plan {
    const int32_t* n_tiles;
    const int32_t* start;   // [experts + 1] first tile of each expert
    const int32_t* tokens;  // [experts] rows of each
    const Tile* tiles;      // [n_tiles]
    // An expert's tiles two by two, as the weight gradients add them up (backward).
    const int32_t* n_pairs;
    const int32_t* pair_start;  // [experts] first pair of each
    const int32_t* pairs;       // [n_pairs] twice the first tile, and 1 when there is a second
};

// FP8 pairs: value = (hi + lo) * scale[k / 128][row]; see pair_encode
struct Pairs {
    uint8_t *hi, *lo;  // [rows, pitch]
    float* scale;      // [pitch / 128, rows]
    int64_t pitch;
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

struct Dims {
    int64_t T, H, F, E;
    int64_t tiles() const { return T / kRows + (E < T ? E : T); }  // at most
    int64_t pairs() const { return (tiles() + (E < tiles() ? E : tiles())) / 2; }  // at most: an odd tile each
    int64_t rows() const { return tiles() * kRows; }
    int64_t Hp() const { return (H + 127) / 128 * 128; }
};

// Buffers cut from one allocation, 256 bytes apart.
struct Cut {
    char* base;
    int64_t at = 0;
    explicit Cut(void* p) : base(static_cast<char*>(p)) {}
    template <class T>
    T* take(int64_t n)
    {
        T* p = base ? reinterpret_cast<T*>(base + at) : nullptr;
        at += align256(n * (int64_t)sizeof(T));
        return p;
    }
};

struct PlanBuffers {
    int32_t *n_tiles, *start, *tokens;
    Tile* tiles;
    int32_t *n_pairs, *pair_start, *pairs;  // NULL in a forward pass
    void cut(Cut& c, const Dims& d, bool backward)
    {
        n_tiles = c.take<int32_t>(1);
        start = c.take<int32_t>(d.E + 1);
        tokens = c.take<int32_t>(d.E);
        tiles = c.take<Tile>(d.tiles());
        n_pairs = pair_start = pairs = nullptr;
        if (!backward) return;
        n_pairs = c.take<int32_t>(1);
        pair_start = c.take<int32_t>(d.E);
        pairs = c.take<int32_t>(d.pairs());
    }
    Plan plan() const { return Plan{n_tiles, start, tokens, tiles, n_pairs, pair_start, pairs}; }
};

inline Pairs cut_pairs(Cut& c, int64_t rows, int64_t pitch)
{
    Pairs p;
    p.hi = c.take<uint8_t>(rows * pitch);
    p.lo = c.take<uint8_t>(rows * pitch);
    p.scale = c.take<float>(rows * (pitch / kBlock));
    p.pitch = pitch;
    return p;
}

// What a forward pass keeps: g | u in FP32 as [tile][column of 2F][row of 128]
// (a warp's 32 rows are consecutive), and each expert's peak of x.
struct Saved {
    Peaks* peaks;
    float* gu;
    void cut(Cut& c, const Dims& d)
    {
        peaks = c.take<Peaks>(d.E);
        gu = c.take<float>(d.rows() * 2 * d.F);
    }
};

// Whether the forward pass is matrix-vector products; see ffn_gemv.cu.
bool few_tokens(const Dims& d);

// CTAs along K of a forward product with N columns (gate_up: 2F) and K rows.  With
// few tiles of 128 x 256 most SMs would have no work, and one CTA takes 0.8 us for
// 128 rows of codes from memory: parts of at least 512 rows, for about 128 CTAs.
// (6 tokens of 7168 x 2048: gate_up 59 us whole.)
inline int32_t k_splits(const Dims& d, int64_t N, int64_t K)
{
    if (d.T == 0) return 1;
    int64_t n = 128 / (d.tiles() * ceil_div(N, 256));
    if (n > K / (4 * kBlock)) n = K / (4 * kBlock);
    return (int32_t)(n < 1 ? 1 : n > 16 ? 16 : n);
}
inline int64_t part_floats(const Dims& d, int64_t N, int64_t K)
{
    const int64_t n = k_splits(d, N, K);
    return n > 1 ? n * d.rows() * N : 0;
}

struct Forward {
    PlanBuffers plan;
    float* part;  // a split product's sums, [splits, rows, N]; few tokens: h, [T, F]
    Pairs x, h;
    void cut(Cut& c, const Dims& d)
    {
        plan.cut(c, d, false);
        part = c.take<float>(
            std::max<int64_t>({few_tokens(d) ? d.T * d.F : 0, part_floats(d, 2 * d.F, d.H), part_floats(d, d.H, d.F)}));
        x = cut_pairs(c, d.rows(), d.Hp());
        h = cut_pairs(c, d.rows(), d.F);
    }
};

struct Backward {
    PlanBuffers plan;
    Peaks* peaks;
    Pairs dy, dgu;
    float* dh;           // [tile][column of F][row of 128]
    __half *x16, *dy16;  // [rows, Hp]
    __half *h_hi, *h_lo;      // [rows, F]
    __half *dgu_hi, *dgu_lo;  // [rows, 2F]
    float* factors;           // [pairs of tiles][3F], of the columns of dg, du, h: see column_scale
    void cut(Cut& c, const Dims& d)
    {
        plan.cut(c, d, true);
        peaks = c.take<Peaks>(d.E);
        dy = cut_pairs(c, d.rows(), d.Hp());
        dgu = cut_pairs(c, d.rows(), 2 * d.F);
        dh = c.take<float>(d.rows() * d.F);
        x16 = c.take<__half>(d.rows() * d.Hp());
        dy16 = c.take<__half>(d.rows() * d.Hp());
        h_hi = c.take<__half>(d.rows() * d.F);
        h_lo = c.take<__half>(d.rows() * d.F);
        dgu_hi = c.take<__half>(d.rows() * 2 * d.F);
        dgu_lo = c.take<__half>(d.rows() * 2 * d.F);
        factors = c.take<float>(d.pairs() * 3 * d.F);
    }
};

struct Weight {
    const uint8_t* codes;
    const float* scale;
    int64_t R, C;  // of one expert
};

using bf16 = __nv_bfloat16;

// An FP8 pair: hi = e4m3(v), lo = v - hi, for v scaled by a power of two so that the
// largest of its 128 lies in (224, 448], the top of E4M3.  hi leaves at most 8 units of a
// BF16 value's last place.
//
// x and dy are BF16 values, and their lo is E5M2, whose 3 bits hold every number of
// units up to 8: a value down to 2^-13.8 of the largest one is held exactly, a smaller one
// to 2^-21.8 of it.  (An outlier channel 300 times the others needs that range: with the
// largest in [128, 256) one gate in 10^4 was off by 2^-16 of its terms and a weight gradient
// that hung on it by 6e-5; with lo in E4M3 the exact range would end at 2^-10.)
//
// h, dg and du are FP32 and rounded by their pair on the way to the second product (to y,
// to dx), as a BF16 activation between two products would be.  Their lo is E4M3, of 4
// bits: values are held to 2^-9 of themselves, twice as fine as BF16's 2^-8, or to 2^-17.8
// of the largest: y and dx, rounded to BF16, are off by 1.8e-3 of their norm (2.1e-3 with
// two roundings of BF16's, 1.66e-3 with the last alone).  A third FP8 term would hold 12
// bits and make these products half as long again.
struct PairScale {
    float up, down;  // multiply by `up` to encode, by `down` to decode
};
__device__ __forceinline__ PairScale pair_scale(float amax)
{
    const uint32_t bits = __float_as_uint(amax);  // amax >= 0
    const uint32_t e = min(max((bits + 0x1fffffu) >> 23, 9u), 255u);  // one more from 1.75 times a power of two on
    // an infinity makes its 128 values NaN (E4M3 has none)
    return PairScale{__uint_as_float(bits < 0x7f800000u ? (262u - e) << 23 : 0x7fffffffu), __uint_as_float((e - 8u) << 23)};
}
enum class Lo { kE5M2, kE4M3 };
// v's pair as two codes each for (a, b): bits 0-15 of hi and lo.  FP16 on the way
// holds more bits than the pair does, down to 2^-32 of the largest value, and takes
// half the instructions of FP32.
template <Lo kLo>
__device__ __forceinline__ void pair_encode(float a, float b, float up, uint32_t& hi, uint32_t& lo)
{
    const __half2 v = __floats2half2_rn(a * up, b * up);
    unsigned short h, l;
    uint32_t back;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(h) : "r"(*reinterpret_cast<const uint32_t*>(&v)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(back) : "h"(h));
    const __half2 rest = __hsub2(v, *reinterpret_cast<const __half2*>(&back));
    if constexpr (kLo == Lo::kE5M2)
        asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(l) : "r"(*reinterpret_cast<const uint32_t*>(&rest)));
    else
        asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(l) : "r"(*reinterpret_cast<const uint32_t*>(&rest)));
    hi = h;
    lo = l;
}

// 2^k as two factors, for |k| <= 252
struct Pow2 {
    float a, b;
    __device__ __forceinline__ float times(float v) const { return v * a * b; }
};
__device__ __forceinline__ Pow2 pow2(int k)
{
    k = min(max(k, -252), 252);
    const int h = min(max(k, -126), 126);  // b is 1 unless k leaves FP32's exponents
    return Pow2{__uint_as_float((uint32_t)(127 + h) << 23), __uint_as_float((uint32_t)(127 + k - h) << 23)};
}
// floor(log2) of a positive float's bits (-127 for 0 and subnormals, 128 for inf)
__device__ __forceinline__ int exponent(uint32_t bits) { return (int)(bits >> 23) - 127; }

// The FP16 operands of the weight gradients lie below 2^15.  x and dy take one power
// of two for an expert: 2^shift to encode, 2^exponent to decode numbers of 2^14.
__device__ __forceinline__ int peak_exponent(uint32_t bits) { return max(exponent(bits), -126); }
__device__ __forceinline__ int peak_shift(uint32_t bits) { return 14 - peak_exponent(bits); }
__device__ __forceinline__ float peak_factor(uint32_t bits)
{
    return __uint_as_float((uint32_t)(127 + min(peak_exponent(bits), 127)) << 23);
}
// dg, du and h take one for every column of a pair of tiles, from its largest number there: an
// element keeps 22 bits, or what lies above 2^-40 of that number, whatever the other
// columns hold.  `down` brings products with numbers of 2^14 back to numbers of 1.
struct ColumnScale {
    float up, down;
};
__device__ __forceinline__ ColumnScale column_scale(uint32_t exponent)  // the bits of it, 127 for [1, 2)
{
    const int shift = min(141 - (int)exponent, 112);
    return ColumnScale{__uint_as_float((uint32_t)(127 + shift) << 23), __uint_as_float((uint32_t)(113 - shift) << 23)};
}

// ---- launches (each returns a status) -------------------------------------------

// The FP8 products of one K-blocked shape; see ffn_gemm.cu.
int launch_gate_up(const Dims& d, const Plan& p, const Pairs& x, const Weight& w, const Pairs& h, float* gu, float* part,
                   cudaStream_t s);
int launch_down(const Dims& d, const Plan& p, const Pairs& h, const Weight& w, bf16* y, int64_t ld, float* part,
                cudaStream_t s);
int launch_dh(const Dims& d, const Plan& p, const Pairs& dy, const Weight& w, float* dh, cudaStream_t s);
int launch_dx(const Dims& d, const Plan& p, const Pairs& dgu, const Weight& w, bf16* dx, int64_t ld, cudaStream_t s);
// y of a few tokens (h: FP32 [T, F]); see ffn_gemv.cu.
int launch_gemv(const Dims& d, const Runs& runs, const bf16* x, int64_t ld_x, const Weight& wgu, const Weight& wd, float* h,
                bf16* y, int64_t ld_y, cudaStream_t s);
// The weight gradients; see ffn_wgrad.cu.
int launch_d_gate_up(const Dims& d, const Plan& p, const Backward& b, float* out, cudaStream_t s);
int launch_d_down(const Dims& d, const Plan& p, const Backward& b, float* out, cudaStream_t s);

// A pass is a chain of short kernels: each may start while the one before it ends
// (its launch and set-up cost 2 to 3 us otherwise) and touches memory only when
// all that one wrote is there.
__device__ __forceinline__ void next_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launches a kernel that calls both, right behind another of the pass, in clusters of kCluster CTAs.
template <int kCluster = 1, class... A, class... P>
int launch_after(void (*kernel)(A...), dim3 grid, int threads, uint32_t smem, cudaStream_t s, const P&... args)
{
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = kCluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.gridDim = grid;
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = at;
    c.numAttrs = kCluster > 1 ? 2 : 1;
    count_launch();
    if (cudaLaunchKernelEx(&c, kernel, A(args)...) != cudaSuccess) {
        cudaGetLastError();
        return FP8Z1_ECUDA;
    }
    return launch_status();
}

// Launches, right behind another kernel of the pass, a persistent one of one CTA an SM, in clusters of kCluster: as many as
// run at once, `most` at most.
template <auto kKernel, int kCluster, class... P>
int launch_persistent(int threads, uint32_t smem, int64_t most, cudaStream_t s, const P&... args)
{
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = at;
    c.numAttrs = 1;
    // what the device holds at once, asked once for each kernel and device
    static std::atomic<int> holds[16];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return FP8Z1_ECUDA;
    int n = dev < 16 ? holds[dev].load(std::memory_order_relaxed) : 0;
    if (n == 0) {
        c.gridDim = dim3(kCluster);
        if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kKernel, &c) != cudaSuccess || n < 1) {
            cudaGetLastError();
            return FP8Z1_ECUDA;
        }
        if (dev < 16) holds[dev].store(n, std::memory_order_relaxed);
    }
    c.gridDim = dim3((unsigned)((most < n ? most : n) * kCluster));
    c.numAttrs = 2;
    count_launch();
    if (cudaLaunchKernelEx(&c, kKernel, args...) != cudaSuccess) {
        cudaGetLastError();
        return FP8Z1_ECUDA;
    }
    return launch_status();
}

// A tensor map over `rank` dimensions (innermost first; strides in bytes of
// dimensions 1..).  Returns a status.
int tensor_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const uint64_t* dims,
               const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);

// Waits that ran out in each translation unit's kernels on the current device
// (synchronous).  Returns a status.
int read_timeouts_gemm(unsigned* n);
int read_timeouts_wgrad(unsigned* n);
#if FP8Z1_CHECKED
int stall_gemm(unsigned kernels);
int stall_wgrad(unsigned kernels);
#endif

}  // namespace ffn
}  // namespace fp8z1
