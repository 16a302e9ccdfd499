// The gradient of the product's weight: sums over the token rows,
//
//   d_weight[k, n] = sum_t x[t, k] dz[t, n]        (of a transposed weight d_weight[n, k])
//
// in FP32 accuracy.  Where dz is dy itself, both operands are BF16 rows and enter as they lie:
// one product, every term exact.  Where dz is FP32 (an activation's, or FP32 dy) it
// enters as two FP16 numbers of 22 bits, every column of 256 rows at its own power of
// two, beside x in FP16, 256 rows x 128 columns at one: BF16's 8 bits fit whole.  One BF16
// product of a rounded dz would be twice as fast and lose 16 bits of it; three BF16 terms
// would hold all and take half as long again.
//
// A pair of CTAs owns 256 x 256 of the gradient: each 128 columns of dz (the lanes of its
// tensor memory) and half of x's 256 columns.  Both operands are row-major over tokens, M-
// and N-major to the tensor cores.  TMA steps of 64 rows, products into two accumulators,
// each 256 rows added up there (its adds do not round to nearest: 256 rows leave 7e-7 of
// the gradient's norm) and then scaled and added in registers.
//
// 2051 rows to 4096 x 14336 of FP32 dz: 303 us, 1.6 PFLOP/s of FP16 products; the tensor cores are busy 89 % of
// the time at 2048 rows and 7168 x 4096, 75 % with BF16 rows, whose half as many products share the same ends of tiles.
#include "linear.cuh"

namespace fp8z1 {
namespace linear {
namespace {

using namespace tc;
using ffn::after_previous;
using ffn::next_may_start;

__device__ unsigned g_timeouts;
#if FP8Z1_CHECKED
__device__ unsigned g_stall;  // bit kTurned: that kernel's first pair does not announce its first sums
#endif

constexpr int kCols = 256;
constexpr int kStep = 64;  // token rows of a stage
constexpr int kAdd = kTall / kStep;
constexpr int kThreads = 640;                // 4 warps that feed, 16 that add up
constexpr uint32_t kChunk = 64 * kStep * 2;  // bytes of 64 columns of a stage

template <int kTerms>
struct Shape {
    static constexpr int kStages = kTerms == 2 ? 4 : 6;
    static constexpr uint32_t kStageBytes = (2 * kTerms + 2) * kChunk;  // the terms of dz, half of x: 2 chunks each
    static constexpr uint32_t kSmem = kStages * kStageBytes + 16 * 2048 + 1024 + 256;
};

struct Args {
    const float *dz_factor, *x_factor;  // of 256 rows: a column of dz, 128 columns of x
    int64_t Np, x_blocks;
    float* out;
    int64_t N, K;
    int32_t T, m_tiles, n_tiles;  // m_tiles: of 128 columns of dz
};

// kTurned: the gradient is [N, K], dz's columns are its rows.
template <bool kTurned, int kTerms>
__global__ void __launch_bounds__(kThreads, 1)
wgrad_kernel(const __grid_constant__ CUtensorMap map_hi, const __grid_constant__ CUtensorMap map_lo,
             const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_out,
             const __grid_constant__ Args a)
{
    constexpr int kStages = Shape<kTerms>::kStages;
    constexpr uint32_t kStageBytes = Shape<kTerms>::kStageBytes;
    extern __shared__ uint8_t smem_raw[];
    next_may_start();
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    const uint32_t staging = base + kStages * kStageBytes, extra = staging + 16 * 2048;
    const uint32_t bar_full = extra, bar_empty = extra + 48, bar_acc = extra + 96, bar_free = extra + 112;
    volatile uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem_raw + (extra + 128 - smem_addr(smem_raw)));

    const int warp = of_warp((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const int sub = blockIdx.x & 1;  // of the pair
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(bar_full + 8 * i, 1);
            bar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(bar_acc + 8 * i, 1);
            bar_init(bar_free + 8 * i, 32);  // the adding warps of both CTAs
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
        prefetch_map(&map_hi);
        if (kTerms == 2) prefetch_map(&map_lo);
        prefetch_map(&map_x);
    }
    if (warp == 2) tmem_alloc<2, 512>(extra + 128);
    fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();  // the other CTA counts on this one's barriers from here on
    fence_after();
    after_previous();
    const uint32_t tmem = of_warp(*tmem_at);
    const int m_pairs = (a.m_tiles + 1) / 2;
    const int64_t total = (int64_t)m_pairs * a.n_tiles, i0 = blockIdx.x / 2, step = gridDim.x / 2;
    bool ok = true;

    if (warp < 4) {
        regs_less<48>();
        const bool one = one_lane();
        if (warp == 0) {
            Turn<kStages> turn;
            for (int64_t i = i0; i < total && ok; i += step) {
                const int n = (int)(i / m_pairs), m = (int)(i - (int64_t)n * m_pairs) * 2 + sub;
                for (int t = 0; t < a.T; t += kStep, turn.next()) {
                    if (!bar_wait_warp(bar_empty + 8 * turn.slot, turn.phase ^ 1)) {
                        ok = false;
                        break;
                    }
                    if (!one) continue;
                    // both CTAs' copies are counted in the first one, whose thread multiplies
                    if (sub == 0) bar_expect(bar_full + 8 * turn.slot, 2 * kStageBytes);
                    const uint32_t full = first_of_pair(bar_full + 8 * turn.slot), dst = base + turn.slot * kStageBytes;
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        load_2d_pair(dst + c * kChunk, &map_hi, full, m * 128 + c * 64, t);
                        if (kTerms == 2) load_2d_pair(dst + (2 + c) * kChunk, &map_lo, full, m * 128 + c * 64, t);
                        load_2d_pair(dst + (2 * kTerms + c) * kChunk, &map_x, full, n * kCols + sub * 128 + c * 64, t);
                    }
                }
            }
            // the copies in flight are read before the CTA ends, whatever became of the other warps
            for (int j = 0; j < kStages; ++j, turn.next()) ok &= bar_wait_warp(bar_empty + 8 * turn.slot, turn.phase ^ 1);
        } else if (warp == 1 && sub == 0) {
            constexpr uint32_t format = kTerms == 2 ? 0 : 1;  // F16, BF16
            constexpr uint32_t idesc = instruction_of(256, kCols, true, true, format, format);
            Turn<kStages> turn;
            Turn<2> acc;
            for (int64_t i = i0; i < total && ok; i += step) {
                for (int t0 = 0; t0 < a.T && ok; t0 += kTall, acc.next()) {
                    const uint32_t d = tmem + acc.slot * kCols;
                    ok = bar_wait_warp(bar_free + 8 * acc.slot, acc.phase ^ 1);
                    for (int s = 0; s < kAdd && t0 + s * kStep < a.T && ok; ++s, turn.next()) {
                        if (!bar_wait_warp(bar_full + 8 * turn.slot, turn.phase)) {
                            ok = false;
                            break;
                        }
                        fence_after();
                        if (!one) continue;
                        const uint32_t src = base + turn.slot * kStageBytes;
                        // 16 rows a product; rows past the end came as zeros
                        const int left = a.T - t0 - s * kStep, steps = left >= kStep ? 4 : (left + 15) / 16;
                        for (int k = 0; k < steps; ++k) {
                            // 8 rows are 1024 bytes; the next 64 columns follow a chunk later
                            const uint64_t db = operand(src + 2 * kTerms * kChunk + k * 2048, 1024, kChunk);
#pragma unroll
                            for (int q = 0; q < kTerms; ++q)
                                mma_f16_pair(d, operand(src + 2 * q * kChunk + k * 2048, 1024, kChunk), db, idesc, s + k + q > 0);
                        }
                        commit_pair(bar_empty + 8 * turn.slot);
                    }
#if FP8Z1_CHECKED
                    if (g_stall >> kTurned & 1 && blockIdx.x == 0 && i == i0 && t0 == 0) continue;
#endif
                    if (ok && one) commit_pair(bar_acc + 8 * acc.slot);
                }
            }
            // every product issued ends, and its sums are read, before the tensor memory is freed
            for (int j = 0; j < 2; ++j, acc.next()) ok = bar_wait_warp(bar_free + 8 * acc.slot, acc.phase ^ 1) && ok;
        }
    } else {
        regs_more<104>();
        const int group = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16, mine = staging + (warp - 4) * 2048;
        Turn<2> acc;
        for (int64_t i = i0; i < total; i += step) {
            const int n = (int)(i / m_pairs), m = (int)(i - (int64_t)n * m_pairs) * 2 + sub;
            uint64_t sums2[2][16];  // pairs of columns
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < 16; ++j) sums2[c][j] = 0;
            for (int t0 = 0; t0 < a.T; t0 += kTall, acc.next()) {
                float f0 = 1.0f, f1 = 1.0f;
                if (kTerms == 2) {  // read while the products run
                    const int64_t b = t0 / kTall;
                    const float f = m < a.m_tiles ? a.dz_factor[b * a.Np + m * 128 + row] : 0.0f;
                    f0 = f * a.x_factor[b * a.x_blocks + n * 2];
                    f1 = f * a.x_factor[b * a.x_blocks + min((int64_t)n * 2 + 1, a.x_blocks - 1)];
                }
                ok = ok && __all_sync(0xffffffffu, bar_wait(bar_acc + 8 * acc.slot, acc.phase));
                if (!ok) break;
                fence_after();
                const uint64_t f[2] = {pair(f0, f0), pair(f1, f1)};
                const uint32_t t = tmem + acc.slot * kCols + lanes + group * 32;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t r[16];
                    tmem_load(t + q / 2 * 128 + q % 2 * 16, r);
                    tmem_wait(r);
                    if (q == 3) {
                        fence_before();
                        __syncwarp();
                        if (lane == 0) bar_arrive_pair(first_of_pair(bar_free + 8 * acc.slot));
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sums2[q / 2][q % 2 * 8 + j] =
                            fma_pair(pair(r[2 * j], r[2 * j + 1]), f[q / 2], sums2[q / 2][q % 2 * 8 + j]);
                }
            }
            // a wait ran out: this tile and the pair's further ones are NaN
            if (!ok)
#pragma unroll
                for (int j = 0; j < 32; ++j) sums2[j / 16][j % 16] = pair(NAN, NAN);
            if (m >= a.m_tiles) continue;  // an odd last tile's other half
            float sum[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float2 v = unpair(sums2[c][j]);
                    sum[c][2 * j] = v.x;
                    sum[c][2 * j + 1] = v.y;
                }
            const int64_t col = (int64_t)m * 128 + row;  // of dz
            if constexpr (!kTurned) {
                // lanes are consecutive columns of the gradient
                if (col < a.N)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int64_t k0 = (int64_t)n * kCols + c * 128 + group * 32;
                        float* o = a.out + k0 * a.N + col;
#pragma unroll
                        for (int j = 0; j < 32; ++j, o += a.N)
                            if (k0 + j < a.K) __stcs(o, sum[c][j]);
                    }
            } else {
                // lanes are rows: pieces of 32 rows x 16 columns turn in shared memory and leave by TMA
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    if (lane == 0) store_wait_read<0>();
                    __syncwarp();
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const float* x = &sum[q / 2][q % 2 * 16 + v * 4];
                        // 64-byte swizzle: 16-byte units of a row change places with bits 1-2 of the row
                        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         mine + lane * 64 + ((v ^ (lane >> 1 & 3)) << 4)),
                                     "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3])
                                     : "memory");
                    }
                    fence_async();
                    __syncwarp();
                    const int64_t k0 = (int64_t)n * kCols + q / 2 * 128 + group * 32 + q % 2 * 16;
                    if (lane == 0) {
                        if (k0 < a.K && col < a.N) store_2d(&map_out, mine, (int)k0, (int)col);
                        store_commit();
                    }
                }
            }
        }
        if (kTurned && lane == 0) store_wait_all();
    }
    if (!ok) atomicAdd(&g_timeouts, 1u);
    fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();  // no CTA leaves while the other may still write to it
    fence_after();
    if (warp == 2) tmem_free<2, 512>(tmem);
}

// 64 columns x 64 rows of row-major 16-bit numbers
int map_16(CUtensorMap* map, CUtensorMapDataType type, const void* p, int64_t rows, int64_t cols, int64_t ld)
{
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, stride[1] = {(uint64_t)ld * 2};
    const uint32_t box[2] = {64, kStep};
    return ffn::tensor_map(map, type, 2, p, dims, stride, box);
}

template <bool kTurned, int kTerms>
int launch(const Wgrad& g, cudaStream_t s)
{
    CUtensorMap hi, lo, x, out;
    int st;
    if (kTerms == 2) {
        if ((st = map_16(&hi, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, g.b.dz_hi, g.T, g.Np, g.Np)) != FP8Z1_OK ||
            (st = map_16(&lo, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, g.b.dz_lo, g.T, g.Np, g.Np)) != FP8Z1_OK ||
            (st = map_16(&x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, g.b.x16, g.T, g.Kp, g.Kp)) != FP8Z1_OK)
            return st;
    } else {
        if ((st = map_16(&hi, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.dz, g.T, g.N, g.ld_dz)) != FP8Z1_OK ||
            (st = map_16(&x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, g.x, g.T, g.K, g.ld_x)) != FP8Z1_OK)
            return st;
        lo = hi;
    }
    out = x;
    if (kTurned) {
        const uint64_t dims[2] = {(uint64_t)g.K, (uint64_t)g.N}, stride[1] = {(uint64_t)g.K * 4};
        const uint32_t box[2] = {16, 32};
        if ((st = ffn::tensor_map(&out, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, g.out, dims, stride, box,
                                  CU_TENSOR_MAP_SWIZZLE_64B)) != FP8Z1_OK)
            return st;
    }
    Args a = {};
    a.dz_factor = g.b.dz_factor;
    a.x_factor = g.b.x_factor;
    a.Np = g.Np;
    a.x_blocks = g.Kp / 128;
    a.out = g.out;
    a.N = g.N;
    a.K = g.K;
    a.T = (int32_t)g.T;
    a.m_tiles = (int32_t)ceil_div(g.N, 128);
    a.n_tiles = (int32_t)ceil_div(g.K, kCols);
    const int64_t total = (int64_t)((a.m_tiles + 1) / 2) * a.n_tiles;
    return ffn::launch_persistent<wgrad_kernel<kTurned, kTerms>, 2>(kThreads, Shape<kTerms>::kSmem, total, s, hi, lo, x, out, a);
}

}  // namespace

int launch_wgrad(const Wgrad& g, cudaStream_t s)
{
    if (g.exact) return g.k_major ? launch<true, 1>(g, s) : launch<false, 1>(g, s);
    return g.k_major ? launch<true, 2>(g, s) : launch<false, 2>(g, s);
}

int read_timeouts_wgrad(unsigned* n)
{
    return cudaMemcpyFromSymbol(n, g_timeouts, 4) == cudaSuccess ? FP8Z1_OK : FP8Z1_ECUDA;
}

#if FP8Z1_CHECKED
int stall_wgrad(unsigned kernels)
{
    return cudaMemcpyToSymbol(g_stall, &kernels, 4) == cudaSuccess ? FP8Z1_OK : FP8Z1_ECUDA;
}
#endif

}  // namespace linear
}  // namespace fp8z1
