// The products of rows with an FP8 weight, y = act(x w + bias) + residual.
//
// A row is one FP8 number an element with a scale for every 128 (8-bit rows), or a pair
// of them (BF16 rows: E4M3 and E5M2 hold their 8 bits; FP32 rows, rounded to 9 bits: E4M3
// twice), so the weight's codes enter the tensor cores as they are:
//
//   sum_k x_k w_kn = sum over blocks b of 128 of k  s_b c_bn  sum_{k in b} (hi + lo)_k w_kn.
//
// The inner sums are exact products accumulated in FP32 in tensor memory; other
// warps scale each block's and add it to the tile's sums in registers while the
// next is multiplied.
//
// Many rows: a pair of CTAs has 256 rows x 256 columns, each the sums of 128 rows and half
// the weight's columns in shared memory, as a CTA alone would need 96 bytes of operands a
// clock for 8-bit rows, more than L2 delivers to every SM at once.
//
// Few rows: the weight's columns take the rows' place, 128 to a CTA, and 16 to 128 rows of x
// the columns': the products' time follows the rows, and the codes are what is read.  K is
// split over a cluster's CTAs, whose sums are added in shared memory in their order.
//
// Many rows: 4096 8-bit rows of 7168 x 4096 take 120 us, 2.0 PFLOP/s, 8192 207 us, 2.3 PFLOP/s: the additions and the
// way from product to additions and back bound it, and 256 tiles are 3.4 rounds of 76 pairs.  2051
// BF16 rows of 4096 x 14336 169 us with the 9 of their pairs, 1.4 PFLOP/s (a ninth of the tiles' rows is padding), with GELU
// and the saved z 215: the end of a tile, which nothing overlaps.  Few rows, in a captured graph with cold caches: 1 8-bit row of 4096 x 14336 14 us,
// 61 BF16 rows of 7168 x 4096 16: the first codes' way and the split's join, not the codes' rate.
#include <cooperative_groups.h>

#include <atomic>

#include "linear.cuh"

namespace fp8z1 {
namespace linear {
namespace {

using namespace tc;
using ffn::after_previous;
using ffn::next_may_start;
namespace cg = cooperative_groups;

__device__ unsigned g_timeouts;
#if FP8Z1_CHECKED
__device__ unsigned g_stall;  // bit 0: many rows, 1: few rows: the first CTA does not announce its first sums
std::atomic<bool> g_all_few{false};  // every product by the kernel of few rows
#endif

constexpr uint32_t kOperand = 128 * 128;  // bytes of a 128 x 128 operand tile
constexpr int kStagePitch = 48;           // of a row's 32 bytes on their way out

struct Args {
    Out o;
    const float* a_scale;
    int64_t scale_row, scale_block;
    const float* b_scale;
    int32_t b_col, b_step;  // strides of b_scale: a block of columns, a block of k
    int32_t b_cols;         // blocks of columns
    int32_t k_blocks;
    uint32_t idesc[2];      // of the products with hi, with lo
    int32_t m_tiles, n_tiles;
    int32_t splits;         // few rows: CTAs of a cluster
};

// ---- what becomes of the sums -----------------------------------------------------------

// 32 bytes of each of a warp's rows, a lane's own in w[2], through shared memory: two lanes store a row's, so that a
// sector is written whole.
__device__ __forceinline__ void store_rows(uint8_t* stage, int lane, int rows, const uint4 (&w)[2], uint8_t* to, int64_t pitch)
{
    *reinterpret_cast<uint4*>(stage + lane * kStagePitch) = w[0];
    *reinterpret_cast<uint4*>(stage + lane * kStagePitch + 16) = w[1];
    __syncwarp();
#pragma unroll
    for (int r = lane >> 1; r < 32; r += 16)
        if (r < rows)
            *reinterpret_cast<uint4*>(to + r * pitch + (lane & 1) * 16) =
                *reinterpret_cast<const uint4*>(stage + r * kStagePitch + (lane & 1) * 16);
    __syncwarp();
}

// 8 columns of each of a warp's rows, a lane's own in v, to rows of any alignment (of `cols` columns from here on):
// eight lanes store a row's, so that an instruction touches a few sectors, not 32.
template <class T>
__device__ __forceinline__ void store_any(uint8_t* stage, int lane, int rows, const float (&v)[8], T* to, int64_t ld, int64_t cols)
{
    *reinterpret_cast<float4*>(stage + lane * kStagePitch) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(stage + lane * kStagePitch + 16) = make_float4(v[4], v[5], v[6], v[7]);
    __syncwarp();
    const int c = lane & 7;
#pragma unroll
    for (int r = lane >> 3; r < 32; r += 4)
        if (r < rows && c < cols) to[r * ld + c] = from_float<T>(*reinterpret_cast<const float*>(stage + r * kStagePitch + c * 4));
    __syncwarp();
}

// 16 neighbouring columns of a row a lane (a warp: 32 rows, of which `rows` exist), from column n0 on; `first` the
// warp's first row.  Eight at a time: the sums of the other columns wait in registers.
__device__ __forceinline__ void finish(const Out& o, const uint64_t (&sums)[8], int64_t first, int lane, int rows, int64_t n0,
                                       uint8_t* stage)
{
    const bool here = lane < rows, whole = n0 + 16 <= o.N, staged = whole && o.vec_y;
    const int64_t row = first + lane;
    uint4 w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int64_t c = n0 + 8 * h;
        float v[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 two = unpair(sums[4 * h + j]);
            v[2 * j] = two.x;
            v[2 * j + 1] = two.y;
        }
        if (o.bias && whole && o.vec_bias) {
            const float4 p = __ldg(reinterpret_cast<const float4*>(o.bias + c)), q = __ldg(reinterpret_cast<const float4*>(o.bias + c + 4));
            v[0] += p.x, v[1] += p.y, v[2] += p.z, v[3] += p.w, v[4] += q.x, v[5] += q.y, v[6] += q.z, v[7] += q.w;
        } else if (o.bias) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < o.N) v[j] += __ldg(o.bias + c + j);
        }
        if (o.pre && whole && o.vec_pre) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                w[q] = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                                  __float_as_uint(v[4 * q + 3]));
            store_rows(stage, lane, rows, w, reinterpret_cast<uint8_t*>(o.pre + first * o.N + c), o.N * 4);
        } else if (o.pre) {
            store_any(stage, lane, rows, v, o.pre + first * o.N + c, o.N, o.N - c);
        }
        if (o.act != FP8Z1_ACT_NONE)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = activate(v[j], o.act);
        if (o.residual && here) {
            const bf16* p = o.residual + row * o.ld_r + c;
            if (whole && o.vec_r) {
                const uint4 u = *reinterpret_cast<const uint4*>(p);
                const uint32_t r[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[2 * j] += __uint_as_float(r[j] << 16);
                    v[2 * j + 1] += __uint_as_float(r[j] & 0xffff0000u);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < o.N) v[j] += to_float(p[j]);
            }
        }
        if (!staged) {
            if (o.f32)
                store_any(stage, lane, rows, v, static_cast<float*>(o.y) + first * o.ld_y + c, o.ld_y, o.N - c);
            else
                store_any(stage, lane, rows, v, static_cast<bf16*>(o.y) + first * o.ld_y + c, o.ld_y, o.N - c);
        } else if (o.f32) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                w[q] = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                                  __float_as_uint(v[4 * q + 3]));
            store_rows(stage, lane, rows, w, reinterpret_cast<uint8_t*>(static_cast<float*>(o.y) + first * o.ld_y + c), o.ld_y * 4);
        } else {
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                u[j] = *reinterpret_cast<const uint32_t*>(&two);
            }
            // 16 bytes wait for the next
            if (h == 0) {
                *reinterpret_cast<uint4*>(stage + lane * kStagePitch + 32) = make_uint4(u[0], u[1], u[2], u[3]);
            } else {
                w[0] = *reinterpret_cast<const uint4*>(stage + lane * kStagePitch + 32);
                w[1] = make_uint4(u[0], u[1], u[2], u[3]);
                store_rows(stage, lane, rows, w, reinterpret_cast<uint8_t*>(static_cast<bf16*>(o.y) + first * o.ld_y + n0), o.ld_y * 2);
            }
        }
    }
}

// The same for a warp's columns n0 .. n0 + 31 and n0 + 128 .. n0 + 159 of 32 rows where all lies on 16 bytes; without
// kMore a bias at most and BF16 rows.  The products of a tile run two steps on while its results leave, so what
// `finish` asks of every element cost 1400 to 2200 clocks a 16 columns: 8192 8-bit rows of 7168 x 4096 217 us with it, 205
// with this, 2051 BF16 rows of 4096 x 14336 179 and 168, with GELU by __expf and z 214 and 206.  In a kernel without `finish`: beside it
// the sums of the loop spilled.
bool is_whole(const Out& o)
{
    return o.vec_y && o.N % 16 == 0 && (!o.bias || o.vec_bias) && (!o.residual || o.vec_r) && (!o.pre || o.vec_pre);
}
template <bool kMore>
__device__ __forceinline__ void finish_whole(const Out& o, const float (&sums)[2][32], int64_t first, int lane, int rows, int64_t n0,
                                             uint8_t* stage)
{
    const int r = lane >> 1;
    const bool upper = r < rows, lower = r + 16 < rows;
    uint4* put = reinterpret_cast<uint4*>(stage + lane * kStagePitch);
    const uint4* get = reinterpret_cast<const uint4*>(stage + r * kStagePitch + (lane & 1) * 16);
    const uint4* get_lower = reinterpret_cast<const uint4*>(stage + (r + 16) * kStagePitch + (lane & 1) * 16);
    // 32 bytes a row, two lanes each
    auto leave = [&](const uint4& w0, const uint4& w1, uint8_t* to, int64_t pitch) {
        put[0] = w0, put[1] = w1;
        __syncwarp();
        if (upper) *reinterpret_cast<uint4*>(to + r * pitch + (lane & 1) * 16) = *get;
        if (lower) *reinterpret_cast<uint4*>(to + (r + 16) * pitch + (lane & 1) * 16) = *get_lower;
        __syncwarp();
    };
    // 64 bytes a row, 16 rows at a time, four lanes each
    auto leave_floats = [&](const float (&v)[16], float* to, int64_t ld) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (lane >> 4 == h)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float4*>(stage + (lane & 15) * 80 + i * 16) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = i * 8 + (lane >> 2), row = h * 16 + at;
                if (row < rows)
                    *reinterpret_cast<float4*>(to + row * ld + (lane & 3) * 4) = *reinterpret_cast<const float4*>(stage + at * 80 + (lane & 3) * 16);
            }
            __syncwarp();
        }
    };
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int64_t c = n0 + q / 2 * 128 + q % 2 * 16;
        if (c >= o.N) break;  // with the whole warp
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = sums[q / 2][q % 2 * 16 + j];
        if (o.bias)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 b = __ldg(reinterpret_cast<const float4*>(o.bias + c) + j);
                v[4 * j] += b.x, v[4 * j + 1] += b.y, v[4 * j + 2] += b.z, v[4 * j + 3] += b.w;
            }
        if constexpr (kMore) {
            if (o.pre) leave_floats(v, o.pre + first * o.N + c, o.N);
            if (o.act == FP8Z1_ACT_SILU)
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = activate(v[j], FP8Z1_ACT_SILU);
            else if (o.act != FP8Z1_ACT_NONE)
#pragma unroll
                for (int j = 0; j < 16; ++j) v[j] = activate(v[j], FP8Z1_ACT_GELU_TANH);
            if (o.residual && lane < rows) {
                const uint4* p = reinterpret_cast<const uint4*>(o.residual + (first + lane) * o.ld_r + c);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 u = p[i];
                    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[8 * i + 2 * j] += __uint_as_float(w[j] << 16);
                        v[8 * i + 2 * j + 1] += __uint_as_float(w[j] & 0xffff0000u);
                    }
                }
            }
            if (o.f32) {
                leave_floats(v, static_cast<float*>(o.y) + first * o.ld_y + c, o.ld_y);
                continue;
            }
        }
        uint32_t u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
            u[j] = *reinterpret_cast<const uint32_t*>(&two);
        }
        leave(make_uint4(u[0], u[1], u[2], u[3]), make_uint4(u[4], u[5], u[6], u[7]),
              reinterpret_cast<uint8_t*>(static_cast<bf16*>(o.y) + first * o.ld_y + c), o.ld_y * 2);
    }
}

// And for FP32 rows of any alignment with a bias at most: 16 columns of 16 rows at a time, 16 lanes a row.  1001 rows of
// 4096 to 50001 logits: 280 us, with `finish` 305.
__device__ __forceinline__ void finish_odd(const Out& o, const float (&sums)[2][32], int64_t first, int lane, int rows, int64_t n0,
                                           uint8_t* stage)
{
    const int r = lane >> 4, k = lane & 15;
    const float* get = reinterpret_cast<const float*>(stage + r * 80 + k * 4);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int64_t c = n0 + q / 2 * 128 + q % 2 * 16;
        if (c >= o.N) break;  // with the whole warp
        const bool in = c + k < o.N;
        const float b = o.bias && in ? __ldg(o.bias + c + k) : 0.0f;
        float* to = static_cast<float*>(o.y) + (first + r) * o.ld_y + c + k;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (r == h)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float* v = &sums[q / 2][q % 2 * 16 + 4 * i];
                    *reinterpret_cast<float4*>(stage + k * 80 + i * 16) = make_float4(v[0], v[1], v[2], v[3]);
                }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 8; ++i, to += 2 * o.ld_y)
                if (in && h * 16 + 2 * i + r < rows) *to = get[i * 40] + b;
            __syncwarp();
        }
    }
}

// ---- many rows ------------------------------------------------------------------------------

constexpr int kCols = 256;
constexpr int kManyThreads = 640;  // 4 warps that feed, 16 that add up
template <int kTerms>
struct Many {
    static constexpr int kStages = kTerms == 2 ? 4 : 6;
    static constexpr uint32_t kStageBytes = (kTerms + 1) * kOperand;  // hi, lo, half of the weight's columns
    // stages, barriers, factors, rows on their way out
    static constexpr uint32_t kSmem = kStages * kStageBytes + 1024 + 256 + 8192 + 16 * 32 * kStagePitch;
};

template <int kTerms, bool kKMajor, bool kWhole>
__global__ void __launch_bounds__(kManyThreads, 1)
many_kernel(const __grid_constant__ CUtensorMap map_hi, const __grid_constant__ CUtensorMap map_lo,
            const __grid_constant__ CUtensorMap map_w, const __grid_constant__ Args a)
{
    constexpr int kStages = Many<kTerms>::kStages;
    constexpr uint32_t kStageBytes = Many<kTerms>::kStageBytes;
    extern __shared__ uint8_t smem_raw[];
    next_may_start();
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    const uint32_t extra = base + kStages * kStageBytes;
    // extra: full, empty [kStages], accumulators ready, free [2], factors ready, read [2], tensor memory base; factors
    // [2][4 steps][2][128]; rows on their way out
    const uint32_t bar_full = extra, bar_empty = extra + 48, bar_acc = extra + 96, bar_free = extra + 112,
                   bar_factors = extra + 128, bar_read = extra + 144, factors = extra + 256;
    uint8_t* extra_ptr = smem_raw + (extra - smem_addr(smem_raw));
    volatile uint32_t* tmem_at = reinterpret_cast<uint32_t*>(extra_ptr + 192);

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
        for (int i = 0; i < 2; ++i) {
            bar_init(bar_factors + 8 * i, 32);
            bar_init(bar_read + 8 * i, 16);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
        prefetch_map(&map_hi);
        if (kTerms == 2) prefetch_map(&map_lo);
        prefetch_map(&map_w);
    }
    if (warp == 2) tmem_alloc<2, 512>(extra + 192);
    fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();  // the other CTA counts on this one's barriers from here on
    fence_after();
    after_previous();
    const uint32_t tmem = of_warp(*tmem_at);
    const int64_t total = (int64_t)a.m_tiles * a.n_tiles, i0 = blockIdx.x / 2, step = gridDim.x / 2;
    bool ok = true;

    if (warp < 4) {
        regs_less<48>();
        const bool one = one_lane();
        if (warp == 0) {
            Turn<kStages> turn;
            for (int64_t i = i0; i < total && ok; i += step) {
                const int n = (int)(i / a.m_tiles), m = (int)(i - (int64_t)n * a.m_tiles);
                const int row = m * 256 + sub * 128, col = n * kCols + sub * 128;
                for (int kb = 0; kb < a.k_blocks; ++kb, turn.next()) {
                    if (!bar_wait_warp(bar_empty + 8 * turn.slot, turn.phase ^ 1)) {
                        ok = false;
                        break;
                    }
                    if (!one) continue;
                    // both CTAs' copies are counted in the first one, whose thread multiplies
                    if (sub == 0) bar_expect(bar_full + 8 * turn.slot, 2 * kStageBytes);
                    const uint32_t full = first_of_pair(bar_full + 8 * turn.slot), dst = base + turn.slot * kStageBytes;
                    load_2d_pair(dst, &map_hi, full, kb * 128, row);
                    if (kTerms == 2) load_2d_pair(dst + kOperand, &map_lo, full, kb * 128, row);
                    if (kKMajor)
                        load_2d_pair(dst + kTerms * kOperand, &map_w, full, kb * 128, col);
                    else
                        load_2d_pair(dst + kTerms * kOperand, &map_w, full, col, kb * 128);
                }
            }
            // the copies in flight are read before the CTA ends, whatever became of the other warps
            for (int j = 0; j < kStages; ++j, turn.next()) ok &= bar_wait_warp(bar_empty + 8 * turn.slot, turn.phase ^ 1);
        } else if (warp & 1 && sub == 0) {
            // Two warps take the steps in turn, each with its accumulator: a step's barriers take one some 250 clocks,
            // while the other's products run.  An even number of stages gives each warp stages of its own: one that the
            // other has not seen filled would pass for filled again.
            static_assert(kStages % 2 == 0, "stages of its own");
            const int odd = warp >> 1;
            Turn<kStages> turn;
            if (odd) turn.next();
            uint32_t phase = 0;
            const int64_t count = (total > i0 ? (total - i0 + step - 1) / step : 0) * a.k_blocks;  // of all tiles
            for (int64_t n = odd; n < count; n += 2, turn.next(), turn.next(), phase ^= 1) {
                if (!bar_wait_warp(bar_full + 8 * turn.slot, turn.phase) || !bar_wait_warp(bar_free + 8 * odd, phase ^ 1)) {
                    ok = false;
                    break;
                }
                fence_after();
                if (!one) continue;
                const uint32_t src = base + turn.slot * kStageBytes, d = tmem + odd * kCols;
#pragma unroll
                for (int t = 0; t < kTerms; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint64_t da = operand(src + t * kOperand + k * 32, 1024, 16);
                        // K-major: 8 columns are 1024 bytes; N-major: 8 k are
                        const uint64_t db = operand(src + kTerms * kOperand + k * (kKMajor ? 32 : 4096), 1024, 16);
                        mma_f8_pair(d, da, db, a.idesc[t], t + k > 0);
                    }
                commit_pair(bar_empty + 8 * turn.slot);
#if FP8Z1_CHECKED
                if (g_stall & 1 && blockIdx.x == 0 && n == 0) continue;
#endif
                commit_pair(bar_acc + 8 * odd);
            }
            // every product issued ends, and its sums are read, before the tensor memory is freed
            ok = bar_wait_warp(bar_free + 8 * odd, phase ^ 1) && ok;
        } else if (warp == 2) {
            // the factors of four steps at a time, s_b c_bn of both chunks of 128 columns for four rows a thread
            Turn<2> turn;
            for (int64_t i = i0; i < total && ok; i += step) {
                const int n = (int)(i / a.m_tiles), m = (int)(i - (int64_t)n * a.m_tiles);
                const int64_t row = (int64_t)m * 256 + sub * 128 + lane;  // rows and columns past the end: any others' scales
                const float* pa[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) pa[j] = a.a_scale + min(row + 32 * j, a.o.T - 1) * a.scale_row;
                const float* p0 = a.b_scale + (int64_t)min(n * 2, a.b_cols - 1) * a.b_col;
                const float* p1 = a.b_scale + (int64_t)min(n * 2 + 1, a.b_cols - 1) * a.b_col;
                for (int kb = 0; kb < a.k_blocks; kb += 4, turn.next()) {
                    float v[4][4], c0[4], c1[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int64_t at = min(kb + k, a.k_blocks - 1);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[k][j] = pa[j][at * a.scale_block];
                        c0[k] = p0[at * a.b_step];
                        c1[k] = p1[at * a.b_step];
                    }
                    if (!bar_wait_warp(bar_read + 8 * turn.slot, turn.phase ^ 1)) {
                        ok = false;
                        break;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t f = factors + (turn.slot * 4 + k) * 1024 + (lane + 32 * j) * 4;
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(f), "f"(v[k][j] * c0[k]) : "memory");
                            asm volatile("st.shared.f32 [%0], %1;" ::"r"(f + 512), "f"(v[k][j] * c1[k]) : "memory");
                        }
                    bar_arrive(bar_factors + 8 * turn.slot);
                }
            }
        }
    } else {
        regs_more<104>();
        const int group = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16;
        uint8_t* stage = extra_ptr + 256 + 8192 + (warp - 4) * 32 * kStagePitch;
        const uint32_t bar_free_first = first_of_pair(bar_free);
        Turn<2> acc, turn;
        for (int64_t i = i0; i < total; i += step) {
            const int n = (int)(i / a.m_tiles), m = (int)(i - (int64_t)n * a.m_tiles);
            float sums[2][32];  // scalars: pairs for two additions an instruction cost the moves that made them (130 us for 120)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < 32; ++j) sums[c][j] = 0.0f;
            bool ready = false;  // the step's sums are known to be there
            for (int kb = 0; kb < a.k_blocks; ++kb) {
                // a warp's lanes agree on the outcome: the loads below are warp-wide
                if ((kb & 3) == 0) ok = ok && bar_wait_warp(bar_factors + 8 * turn.slot, turn.phase);
                const uint32_t at = factors + (turn.slot * 4 + (kb & 3)) * 1024 + row * 4;
                float f[2];
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[0]) : "r"(at));
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[1]) : "r"(at + 512));
                if (!ready) ok = ok && bar_wait_warp(bar_acc + 8 * acc.slot, acc.phase);
                if (!ok) break;
                fence_after();
                const uint32_t t = tmem + acc.slot * kCols + lanes + group * 32, free = bar_free_first + 8 * acc.slot;
                acc.next();
                bool next = false;
                // columns 32 group + {0 .. 31, 128 .. 159}, 32 on their way at once
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t r[32];
                    tmem_load(t + c * 128, r);
                    tmem_wait(r);
                    if (c) {
                        fence_before();
                        __syncwarp();
                        bar_arrive_pair_first(free, lane);
                        // asked beside the additions: a wait takes some 130 clocks, and a step's chain is what bounds 8-bit rows
                        next = bar_test(bar_acc + 8 * acc.slot, acc.phase);
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) sums[c][j] = __fmaf_rn(__uint_as_float(r[j]), f[c], sums[c][j]);
                }
                ready = __all_sync(0xffffffffu, next);
                if ((kb & 3) == 3 || kb + 1 == a.k_blocks) {
                    if (lane == 0) bar_arrive(bar_read + 8 * turn.slot);
                    turn.next();
                }
            }
            // a wait ran out: this tile and the pair's further ones are NaN
            if (!ok)
#pragma unroll
                for (int j = 0; j < 64; ++j) sums[j / 32][j % 32] = NAN;
            const int64_t first = (int64_t)m * 256 + sub * 128 + (warp & 3) * 32;  // row of the warp
            const int rows = (int)min(max(a.o.T - first, (int64_t)0), (int64_t)32);
            const int64_t n0 = (int64_t)n * kCols + group * 32;
            const bool plain = a.o.act == FP8Z1_ACT_NONE && !a.o.residual && !a.o.pre;
            if constexpr (kWhole) {
                if (plain && !a.o.f32)
                    finish_whole<false>(a.o, sums, first, lane, rows, n0, stage);
                else
                    finish_whole<true>(a.o, sums, first, lane, rows, n0, stage);
            } else if (plain && a.o.f32) {
                finish_odd(a.o, sums, first, lane, rows, n0, stage);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int64_t c = n0 + q / 2 * 128 + q % 2 * 16;
                    if (c >= a.o.N || rows == 0) continue;  // with the whole warp
                    uint64_t v[8];  // in pairs they need no registers of their own
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = pair(sums[q / 2][q % 2 * 16 + 2 * j], sums[q / 2][q % 2 * 16 + 2 * j + 1]);
                    finish(a.o, v, first, lane, rows, c, stage);
                }
            }
        }
    }
    if (!ok) atomicAdd(&g_timeouts, 1u);
    fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();  // no CTA leaves while the other may still write to it
    fence_after();
    if (warp == 2) tmem_free<2, 512>(tmem);
}

// ---- few rows ---------------------------------------------------------------------------------

// kN rows of x; 4 warps feed, 4 for each 32 rows add up.  Two CTAs share an SM up to 64 rows.
template <int kTerms, int kN>
struct Few {
    static constexpr int kGroups = kN <= 32 ? 1 : kN / 32, kMine = kN / kGroups;  // rows of an adding warp
    static constexpr int kThreads = 128 + 128 * kGroups;
    static constexpr uint32_t kRowBytes = kN * 128;  // of a term
    static constexpr uint32_t kStageBytes = kOperand + kTerms * kRowBytes;
    static constexpr int kResident = kN <= 64 ? 2 : 1;
    static constexpr int kStages = kN <= 64 ? (int)(100 * 1024 / kStageBytes) : 4;
    static constexpr uint32_t kAt = 256, kSmem = kStages * kStageBytes + 1024 + kAt + 8 * kN * 4;
    static constexpr int kTmem = 2 * kN < 32 ? 32 : 2 * kN;
    static_assert(kStages >= 3 && kStages <= 6 && kStages * kStageBytes >= kN * 512, "the sums of a split fit the stages");
};

template <int kTerms, int kN, bool kKMajor>
__global__ void __launch_bounds__(Few<kTerms, kN>::kThreads, Few<kTerms, kN>::kResident)
few_kernel(const __grid_constant__ CUtensorMap map_hi, const __grid_constant__ CUtensorMap map_lo,
           const __grid_constant__ CUtensorMap map_w, const __grid_constant__ Args a)
{
    using S = Few<kTerms, kN>;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    next_may_start();
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    const uint32_t extra = base + kStages * S::kStageBytes;
    // extra: full, empty [kStages], accumulators ready, free [2], factors ready, read [2], tensor memory base, whether
    // a wait ran out; factors [2][4 steps][kN]
    const uint32_t bar_full = extra, bar_empty = extra + 48, bar_acc = extra + 96, bar_free = extra + 112,
                   bar_factors = extra + 128, bar_read = extra + 144, factors = extra + S::kAt;
    uint8_t* extra_ptr = smem_raw + (extra - smem_addr(smem_raw));
    volatile uint32_t* tmem_at = reinterpret_cast<uint32_t*>(extra_ptr + 192);
    uint32_t* failed = reinterpret_cast<uint32_t*>(extra_ptr + 196);
    float* sums_at = reinterpret_cast<float*>(extra_ptr - kStages * S::kStageBytes);  // [kN][128], over the stages
    cg::cluster_group cluster = cg::this_cluster();

    const int warp = of_warp((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    // the rows' tiles outermost, in one dimension of the grid (another would hold 65535; the rule below takes some 1600 at
    // most for K up to 11000, and a larger K leaves no memory for 65535: its gain is a part of a round of the SMs)
    const int tile = blockIdx.x / a.splits, split = blockIdx.x - tile * a.splits, m = tile / a.n_tiles, n = tile - m * a.n_tiles;
    const int token0 = m * kN;
    const int k0 = a.k_blocks * split / a.splits, k1 = a.k_blocks * (split + 1) / a.splits;
    if (threadIdx.x == 0) {
        *failed = 0;
        for (int i = 0; i < kStages; ++i) {
            bar_init(bar_full + 8 * i, 1);
            bar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(bar_acc + 8 * i, 1);
            bar_init(bar_free + 8 * i, 4 * S::kGroups);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(bar_factors + 8 * i, 32);
            bar_init(bar_read + 8 * i, 4 * S::kGroups);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
        prefetch_map(&map_hi);
        if (kTerms == 2) prefetch_map(&map_lo);
        prefetch_map(&map_w);
    }
    if (warp == 2) tmem_alloc<1, S::kTmem>(extra + 192);
    fence_before();
    __syncthreads();
    __syncwarp();
    fence_after();
    const uint32_t tmem = of_warp(*tmem_at);
    bool ok = true;

    if (warp == 0) {
        const bool one = one_lane();
        auto codes = [&](int kb, uint32_t full, uint32_t dst) {
            bar_expect(full, S::kStageBytes);
            if (kKMajor)
                load_2d(dst, &map_w, full, kb * 128, n * 128);
            else
                load_2d(dst, &map_w, full, n * 128, kb * 128);
        };
        // the first codes are on their way before the kernel ahead has ended: it does not write them
        const int ahead = min(kStages, k1 - k0);
        if (one)
            for (int i = 0; i < ahead; ++i) codes(k0 + i, bar_full + 8 * i, base + i * S::kStageBytes);
        after_previous();
        Turn<kStages> turn;
        for (int kb = k0; kb < k1; ++kb, turn.next()) {
            const uint32_t full = bar_full + 8 * turn.slot, dst = base + turn.slot * S::kStageBytes;
            if (kb >= k0 + ahead && !bar_wait_warp(bar_empty + 8 * turn.slot, turn.phase ^ 1)) {
                ok = false;
                break;
            }
            if (!one) continue;
            if (kb >= k0 + ahead) codes(kb, full, dst);
            load_2d(dst + kOperand, &map_hi, full, kb * 128, token0);
            if (kTerms == 2) load_2d(dst + kOperand + S::kRowBytes, &map_lo, full, kb * 128, token0);
        }
        // the copies in flight are read before the CTA ends, whatever became of the other warps
        for (int j = 0; j < kStages; ++j, turn.next()) ok &= bar_wait_warp(bar_empty + 8 * turn.slot, turn.phase ^ 1);
    } else if (warp == 1) {
        const bool one = one_lane();
        Turn<kStages> turn;
        Turn<2> acc;
        for (int kb = k0; kb < k1; ++kb, turn.next(), acc.next()) {
            if (!bar_wait_warp(bar_full + 8 * turn.slot, turn.phase) || !bar_wait_warp(bar_free + 8 * acc.slot, acc.phase ^ 1)) {
                ok = false;
                break;
            }
            fence_after();
            if (!one) continue;
            const uint32_t src = base + turn.slot * S::kStageBytes, d = tmem + acc.slot * kN;
#pragma unroll
            for (int t = 0; t < kTerms; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint64_t da = operand(src + k * (kKMajor ? 32 : 4096), 1024, 16);
                    const uint64_t db = operand(src + kOperand + t * S::kRowBytes + k * 32, 1024, 16);
                    mma_f8(d, da, db, a.idesc[t], t + k > 0);
                }
            commit(bar_empty + 8 * turn.slot);
#if FP8Z1_CHECKED
            if (g_stall & 2 && blockIdx.x == 0 && kb == k0) continue;
#endif
            commit(bar_acc + 8 * acc.slot);
        }
        // every product issued ends, and its sums are read, before the tensor memory is freed
        for (int j = 0; j < 2; ++j, acc.next()) ok = bar_wait_warp(bar_free + 8 * acc.slot, acc.phase ^ 1) && ok;
    } else if (warp == 2) {
        after_previous();
        // the factors of four steps at a time
        Turn<2> turn;
        constexpr int kEach = (kN + 31) / 32;
        const float* pb = a.b_scale + (int64_t)n * a.b_col;
        const float* pa[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i)
            pa[i] = a.a_scale + min((int64_t)token0 + min(lane + 32 * i, kN - 1), a.o.T - 1) * a.scale_row;
        for (int kb = k0; kb < k1; kb += 4, turn.next()) {
            float c[4], v[4][kEach];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t at = min(kb + k, k1 - 1);
                c[k] = pb[at * a.b_step];
#pragma unroll
                for (int i = 0; i < kEach; ++i) v[k][i] = pa[i][at * a.scale_block];
            }
            if (!bar_wait_warp(bar_read + 8 * turn.slot, turn.phase ^ 1)) {
                ok = false;
                break;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < kEach; ++i)
                    if (lane + 32 * i < kN)
                        asm volatile("st.shared.f32 [%0], %1;" ::"r"(factors + ((turn.slot * 4 + k) * kN + lane + 32 * i) * 4),
                                     "f"(v[k][i] * c[k])
                                     : "memory");
            bar_arrive(bar_factors + 8 * turn.slot);
        }
    }
    const int adder = threadIdx.x - 128, group = adder >> 7, out = adder & 127;  // the sums' column of y in this CTA
    float sums[S::kMine];
    if (warp >= 4) {
        const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16;
        Turn<2> acc, turn;
#pragma unroll
        for (int j = 0; j < S::kMine; ++j) sums[j] = 0.0f;
        for (int kb = k0; kb < k1; ++kb, acc.next()) {
            const int k = (kb - k0) & 3;
            if (k == 0) ok = ok && bar_wait_warp(bar_factors + 8 * turn.slot, turn.phase);
            ok = ok && bar_wait_warp(bar_acc + 8 * acc.slot, acc.phase);
            if (!ok) break;
            fence_after();
            const uint32_t f = factors + ((turn.slot * 4 + k) * kN + group * S::kMine) * 4;
            uint32_t r[S::kMine];
            tmem_load(tmem + acc.slot * kN + lanes + group * S::kMine, r);
            tmem_wait(r);
            fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(bar_free + 8 * acc.slot);
#pragma unroll
            for (int j = 0; j < S::kMine; j += 4) {
                float4 s;
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(s.x), "=f"(s.y), "=f"(s.z), "=f"(s.w) : "r"(f + j * 4));
                sums[j] = __fmaf_rn(__uint_as_float(r[j]), s.x, sums[j]);
                sums[j + 1] = __fmaf_rn(__uint_as_float(r[j + 1]), s.y, sums[j + 1]);
                sums[j + 2] = __fmaf_rn(__uint_as_float(r[j + 2]), s.z, sums[j + 2]);
                sums[j + 3] = __fmaf_rn(__uint_as_float(r[j + 3]), s.w, sums[j + 3]);
            }
            if (k == 3 || kb + 1 == k1) {
                __syncwarp();
                if (lane == 0) bar_arrive(bar_read + 8 * turn.slot);
                turn.next();
            }
        }
    }
    if (!ok) {
        atomicAdd(&g_timeouts, 1u);
        *failed = 1;
    }
    const Out& o = a.o;
    const int64_t col = (int64_t)n * 128 + out;
    const float bias = warp >= 4 && o.bias && col < o.N ? __ldg(o.bias + col) : 0.0f;
    // row `j` of the CTA's; neighbouring lanes are neighbouring columns
    auto store = [&](int j, float z) {
        const int64_t row = token0 + j;
        if (row >= o.T || col >= o.N) return;
        z += bias;
        if (o.pre) o.pre[row * o.N + col] = z;
        float v = activate(z, o.act);
        if (o.residual) v += to_float(o.residual[row * o.ld_r + col]);
        if (o.f32)
            static_cast<float*>(o.y)[row * o.ld_y + col] = v;
        else
            static_cast<bf16*>(o.y)[row * o.ld_y + col] = __float2bfloat16_rn(v);
    };
    __syncwarp();
    if (a.splits > 1) {
        // every stage has been read: the last sums came after the last product
        if (warp >= 4)
#pragma unroll
            for (int j = 0; j < S::kMine; ++j) sums_at[(group * S::kMine + j) * 128 + out] = sums[j];
        cluster.sync();
        if (warp >= 4) {
            bool whole = true;
            for (int q = 0; q < a.splits; ++q) whole &= *cluster.map_shared_rank(failed, q) == 0;
            const int rows = (int)min((int64_t)kN, o.T - token0);
            for (int j = split + group * a.splits; j < rows; j += S::kGroups * a.splits) {
                float z = 0.0f;
#pragma unroll 4
                for (int q = 0; q < a.splits; ++q) z += cluster.map_shared_rank(sums_at, q)[j * 128 + out];
                store(j, whole ? z : NAN);
            }
        }
        cluster.sync();  // no CTA leaves before its sums are read
    } else {
        __syncthreads();  // `failed` is set
        if (warp >= 4) {
            const bool whole = *failed == 0;
#pragma unroll
            for (int j = 0; j < S::kMine; ++j) store(group * S::kMine + j, whole ? sums[j] : NAN);
        }
    }
    fence_before();
    __syncthreads();
    __syncwarp();
    fence_after();
    if (warp == 2) tmem_free<1, S::kTmem>(tmem);
}

// ---- launches -----------------------------------------------------------------------------------

// Tiles of `box_rows` rows x 128 bytes of row-major bytes.
int map_bytes(CUtensorMap* map, const uint8_t* p, int64_t rows, int64_t cols, int64_t pitch, int box_rows)
{
    const uint64_t dims[2] = {(uint64_t)cols, (uint64_t)rows}, stride[1] = {(uint64_t)pitch};
    const uint32_t box[2] = {128, (uint32_t)box_rows};
    return ffn::tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p, dims, stride, box);
}

int maps(CUtensorMap* hi, CUtensorMap* lo, CUtensorMap* wm, const Rows& x, const Weight& w, int64_t K, int box_rows)
{
    // bytes of a row behind its K (a pair's padding is zeros, of 8-bit rows the map ends there)
    const int64_t cols = x.lo ? x.pitch : K;
    int st = map_bytes(hi, x.hi, x.T, cols, x.pitch, box_rows);
    if (st != FP8Z1_OK) return st;
    if ((st = map_bytes(lo, x.lo ? x.lo : x.hi, x.T, cols, x.pitch, box_rows)) != FP8Z1_OK) return st;
    return map_bytes(wm, w.codes, w.R, w.C, w.C, 128);
}

template <int kTerms, bool kKMajor>
int launch_many(const Rows& x, const Weight& w, Args a, cudaStream_t s)
{
    CUtensorMap hi, lo, wm;
    const int st = maps(&hi, &lo, &wm, x, w, w.K(), 128);
    if (st != FP8Z1_OK) return st;
    a.m_tiles = (int32_t)ceil_div(x.T, 256);
    a.n_tiles = (int32_t)ceil_div(a.o.N, kCols);
    for (int t = 0; t < 2; ++t)
        a.idesc[t] = instruction_of(256, kCols, false, !kKMajor, t && x.lo_format == Lo::kE5M2, 0);
    const int64_t tiles = (int64_t)a.m_tiles * a.n_tiles;
    return is_whole(a.o) ? ffn::launch_persistent<many_kernel<kTerms, kKMajor, true>, 2>(kManyThreads, Many<kTerms>::kSmem, tiles, s, hi, lo, wm, a)
                         : ffn::launch_persistent<many_kernel<kTerms, kKMajor, false>, 2>(kManyThreads, Many<kTerms>::kSmem, tiles, s, hi, lo, wm, a);
}

// CTAs along K: as few rounds of K steps as the SMs' CTAs need, a CTA's start and end worth 4 of them.
int splits_of(int64_t groups, int64_t slots, int64_t k_blocks)
{
    int best = 1;
    int64_t least = INT64_MAX;
    for (int n = 1; n <= 8 && n <= k_blocks; n *= 2) {
        const int64_t t = ceil_div(groups * n, slots) * (ceil_div(k_blocks, n) + 4);
        if (t < least) least = t, best = n;
    }
    return best;
}

template <int kTerms, int kN, bool kKMajor>
int launch_few(const Rows& x, const Weight& w, Args a, cudaStream_t s)
{
    using S = Few<kTerms, kN>;
    CUtensorMap hi, lo, wm;
    const int st = maps(&hi, &lo, &wm, x, w, w.K(), kN);
    if (st != FP8Z1_OK) return st;
    a.n_tiles = (int32_t)ceil_div(a.o.N, 128);
    a.m_tiles = (int32_t)ceil_div(x.T, kN);
    a.splits = splits_of((int64_t)a.n_tiles * a.m_tiles, (int64_t)kSms * S::kResident, a.k_blocks);
    for (int t = 0; t < 2; ++t)
        a.idesc[t] = instruction_of(128, kN, !kKMajor, false, 0, t && x.lo_format == Lo::kE5M2);
    if (!allow_smem<few_kernel<kTerms, kN, kKMajor>>((int)S::kSmem)) return FP8Z1_ECUDA;
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)a.splits;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    c.gridDim = dim3((unsigned)((int64_t)a.n_tiles * a.splits * a.m_tiles));
    c.blockDim = dim3(S::kThreads);
    c.dynamicSmemBytes = S::kSmem;
    c.stream = s;
    c.attrs = at;
    c.numAttrs = x.lo ? 2 : 1;  // 8-bit rows are the caller's: no kernel of this call goes ahead
    count_launch();
    if (cudaLaunchKernelEx(&c, few_kernel<kTerms, kN, kKMajor>, hi, lo, wm, a) != cudaSuccess) {
        cudaGetLastError();
        return FP8Z1_ECUDA;
    }
    return launch_status();
}

// Whether CTAs of 128 columns by 128 rows take less time than pairs with 256 x 256.  A step of K takes both about
// as long, so the rounds of the SMs decide; a round's start and end are worth 4 steps.  Measured, us of few and many, BF16
// rows and 8-bit ones: 512 rows of 7168 x 4096 42 and 40, 30 and 32; 256 29 and 39, 22 and 31; 1001 82 and 44, 58 and 32; 200 of
// 4096 x 14336 59 and 28, 50 and 22; 1001 of 4096 x 1024 23 and 27, 17 and 19, 2051 32 and 30, 21 and 20; 4096 of 1024 x 512
// 16 and 15, 12 and 9.
bool few_tiles(int64_t T, int64_t N, int64_t k_blocks)
{
    const int64_t tiles = ceil_div(T, 128) * ceil_div(N, 128);
    const int n = splits_of(tiles, kSms, k_blocks);
    return ceil_div(tiles * n, kSms) * (ceil_div(k_blocks, n) + 4) <
           ceil_div(ceil_div(T, 256) * ceil_div(N, 256), kSms / 2) * (k_blocks + 4);
}

template <int kTerms, bool kKMajor>
int launch(const Rows& x, const Weight& w, const Args& a, cudaStream_t s)
{
    if (x.T <= 16) return launch_few<kTerms, 16, kKMajor>(x, w, a, s);
    if (x.T <= 32) return launch_few<kTerms, 32, kKMajor>(x, w, a, s);
    if (x.T <= 64) return launch_few<kTerms, 64, kKMajor>(x, w, a, s);
#if FP8Z1_CHECKED
    if (g_all_few.load(std::memory_order_relaxed)) return launch_few<kTerms, 128, kKMajor>(x, w, a, s);
#endif
    if (x.T <= 128 || few_tiles(x.T, a.o.N, a.k_blocks)) return launch_few<kTerms, 128, kKMajor>(x, w, a, s);
    return launch_many<kTerms, kKMajor>(x, w, a, s);
}

}  // namespace

int launch_product(const Rows& x, const Weight& w, const Out& o, cudaStream_t s)
{
    Args a = {};
    a.o = o;
    a.a_scale = x.scale;
    a.scale_row = x.scale_row;
    a.scale_block = x.scale_block;
    a.b_scale = w.scale;
    const int32_t sc = (int32_t)ceil_div(w.C, 128);
    a.b_col = w.k_major ? sc : 1;
    a.b_step = w.k_major ? 1 : sc;
    a.b_cols = (int32_t)ceil_div(o.N, 128);
    a.k_blocks = (int32_t)ceil_div(w.K(), kBlock);
    a.splits = 1;
    if (x.lo) return w.k_major ? launch<2, true>(x, w, a, s) : launch<2, false>(x, w, a, s);
    return w.k_major ? launch<1, true>(x, w, a, s) : launch<1, false>(x, w, a, s);
}

int read_timeouts_product(unsigned* n)
{
    return cudaMemcpyFromSymbol(n, g_timeouts, 4) == cudaSuccess ? FP8Z1_OK : FP8Z1_ECUDA;
}

#if FP8Z1_CHECKED
int stall_product(unsigned kernels)
{
    g_all_few.store(kernels >> 4 & 1, std::memory_order_relaxed);
    kernels &= 3;
    return cudaMemcpyToSymbol(g_stall, &kernels, 4) == cudaSuccess ? FP8Z1_OK : FP8Z1_ECUDA;
}
#endif

}  // namespace linear
}  // namespace fp8z1
