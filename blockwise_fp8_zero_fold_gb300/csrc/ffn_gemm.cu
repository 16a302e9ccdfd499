// The four products of token rows with FP8 weights:
//
//   gate_up  g | u = x [Wg | Wu], then h = silu(g) u, encoded for the next product
//   down     y = h Wd
//   dh       dh = dy Wd^T
//   dx       dx = [dg | du] [Wg | Wu]^T
//
// A row operand a is a pair of FP8 numbers at a power of two per (row, 128 of
// k): a = 2^s (hi + lo), which carries x's and dy's 8 bits exactly and 9 of h's, dg's
// and du's, so the FP8 codes of a weight enter the tensor cores as they are:
//
//   sum_k a_k w_k c_kn = sum over blocks b of  2^s_b c_bn  sum_{k in b} (hi + lo)_k w_kn.
//
// Two FP8 products cost what one BF16 product does, and no weight is
// converted.  The inner sums are exact products accumulated in FP32 in tensor
// memory, 128 of k at a time; epilogue warps scale each and add it to the
// tile's sums in registers (FP32) while the next 128 are multiplied.
//
// A CTA owns 128 rows x 256 columns.  Warp 0 issues TMA copies of K steps (64
// KB: the rows' hi and lo, 256 weight columns) three steps ahead, warp 1 the
// products into one of two 256-column accumulators, 16 warps add up.  (Pairs of
// CTAs with 256 rows lost a quarter on experts of 100 to 400 rows; transposed
// products of 128 columns, whose time follows an expert's rows, lost half.)
//
// CTAs are persistent; tiles run expert by expert, a column's row tiles next
// to each other, so that an expert's codes are read from memory once.
//
// Bound by the tensor cores from some 100 rows an expert: 8192 tokens over 31
// experts of 7168 x 2048 take 0.42 ms (gate_up), 0.22 (down), 0.22 (dh) and 0.38
// (dx), 1170 TFLOP/s of BF16 products, 1520 with the padded rows; 2051 of 4096 x 14336
// 0.35, 0.16, 0.17 and 0.31, 1460.  A tile's end (SiLU, encoding, stores) is hidden by no
// more than the two accumulators: forward passes without it took 6 and 8 % less; without
// reading the sums of every 128 of k out of tensor memory they took the same.  With few
// rows bound by the codes read: 61 tokens over 27 experts, 1.19 GB in 260 us, 432 column
// tiles in three rounds of 152 CTAs.
#include "ffn.cuh"

namespace fp8z1 {
namespace ffn {
namespace {

using namespace tc;

__device__ unsigned g_timeouts;
#if FP8Z1_CHECKED
__device__ unsigned g_stall;  // bit kMode: that kernel's first CTA does not announce its first sums
#endif

// kPart: gate_up or down with K split over several CTAs, FP32 partial sums
enum Mode { kGateUp, kDown, kDh, kDx, kPart };
__host__ __device__ constexpr bool n_major(int mode) { return mode == kGateUp || mode == kDown || mode == kPart; }

constexpr int kCols = 256;   // columns of a tile, in two chunks of 128
constexpr int kStages = 3;
constexpr int kThreads = 640;  // 4 warps that feed, 16 that add up
constexpr uint32_t kOperand = 128 * 128;          // bytes of a 128 x 128 operand tile
constexpr uint32_t kStageBytes = 4 * kOperand;    // hi, lo, two chunks of the weight
constexpr int kStagePitch = 48;                     // of a row's 32 bytes on their way out
// stages, barriers, exchange, factors, rows on their way out
constexpr uint32_t kSmem = kStages * kStageBytes + 1024 + 256 + 4096 + 4096 + 16 * 32 * kStagePitch;

struct Args {
    Plan plan;
    const float* a_scale;  // [K / 128, rows]
    const float* b_scale;  // [E, ceil(R / 128), ceil(C / 128)]
    int64_t rows;          // of the row operands (pitch of a_scale)
    int64_t F;
    int64_t N;             // columns of the result (kGateUp: F pairs)
    uint32_t idesc[2];     // of the products with hi, with lo
    int32_t n_tiles;       // column tiles
    int32_t splits;        // kPart: CTAs along K, else 1
    int32_t k_blocks;
    int32_t sr, sc;        // the scale grid of an expert
    int32_t b_step;        // from one K block's scale to the next
    Pairs h;               // kGateUp
    float* gu;             // kGateUp (NULL: not kept), [tile][2F][128]
    float* dh;             // kDh, [tile][F][128]
    bf16* out;             // kDown, kDx
    int64_t ld;
    float* part;           // kPart, [splits, rows, N]
};

struct Work {
    int32_t tile, expert, token0, rows, n;
    int32_t split, k0, k1;  // K blocks
};

// The i-th tile of the launch, expert by expert, column by column.
__device__ __forceinline__ Work work_at(const Args& a, int64_t i)
{
    const int32_t per = a.n_tiles * a.splits, t = (int32_t)(i / per);
    const int32_t e = a.plan.tiles[t].expert;
    const int32_t first = a.plan.start[e], count = a.plan.start[e + 1] - first;
    const int64_t local = i - (int64_t)first * per;
    Work w;
    const int32_t column = (int32_t)(local / count);
    w.n = column / a.splits;
    w.split = column - w.n * a.splits;
    w.k0 = (int32_t)((int64_t)a.k_blocks * w.split / a.splits);
    w.k1 = (int32_t)((int64_t)a.k_blocks * (w.split + 1) / a.splits);
    w.tile = first + (int32_t)(local - (int64_t)column * count);
    const Tile tile = a.plan.tiles[w.tile];
    w.expert = e;
    w.token0 = tile.token0;
    w.rows = tile.rows;
    return w;
}

template <int kMode>
__device__ __forceinline__ int chunk_column(const Args& a, const Work& w, int c)
{
    return kMode == kGateUp ? (int)(c * a.F) + w.n * 128 : w.n * kCols + c * 128;
}

// The scales of weight column chunk c, K block by K block b_step apart (a chunk
// past the columns: any of the expert's, its sums are not stored).
template <int kMode>
__device__ __forceinline__ const float* b_scale(const Args& a, const Work& w, int c)
{
    const int n = chunk_column<kMode>(a, w, c) >> 7;
    const float* s = a.b_scale + (int64_t)w.expert * a.sr * a.sc;
    if (n_major(kMode)) return s + min(n, a.sc - 1);
    return s + (int64_t)min(n, a.sr - 1) * a.sc;
}
// 32 bytes of each of a warp's 32 rows, a lane's own in v[2], through shared memory:
// two lanes store a row's, so that a sector is written whole and an instruction
// touches 16 lines, not 32.
__device__ __forceinline__ void store_rows(uint8_t* stage, int lane, const uint4 (&v)[2], uint8_t* to, int64_t pitch,
                                           int rows)
{
    *reinterpret_cast<uint4*>(stage + lane * kStagePitch) = v[0];
    *reinterpret_cast<uint4*>(stage + lane * kStagePitch + 16) = v[1];
    __syncwarp();
#pragma unroll
    for (int r = lane >> 1; r < 32; r += 16)
        if (r < rows)
            *reinterpret_cast<uint4*>(to + r * pitch + (lane & 1) * 16) =
                *reinterpret_cast<const uint4*>(stage + r * kStagePitch + (lane & 1) * 16);
    __syncwarp();
}

// g / (1 + exp(-g)) by t = exp(-|g|) <= 1: nothing overflows, and no branch (the
// branch's code, 32 times a row, cost a small product 10 us of instruction fetches)
__device__ __forceinline__ float silu(float g)
{
    const float t = __expf(-fabsf(g));
    return g * __fdividef(g < 0.0f ? t : 1.0f, 1.0f + t);
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

template <int kMode>
__global__ void __launch_bounds__(kThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap map_hi, const __grid_constant__ CUtensorMap map_lo,
            const __grid_constant__ CUtensorMap map_w, const __grid_constant__ Args a)
{
    extern __shared__ uint8_t smem_raw[];
    next_may_start();
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    const uint32_t extra = base + kStages * kStageBytes;
    // extra: full[3], empty[3], accumulators ready[2], free[2], tensor memory base, exchange, factors ready[4],
    // read[4]; the amax exchange [2][4][128]; the factors [4][2][128]
    const uint32_t bar_full = extra, bar_empty = extra + 32, bar_acc = extra + 64, bar_free = extra + 96,
                   bar_exchange = extra + 136, bar_factors = extra + 144, bar_read = extra + 176,
                   factors = extra + 256 + 4096;
    uint8_t* extra_ptr = smem_raw + (extra - smem_addr(smem_raw));
    volatile uint32_t* tmem_at = reinterpret_cast<uint32_t*>(extra_ptr + 128);
    float* exchange = reinterpret_cast<float*>(extra_ptr + 256);  // [2][4][128]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            bar_init(bar_full + 8 * i, 1);
            bar_init(bar_empty + 8 * i, 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(bar_acc + 8 * i, 1);
            bar_init(bar_free + 8 * i, 16);  // the adding warps
        }
        bar_init(bar_exchange, 512);
        for (int i = 0; i < 4; ++i) {
            bar_init(bar_factors + 8 * i, 64);
            bar_init(bar_read + 8 * i, 16);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
        prefetch_map(&map_hi);
        prefetch_map(&map_lo);
        prefetch_map(&map_w);
    }
    if (warp == 2) tmem_alloc<1, 512>(extra + 128);
    fence_before();
    __syncthreads();
    __syncwarp();
    fence_after();
    after_previous();
    const uint32_t tmem = *tmem_at;
    const int64_t total = (int64_t)*a.plan.n_tiles * a.n_tiles * a.splits, i0 = blockIdx.x, step = gridDim.x;
    bool ok = true;

    if (warp < 4) {
        regs_less<48>();
        if (warp == 0 && lane == 0) {
            // TMA: K steps of every tile, kStages ahead
            Turn<kStages> turn;
            for (int64_t i = i0; i < total && ok; i += step) {
                const Work w = work_at(a, i);
                const int c0 = chunk_column<kMode>(a, w, 0), c1 = chunk_column<kMode>(a, w, 1), y = w.tile * kRows;
                for (int kb = w.k0; kb < w.k1; ++kb, turn.next()) {
                    if (!bar_wait(bar_empty + 8 * turn.slot, turn.phase ^ 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t full = bar_full + 8 * turn.slot, dst = base + turn.slot * kStageBytes;
                    bar_expect(full, kStageBytes);
                    load_2d(dst, &map_hi, full, kb * 128, y);
                    load_2d(dst + kOperand, &map_lo, full, kb * 128, y);
                    if (n_major(kMode)) {
                        load_3d(dst + 2 * kOperand, &map_w, full, c0, kb * 128, w.expert);
                        load_3d(dst + 3 * kOperand, &map_w, full, c1, kb * 128, w.expert);
                    } else {
                        load_3d(dst + 2 * kOperand, &map_w, full, kb * 128, c0, w.expert);
                        load_3d(dst + 3 * kOperand, &map_w, full, kb * 128, c1, w.expert);
                    }
                }
            }
            // the copies in flight are read before the CTA ends, whatever became of the other warps
            for (int j = 0; j < kStages; ++j, turn.next()) ok &= bar_wait(bar_empty + 8 * turn.slot, turn.phase ^ 1);
        } else if (warp == 1 && lane == 0) {
            constexpr bool kMnMajor = n_major(kMode);
            Turn<kStages> turn;
            Turn<2> acc;
            for (int64_t i = i0; i < total && ok; i += step) {
                const Work w = work_at(a, i);
                for (int kb = w.k0; kb < w.k1; ++kb, turn.next(), acc.next()) {
                    if (!bar_wait(bar_free + 8 * acc.slot, acc.phase ^ 1) ||
                        !bar_wait(bar_full + 8 * turn.slot, turn.phase)) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint32_t src = base + turn.slot * kStageBytes, d = tmem + acc.slot * kCols;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint64_t da = operand(src + t * kOperand + k * 32, 1024, 16);
                            // N-major: 8 k are 1024 bytes, the second chunk of 128 columns follows the first;
                            // K-major: 8 columns are 1024 bytes
                            const uint64_t db = kMnMajor ? operand(src + 2 * kOperand + k * 4096, 1024, kOperand)
                                                         : operand(src + 2 * kOperand + k * 32, 1024, 16);
                            mma_f8(d, da, db, a.idesc[t], t + k > 0);
                        }
                    commit(bar_empty + 8 * turn.slot);
#if FP8Z1_CHECKED
                    if (g_stall >> kMode & 1 && blockIdx.x == 0 && i == i0 && kb == w.k0) continue;
#endif
                    commit(bar_acc + 8 * acc.slot);
                }
            }
            // every product issued ends, and its sums are read, before the tensor memory is freed
            for (int j = 0; j < 2; ++j, acc.next()) ok = bar_wait(bar_free + 8 * acc.slot, acc.phase ^ 1) && ok;
        } else if (warp >= 2) {
            // the factors of each step, 2^s_b c_bn of both chunks for two rows a thread
            Turn<4> turn;
            const int mine = threadIdx.x - 64;
            for (int64_t i = i0; i < total && ok; i += step) {
                const Work w = work_at(a, i);
                const float* pa = a.a_scale + (int64_t)w.tile * kRows + mine;
                const float *p0 = b_scale<kMode>(a, w, 0), *p1 = b_scale<kMode>(a, w, 1);
                for (int kb = w.k0; kb < w.k1; ++kb, turn.next()) {
                    const float va = pa[(int64_t)kb * a.rows], vb = pa[(int64_t)kb * a.rows + 64], v0 = p0[kb * a.b_step],
                                v1 = p1[kb * a.b_step];
                    if (!bar_wait(bar_read + 8 * turn.slot, turn.phase ^ 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t f = factors + turn.slot * 1024 + mine * 4;
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(f), "f"(va * v0) : "memory");
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(f + 256), "f"(vb * v0) : "memory");
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(f + 512), "f"(va * v1) : "memory");
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(f + 768), "f"(vb * v1) : "memory");
                    bar_arrive(bar_factors + 8 * turn.slot);
                }
            }
        }
    } else {
        regs_more<104>();
        const int group = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16;
        uint8_t* stage = extra_ptr + 256 + 4096 + 4096 + (warp - 4) * 32 * kStagePitch;
        Turn<2> acc;
        Turn<4> turn;
        int parity = 0;
        bool together = true;  // kGateUp: with the other warps of the row
        for (int64_t i = i0; i < total; i += step) {
            const Work w = work_at(a, i);
            const int64_t at = (int64_t)w.tile * kRows + row;  // row of the internal buffers
            uint64_t sums2[2][16];  // pairs of columns
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < 16; ++j) sums2[c][j] = 0;
            for (int kb = w.k0; kb < w.k1; ++kb, acc.next(), turn.next()) {
                // a warp's lanes agree on the outcome: the loads below are warp-wide
                ok = ok && __all_sync(0xffffffffu, bar_wait(bar_factors + 8 * turn.slot, turn.phase) &&
                                                       bar_wait(bar_acc + 8 * acc.slot, acc.phase));
                if (!ok) break;
                fence_after();
                float f0, f1;
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f0) : "r"(factors + turn.slot * 1024 + row * 4));
                asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f1) : "r"(factors + turn.slot * 1024 + 512 + row * 4));
                const uint64_t f[2] = {pair(f0, f0), pair(f1, f1)};
                const uint32_t t = tmem + acc.slot * kCols + lanes + group * 32;
                // columns 32 group + {0, 16, 128, 144} ..
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t r[16];
                    tmem_load(t + q / 2 * 128 + q % 2 * 16, r);
                    tmem_wait(r);
                    if (q == 3) {
                        fence_before();
                        __syncwarp();
                        if (lane == 0) {
                            bar_arrive(bar_free + 8 * acc.slot);
                            bar_arrive(bar_read + 8 * turn.slot);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        sums2[q / 2][q % 2 * 8 + j] =
                            fma_pair(pair(r[2 * j], r[2 * j + 1]), f[q / 2], sums2[q / 2][q % 2 * 8 + j]);
                }
            }
            // a wait ran out: this tile and the CTA's further ones are NaN, which reaches all that is made of them
            if (!ok)
#pragma unroll
                for (int j = 0; j < 32; ++j) sums2[j / 16][j % 16] = pair(NAN, NAN);
            float sum[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float2 v = unpair(sums2[c][j]);
                    sum[c][2 * j] = v.x;
                    sum[c][2 * j + 1] = v.y;
                }
            if constexpr (kMode == kGateUp) {
                const int n0 = w.n * 128 + group * 32;
                float amax = 0.0f;
                if (a.gu) {
                    float* g = a.gu + ((int64_t)w.tile * 2 * a.F + n0) * kRows + row;
                    float* u = g + a.F * kRows;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        __stcs(g + j * kRows, sum[0][j]);
                        __stcs(u + j * kRows, sum[1][j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    sum[0][j] = silu(sum[0][j]) * sum[1][j];
                    amax = fmaxf(amax, fabsf(sum[0][j]));
                }
                // the largest of the row's 128 columns, 32 each of the four groups
                if (together) {
                    exchange[(parity * 4 + group) * 128 + row] = amax;
                    bar_arrive(bar_exchange);
                    together = __all_sync(0xffffffffu, bar_wait(bar_exchange, parity));
                }
                if (together) {
#pragma unroll
                    for (int o = 0; o < 4; ++o) amax = fmaxf(amax, exchange[(parity * 4 + o) * 128 + row]);
                    parity ^= 1;
                } else {
                    ok = false;
                    amax = INFINITY;  // the row's 128 numbers become NaN
                }
                const PairScale ps = pair_scale(amax);
                if (group == 0) a.h.scale[(int64_t)w.n * a.rows + at] = ps.down;
                uint4 hi[2], lo[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t vh[4], vl[4];
#pragma unroll
                    for (int i2 = 0; i2 < 4; ++i2) {
                        const float* v = &sum[0][q * 16 + i2 * 4];
                        uint32_t h0, l0, h1, l1;
                        pair_encode<Lo::kE4M3>(v[0], v[1], ps.up, h0, l0);
                        pair_encode<Lo::kE4M3>(v[2], v[3], ps.up, h1, l1);
                        vh[i2] = h0 | h1 << 16;
                        vl[i2] = l0 | l1 << 16;
                    }
                    hi[q] = make_uint4(vh[0], vh[1], vh[2], vh[3]);
                    lo[q] = make_uint4(vl[0], vl[1], vl[2], vl[3]);
                }
                const int64_t first = (at - lane) * a.h.pitch + n0;
                store_rows(stage, lane, hi, a.h.hi + first, a.h.pitch, 32);
                store_rows(stage, lane, lo, a.h.lo + first, a.h.pitch, 32);
            } else if constexpr (kMode == kPart) {
                if (row < w.rows)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int64_t n0 = (int64_t)w.n * kCols + c * 128 + group * 32;
                        float* o = a.part + ((int64_t)w.split * a.rows + at) * a.N + n0;
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            if (n0 + q * 4 >= a.N) break;
                            *reinterpret_cast<float4*>(o + q * 4) =
                                make_float4(sum[c][q * 4], sum[c][q * 4 + 1], sum[c][q * 4 + 2], sum[c][q * 4 + 3]);
                        }
                    }
            } else if constexpr (kMode == kDh) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int64_t n0 = (int64_t)w.n * kCols + c * 128 + group * 32;
                    if (n0 >= a.N) continue;  // F is a multiple of 128: a chunk is in or out whole
                    float* o = a.dh + ((int64_t)w.tile * a.F + n0) * kRows + row;
#pragma unroll
                    for (int j = 0; j < 32; ++j) __stcs(o + j * kRows, sum[c][j]);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const int64_t n0 = (int64_t)w.n * kCols + c * 128 + group * 32 + q * 16;
                        if (n0 >= a.N) break;  // N is a multiple of 16
                        uint32_t v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const __nv_bfloat162 two =
                                __floats2bfloat162_rn(sum[c][q * 16 + 2 * j], sum[c][q * 16 + 2 * j + 1]);
                            v[j] = *reinterpret_cast<const uint32_t*>(&two);
                        }
                        const uint4 out[2] = {make_uint4(v[0], v[1], v[2], v[3]), make_uint4(v[4], v[5], v[6], v[7])};
                        store_rows(stage, lane, out,
                                   reinterpret_cast<uint8_t*>(a.out + (int64_t)(w.token0 + row - lane) * a.ld + n0),
                                   a.ld * 2, w.rows - (row - lane));
                    }
                }
            }
        }
    }
    if (!ok) atomicAdd(&g_timeouts, 1u);
    fence_before();
    __syncthreads();
    __syncwarp();
    fence_after();
    if (warp == 2) tmem_free<1, 512>(tmem);
}

// y of the partial sums, in the order of the splits.
__global__ void __launch_bounds__(256) join_kernel(Plan plan, const float* part, int64_t rows, int64_t N, int splits,
                                                   bf16* out, int64_t ld)
{
    next_may_start();
    after_previous();
    if (blockIdx.x / kRows >= *plan.n_tiles) return;
    const Tile t = plan.tiles[blockIdx.x / kRows];
    const int r = blockIdx.x % kRows;
    const int64_t n = (int64_t)(blockIdx.y * 256 + threadIdx.x) * 4;
    if (r >= t.rows || n >= N) return;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int k = 0; k < splits; ++k) {
        const float4 v = *reinterpret_cast<const float4*>(part + ((int64_t)k * rows + blockIdx.x) * N + n);
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(out + (int64_t)(t.token0 + r) * ld + n);
    o[0] = __floats2bfloat162_rn(s.x, s.y);
    o[1] = __floats2bfloat162_rn(s.z, s.w);
}

// h of the partial sums of gate and up, as pairs (a warp 128 columns of a row), and
// what the gate_up product's own epilogue keeps.
__global__ void __launch_bounds__(256) join_gate_kernel(Plan plan, const float* part, int64_t rows, int64_t F, int splits,
                                                        Pairs h, float* gu)
{
    next_may_start();
    after_previous();
    if (blockIdx.x / kRows >= *plan.n_tiles) return;
    const Tile t = plan.tiles[blockIdx.x / kRows];
    const int r = blockIdx.x % kRows, lane = threadIdx.x & 31;
    const int64_t block = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5), n = block * 128 + lane * 4;
    if (r >= t.rows || n >= F) return;
    float4 g = make_float4(0.0f, 0.0f, 0.0f, 0.0f), u = g;
#pragma unroll 4
    for (int k = 0; k < splits; ++k) {
        const float* p = part + ((int64_t)k * rows + blockIdx.x) * 2 * F + n;
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + F);
        g.x += a.x, g.y += a.y, g.z += a.z, g.w += a.w;
        u.x += b.x, u.y += b.y, u.z += b.z, u.w += b.w;
    }
    const float gs[4] = {g.x, g.y, g.z, g.w}, us[4] = {u.x, u.y, u.z, u.w};
    float v[4], amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = silu(gs[j]) * us[j];
        amax = fmaxf(amax, fabsf(v[j]));
        if (gu) {
            float* o = gu + ((int64_t)(blockIdx.x / kRows) * 2 * F + n + j) * kRows + r;
            o[0] = gs[j];
            o[F * kRows] = us[j];
        }
    }
    const PairScale ps = pair_scale(__uint_as_float(__reduce_max_sync(0xffffffffu, abs_bits(amax))));
    uint32_t h0, l0, h1, l1;
    pair_encode<Lo::kE4M3>(v[0], v[1], ps.up, h0, l0);
    pair_encode<Lo::kE4M3>(v[2], v[3], ps.up, h1, l1);
    *reinterpret_cast<uint32_t*>(h.hi + (int64_t)blockIdx.x * h.pitch + n) = h0 | h1 << 16;
    *reinterpret_cast<uint32_t*>(h.lo + (int64_t)blockIdx.x * h.pitch + n) = l0 | l1 << 16;
    if (lane == 0) h.scale[block * rows + blockIdx.x] = ps.down;
}

template <int kMode>
int launch(const Dims& d, const Pairs& rows, Lo lo_format, int64_t K, const Weight& w, Args a, cudaStream_t s)
{
    CUtensorMap hi, lo, wm;
    const uint64_t rdims[2] = {(uint64_t)rows.pitch, (uint64_t)d.rows()}, rstride[1] = {(uint64_t)rows.pitch};
    const uint32_t rbox[2] = {128, 128};
    const uint64_t wdims[3] = {(uint64_t)w.C, (uint64_t)w.R, (uint64_t)d.E},
                   wstride[2] = {(uint64_t)w.C, (uint64_t)(w.C * w.R)};
    const uint32_t wbox[3] = {128, 128, 1};
    int st;
    if ((st = tensor_map(&hi, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, rows.hi, rdims, rstride, rbox)) != FP8Z1_OK ||
        (st = tensor_map(&lo, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, rows.lo, rdims, rstride, rbox)) != FP8Z1_OK ||
        (st = tensor_map(&wm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, w.codes, wdims, wstride, wbox)) != FP8Z1_OK)
        return st;
    for (int t = 0; t < 2; ++t) a.idesc[t] = instruction(128, kCols, false, n_major(kMode), t && lo_format == Lo::kE5M2);
    a.a_scale = rows.scale;
    a.b_scale = w.scale;
    a.rows = d.rows();
    a.F = d.F;
    a.n_tiles = (int32_t)(kMode == kGateUp ? d.F / 128 : ceil_div(a.N, kCols));
    if (kMode != kPart) a.splits = 1;
    a.k_blocks = (int32_t)ceil_div(K, kBlock);
    a.sr = (int32_t)ceil_div(w.R, 128);
    a.sc = (int32_t)ceil_div(w.C, 128);
    a.b_step = n_major(kMode) ? a.sc : 1;
    return launch_persistent<gemm_kernel<kMode>, 1>(kThreads, kSmem, d.tiles() * a.n_tiles * a.splits, s, hi, lo, wm, a);
}

}  // namespace

int launch_gate_up(const Dims& d, const Plan& p, const Pairs& x, const Weight& w, const Pairs& h, float* gu, float* part,
                   cudaStream_t s)
{
    Args a = {};
    a.plan = p;
    a.N = d.F;
    a.h = h;
    a.gu = gu;
    a.splits = k_splits(d, 2 * d.F, d.H);
    if (a.splits == 1) return launch<kGateUp>(d, x, Lo::kE5M2, d.H, w, a, s);
    a.N = 2 * d.F;
    a.part = part;
    const int st = launch<kPart>(d, x, Lo::kE5M2, d.H, w, a, s);
    if (st != FP8Z1_OK) return st;
    return launch_after(join_gate_kernel, dim3((unsigned)d.rows(), (unsigned)ceil_div(d.F, 1024)), 256, 0, s, p, part,
                        d.rows(), d.F, a.splits, h, gu);
}

int launch_down(const Dims& d, const Plan& p, const Pairs& h, const Weight& w, bf16* y, int64_t ld, float* part,
                cudaStream_t s)
{
    Args a = {};
    a.plan = p;
    a.N = d.H;
    a.out = y;
    a.ld = ld;
    a.splits = k_splits(d, d.H, d.F);
    if (a.splits == 1) return launch<kDown>(d, h, Lo::kE4M3, d.F, w, a, s);
    a.part = part;
    const int st = launch<kPart>(d, h, Lo::kE4M3, d.F, w, a, s);
    if (st != FP8Z1_OK) return st;
    return launch_after(join_kernel, dim3((unsigned)d.rows(), (unsigned)ceil_div(d.H, 1024)), 256, 0, s, p, part, d.rows(),
                        d.H, a.splits, y, ld);
}

int launch_dh(const Dims& d, const Plan& p, const Pairs& dy, const Weight& w, float* dh, cudaStream_t s)
{
    Args a = {};
    a.plan = p;
    a.N = d.F;
    a.dh = dh;
    return launch<kDh>(d, dy, Lo::kE5M2, d.H, w, a, s);
}

int launch_dx(const Dims& d, const Plan& p, const Pairs& dgu, const Weight& w, bf16* dx, int64_t ld, cudaStream_t s)
{
    Args a = {};
    a.plan = p;
    a.N = d.H;
    a.out = dx;
    a.ld = ld;
    return launch<kDx>(d, dgu, Lo::kE4M3, 2 * d.F, w, a, s);
}

int read_timeouts_gemm(unsigned* n)
{
    return cudaMemcpyFromSymbol(n, g_timeouts, 4) == cudaSuccess ? FP8Z1_OK : FP8Z1_ECUDA;
}

#if FP8Z1_CHECKED
int stall_gemm(unsigned kernels)
{
    return cudaMemcpyToSymbol(g_stall, &kernels, 4) == cudaSuccess ? FP8Z1_OK : FP8Z1_ECUDA;
}
#endif

}  // namespace ffn
}  // namespace fp8z1
