// The weight gradients: sums over an expert's token rows,
//
//   d_gate_up[h, c] = sum_t x[t, h] dgu[t, c]        d_down[f, h] = sum_t h[t, f] dy[t, h]
//
// in FP32 accuracy.  x and dy are BF16 values and fit FP16 exactly (8
// significant bits; every expert's operand is brought below 2^15 by one power
// of two, and FP16 holds such a number whole down to 2^-32 of the largest);
// dgu and h are FP32 and enter as two FP16 numbers, hi = f16(v), lo = f16(v -
// hi), 22 bits, every column of two tiles' 256 rows at its own power of two, so
// that a column of small numbers (a gate that is shut) keeps its bits beside
// large ones.  Two FP16 products with FP32 accumulators then cost twice one
// BF16 product and keep FP32's accuracy; one BF16 product would lose 16 bits
// of it, and the optimizer's grads are FP32.
//
// A pair of CTAs owns 256 x 256 of a gradient: each 128 columns of the two-term
// operand (the lanes of its tensor memory), and the other operand's 256 columns
// half and half.  Both operands are row-major over tokens, that is M- and
// N-major to the tensor cores.  The pipeline is ffn_gemm.cu's: TMA steps of 64
// token rows (48 KB a CTA), products into two accumulators, each two tiles' 256
// rows scaled and added up in registers.  The last step issues only the 16-row products that hold
// rows; rows past an expert's end are zeros.  A stage is 48 KB for 0.54 us of
// products, more than L2 delivers to every SM at once.
//
// Bound by the FP32 gradients written (4 bytes an element) up to about 250
// tokens an expert, by the tensor cores and what feeds them above: 8192 tokens over 31
// experts of 7168 x 2048 take 800 us (d_gate_up) and 400 (d_down), 4.7 TB/s of stores;
// 2051 of 4096 x 14336 640 and 295, 1550 TFLOP/s of FP16 products.
#include "ffn.cuh"

namespace fp8z1 {
namespace ffn {
namespace {

using namespace tc;

__device__ unsigned g_timeouts;
#if FP8Z1_CHECKED
__device__ unsigned g_stall;  // bit kTransposed: that kernel's first pair does not announce its first sums
#endif

constexpr int kCols = 256;
constexpr int kStep = 64;  // token rows of a stage
constexpr int kStages = 4;
// Stages added up in tensor memory before they go to the registers' sums: two tiles' rows,
// which share their columns' powers of two.  (Tensor memory's adds do not round to
// nearest: sums of 256 rows there leave 7e-7 of the gradient's norm, of 512 1.3e-6.  Powers
// of two and sums of 128 rows let the products run only 256 rows ahead of a tile's stores:
// 300 tokens of 4096 x 14336 then took 290 + 96 us.)
constexpr int kAdd = 2 * kRows / kStep;
constexpr int kThreads = 640;  // 4 warps that feed, 16 that add up
constexpr uint32_t kChunk = 64 * kStep * 2;     // bytes of 64 columns of a stage
constexpr uint32_t kStageBytes = 6 * kChunk;    // hi: 2 chunks, lo: 2, half of the other operand: 2
constexpr uint32_t kSmem = kStages * kStageBytes + 16 * 2048 + 1024 + 256;

struct Args {
    Plan plan;
    const uint32_t* peaks;  // of x or dy, a Peaks apart
    const float* factors;   // of the two-term operand's columns, [pairs of tiles][pitch]
    int64_t pitch;
    float* out;        // kTransposed: [E, N, M]
    int64_t M, N;      // columns of the two-term operand, of the other
    int32_t m_tiles, n_tiles, experts;
};

// kTransposed: the two-term operand's columns are the gradient's columns
// (d_gate_up), else its rows (d_down).
template <bool kTransposed>
__global__ void __launch_bounds__(kThreads, 1)
wgrad_kernel(const __grid_constant__ CUtensorMap map_hi, const __grid_constant__ CUtensorMap map_lo,
             const __grid_constant__ CUtensorMap map_b, const __grid_constant__ CUtensorMap map_out,
             const __grid_constant__ Args a)
{
    extern __shared__ uint8_t smem_raw[];
    next_may_start();
    const uint32_t base = (smem_addr(smem_raw) + 1023) & ~1023u;
    const uint32_t staging = base + kStages * kStageBytes, extra = staging + 16 * 2048;
    const uint32_t bar_full = extra, bar_empty = extra + 32, bar_acc = extra + 64, bar_free = extra + 80;
    volatile uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem_raw + (extra + 96 - smem_addr(smem_raw)));

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = (int)cluster_rank();  // of the pair
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
        prefetch_map(&map_lo);
        prefetch_map(&map_b);
    }
    if (warp == 2) tmem_alloc<2, 512>(extra + 96);
    fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();  // the other CTA counts on this one's barriers from here on
    fence_after();
    after_previous();
    const uint32_t tmem = *tmem_at;
    const int m_pairs = (a.m_tiles + 1) / 2;
    const int64_t per = (int64_t)m_pairs * a.n_tiles, total = per * a.experts;
    const int64_t i0 = blockIdx.x / 2, step = gridDim.x / 2;
    bool ok = true;

    if (warp < 4) {
        regs_less<48>();
        if (warp == 0 && lane == 0) {
            Turn<kStages> turn;
            for (int64_t i = i0; i < total && ok; i += step) {
                const int e = (int)(i / per), local = (int)(i - e * per);
                const int m = local % m_pairs * 2 + sub, n = local / m_pairs;
                const int row0 = a.plan.start[e] * kRows, steps = (a.plan.tokens[e] + kStep - 1) / kStep;
                for (int k = 0; k < steps; ++k, turn.next()) {
                    if (!bar_wait(bar_empty + 8 * turn.slot, turn.phase ^ 1)) {
                        ok = false;
                        break;
                    }
                    // both CTAs' copies are counted in the first one, whose thread multiplies
                    if (sub == 0) bar_expect(bar_full + 8 * turn.slot, 2 * kStageBytes);
                    const uint32_t full = first_of_pair(bar_full + 8 * turn.slot), dst = base + turn.slot * kStageBytes;
                    load_3d_pair(dst, &map_hi, full, 0, row0 + k * kStep, m * 2);
                    load_3d_pair(dst + 2 * kChunk, &map_lo, full, 0, row0 + k * kStep, m * 2);
                    load_3d_pair(dst + 4 * kChunk, &map_b, full, 0, row0 + k * kStep, n * 4 + sub * 2);
                }
            }
            // the copies in flight are read before the CTA ends, whatever became of the other warps
            for (int j = 0; j < kStages; ++j, turn.next()) ok &= bar_wait(bar_empty + 8 * turn.slot, turn.phase ^ 1);
        } else if (warp == 1 && lane == 0 && sub == 0) {
            constexpr uint32_t idesc = instruction(256, kCols, true, true);
            Turn<kStages> turn;
            Turn<2> acc;
            for (int64_t i = i0; i < total && ok; i += step) {
                const int tokens = a.plan.tokens[(int)(i / per)];
                for (int t0 = 0; t0 < tokens && ok; t0 += kAdd * kStep, acc.next()) {
                    const uint32_t d = tmem + acc.slot * kCols;
                    ok = bar_wait(bar_free + 8 * acc.slot, acc.phase ^ 1);
                    for (int sub = 0; sub < kAdd && t0 + sub * kStep < tokens && ok; ++sub, turn.next()) {
                        if (!bar_wait(bar_full + 8 * turn.slot, turn.phase)) {
                            ok = false;
                            break;
                        }
                        fence_after();
                        const uint32_t src = base + turn.slot * kStageBytes;
                        const int left = tokens - t0 - sub * kStep, steps = left >= kStep ? 4 : (left + 15) / 16;
                        for (int k = 0; k < steps; ++k) {
                            // 8 rows are 1024 bytes; the next 64 columns follow a chunk later
                            const uint64_t db = operand(src + 4 * kChunk + k * 2048, 1024, kChunk);
                            mma_f16_pair(d, operand(src + k * 2048, 1024, kChunk), db, idesc, sub + k > 0);
                            mma_f16_pair(d, operand(src + 2 * kChunk + k * 2048, 1024, kChunk), db, idesc, true);
                        }
                        commit_pair(bar_empty + 8 * turn.slot);
                    }
#if FP8Z1_CHECKED
                    if (g_stall >> kTransposed & 1 && blockIdx.x == 0 && i == i0 && t0 == 0) continue;
#endif
                    if (ok) commit_pair(bar_acc + 8 * acc.slot);
                }
            }
            // every product issued ends, and its sums are read, before the tensor memory is freed
            for (int j = 0; j < 2; ++j, acc.next()) ok = bar_wait(bar_free + 8 * acc.slot, acc.phase ^ 1) && ok;
        }
    } else {
        regs_more<104>();
        const int group = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = (uint32_t)(warp & 3) * 32 << 16, mine = staging + (warp - 4) * 2048;
        Turn<2> acc;
        for (int64_t i = i0; i < total; i += step) {
            const int e = (int)(i / per), local = (int)(i - e * per);
            const int m = local % m_pairs * 2 + sub, n = local / m_pairs;
            const int tokens = a.plan.tokens[e];
            const float* factor = a.factors + a.plan.pair_start[e] * a.pitch + m * 128 + row;
            // plain loads: they stay ahead of the waits
            float next = tokens && m < a.m_tiles ? *factor : 0.0f;
            const uint32_t peak = a.peaks[e * (int)(sizeof(Peaks) / 4)];
            uint64_t sums2[2][16];  // pairs of columns
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < 16; ++j) sums2[c][j] = 0;
            for (int t0 = 0; t0 < tokens; t0 += kAdd * kStep, acc.next()) {
                ok = ok && __all_sync(0xffffffffu, bar_wait(bar_acc + 8 * acc.slot, acc.phase));
                if (!ok) break;
                fence_after();
                const uint64_t f = pair(next, next);
                if (t0 + kAdd * kStep < tokens && m < a.m_tiles) next = *(factor += a.pitch);
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
                            fma_pair(pair(r[2 * j], r[2 * j + 1]), f, sums2[q / 2][q % 2 * 8 + j]);
                }
            }
            // a wait ran out: this tile and the pair's further ones are NaN
            if (!ok)
#pragma unroll
                for (int j = 0; j < 32; ++j) sums2[j / 16][j % 16] = pair(NAN, NAN);
            if (m >= a.m_tiles) continue;  // an odd last tile's other half
            const float last = peak_factor(peak);
            float sum[2][32];
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float2 v = unpair(sums2[c][j]);
                    sum[c][2 * j] = v.x * last;
                    sum[c][2 * j + 1] = v.y * last;
                }
            if constexpr (kTransposed) {
                // lanes are consecutive columns of the gradient
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int64_t n0 = (int64_t)n * kCols + c * 128 + group * 32;
                    float* o = a.out + ((int64_t)e * a.N + n0) * a.M + m * 128 + row;
                    if (n0 + 32 <= a.N) {
#pragma unroll
                        for (int j = 0; j < 32; ++j, o += a.M) __stcs(o, sum[c][j]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j, o += a.M)
                            if (n0 + j < a.N) __stcs(o, sum[c][j]);
                    }
                }
            } else {
                // lanes are rows: pieces of 32 rows x 16 columns turn in shared memory and leave by TMA
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t buf = mine;
                    if (lane == 0) store_wait_read<0>();
                    __syncwarp();
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const float* x = &sum[q / 2][q % 2 * 16 + v * 4];
                        // 64-byte swizzle: 16-byte units of a row change places with bits 1-2 of the row
                        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                                         buf + lane * 64 + ((v ^ (lane >> 1 & 3)) << 4)),
                                     "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3])
                                     : "memory");
                    }
                    fence_async();
                    __syncwarp();
                    const int n0 = n * kCols + q / 2 * 128 + group * 32 + q % 2 * 16;
                    if (lane == 0) {
                        if (n0 < a.N) store_3d(&map_out, buf, n0, m * 128 + (warp & 3) * 32, e);
                        store_commit();
                    }
                }
            }
        }
        if (!kTransposed && lane == 0) store_wait_all();
    }
    if (!ok) atomicAdd(&g_timeouts, 1u);
    fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync();  // no CTA leaves while the other may still write to it
    fence_after();
    if (warp == 2) tmem_free<2, 512>(tmem);
}

// [rows, pitch] FP16 as {64, rows, pitch / 64}, fetched 128 columns at a time
int map_f16(CUtensorMap* map, const __half* p, int64_t rows, int64_t pitch)
{
    const uint64_t dims[3] = {64, (uint64_t)rows, (uint64_t)(pitch / 64)}, strides[2] = {(uint64_t)pitch * 2, 128};
    const uint32_t box[3] = {64, kStep, 2};
    return tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, p, dims, strides, box);
}

template <bool kTransposed>
int launch(const Dims& d, const Plan& p, const uint32_t* peaks, const float* factors, const __half* hi, const __half* lo,
           int64_t M, const __half* b, float* out, cudaStream_t s)
{
    CUtensorMap mh, ml, mb, mo;
    const uint64_t odims[3] = {(uint64_t)d.H, (uint64_t)d.F, (uint64_t)d.E},
                   ostride[2] = {(uint64_t)d.H * 4, (uint64_t)(d.H * d.F) * 4};
    const uint32_t obox[3] = {16, 32, 1};
    int st;
    if ((st = map_f16(&mh, hi, d.rows(), M)) != FP8Z1_OK || (st = map_f16(&ml, lo, d.rows(), M)) != FP8Z1_OK ||
        (st = map_f16(&mb, b, d.rows(), d.Hp())) != FP8Z1_OK ||
        (st = kTransposed ? (mo = mb, FP8Z1_OK)
                          : tensor_map(&mo, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, out, odims, ostride, obox,
                                       CU_TENSOR_MAP_SWIZZLE_64B)) != FP8Z1_OK)
        return st;
    Args a = {};
    a.plan = p;
    a.peaks = peaks;
    a.factors = factors;
    a.pitch = 3 * d.F;
    a.out = out;
    a.M = M;
    a.N = d.H;
    a.m_tiles = (int32_t)(M / 128);
    a.n_tiles = (int32_t)ceil_div(d.H, kCols);
    a.experts = (int32_t)d.E;
    const int64_t total = (int64_t)((a.m_tiles + 1) / 2) * a.n_tiles * d.E;
    return launch_persistent<wgrad_kernel<kTransposed>, 2>(kThreads, kSmem, total, s, mh, ml, mb, mo, a);
}

}  // namespace

int launch_d_gate_up(const Dims& d, const Plan& p, const Backward& b, float* out, cudaStream_t s)
{
    return launch<true>(d, p, &b.peaks->x, b.factors, b.dgu_hi, b.dgu_lo, 2 * d.F, b.x16, out, s);
}

int launch_d_down(const Dims& d, const Plan& p, const Backward& b, float* out, cudaStream_t s)
{
    return launch<false>(d, p, &b.peaks->dy, b.factors + 2 * d.F, b.h_hi, b.h_lo, d.F, b.dy16, out, s);
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

}  // namespace ffn
}  // namespace fp8z1
