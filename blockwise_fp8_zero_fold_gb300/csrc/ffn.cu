// Gated feed-forward block on FP8 weights: entry points, the regrouping of
// token rows into tiles, and the elementwise kernels between the products
// (ffn_gemm.cu: products with FP8 weights; ffn_wgrad.cu: weight gradients).
//
// Forward:  plan, split x, gate_up (+ silu, product, encode), down; with few
//           tokens y comes from matrix-vector products (ffn_gemv.cu).
// Backward: plan, split dy, dh, the activation's backward with its encodings,
//           FP16 copies of x and dy, dx, d_gate_up, d_down.
#include <cooperative_groups.h>

#include <mutex>

#include "ffn.cuh"

namespace fp8z1 {
namespace ffn {

int tensor_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const uint64_t* dims,
               const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swizzle)
{
    typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            return Encode(nullptr);
        return reinterpret_cast<Encode>(fn);
    }();
    if (!encode) return FP8Z1_ECUDA;
    cuuint64_t d[5], st[5];
    cuuint32_t b[5], one[5];
    for (int i = 0; i < rank; ++i) {
        d[i] = dims[i];
        b[i] = box[i];
        one[i] = 1;
        if (i + 1 < rank) st[i] = strides[i];
    }
    return encode(map, type, (cuuint32_t)rank, const_cast<void*>(base), d, st, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? FP8Z1_OK
               : FP8Z1_ECUDA;
}

}  // namespace ffn
}  // namespace fp8z1

namespace {

using namespace fp8z1;
using namespace fp8z1::ffn;
namespace cg = cooperative_groups;

// The tiles of every expert.  Rows two experts claim (a table that does not
// ascend) are bounded too: the launch holds at most `most` tiles.
__global__ void __launch_bounds__(1024) plan_kernel(Runs runs, PlanBuffers p, int64_t most, Peaks* clear,
                                                    const Peaks* from)
{
    next_may_start();
    __shared__ int32_t sums[1024];
    const int e = threadIdx.x, n = (int)runs.experts;
    int64_t lo = 0, hi = 0;
    if (e < n) runs.get(e, lo, hi);
    const int64_t mine = (hi - lo + kRows - 1) / kRows;
    // a table that does not ascend could name more than `most` tiles: every expert's share ends there
    sums[e] = (int32_t)min(mine, most);
    __syncthreads();
    for (int o = 1; o < 1024; o <<= 1) {
        const int32_t add = e >= o ? sums[e - o] : 0;
        __syncthreads();
        sums[e] = (int32_t)min((int64_t)sums[e] + add, most);
        __syncthreads();
    }
    const int32_t first = e ? sums[e - 1] : 0, last = sums[e];
    if (e < n) {
        p.start[e] = first;
        p.tokens[e] = (int32_t)min(hi - lo, (int64_t)(last - first) * kRows);
        if (clear) {
            clear[e] = Peaks{from ? from[e].x : 0, 0, {}};
        }
    }
    if (e == n - 1) {
        p.start[n] = last;
        *p.n_tiles = last;
    }
    const int32_t total = sums[n - 1];
    // an expert's tiles two by two: half as many pairs as tiles, and half of one more where their number is odd
    __shared__ int32_t odd_of_warp[32], pair_start[1024];
    if (p.pairs) {
        const unsigned odd = __ballot_sync(0xffffffffu, (last - first) & 1);
        if ((e & 31) == 0) odd_of_warp[e >> 5] = __popc(odd);
        __syncthreads();
        if (e < n) {
            int32_t odds = __popc(odd & ((1u << (e & 31)) - 1));
            for (int w = 0; w < e >> 5; ++w) odds += odd_of_warp[w];
            p.pair_start[e] = pair_start[e] = (first + odds) / 2;
            if (e == n - 1) *p.n_pairs = (last + odds + (last - first & 1)) / 2;
        }
        __syncthreads();
    }
    for (int32_t t = threadIdx.x; t < total; t += 1024) {
        int a = 0, b = n - 1;  // the first expert whose tiles end after t
        while (a < b) {
            const int mid = (a + b) / 2;
            if (sums[mid] > t)
                b = mid;
            else
                a = mid + 1;
        }
        int64_t l, h;
        runs.get(a, l, h);
        const int32_t local = t - (a ? sums[a - 1] : 0);
        const int64_t token0 = l + (int64_t)local * kRows;
        p.tiles[t] = Tile{a, (int32_t)token0, (int32_t)min(h - token0, (int64_t)kRows), 0};
        if (p.pairs && local % 2 == 0) p.pairs[pair_start[a] + local / 2] = 2 * t + (t + 1 < sums[a]);
    }
}

__device__ __forceinline__ float2 bf16_pair(uint32_t two)
{
    return make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
}

// Rows of BF16 activations to FP8 pairs in the tiles' order (a warp kRowColumns
// of a row: with one row of 7168, a warp for all of it took 21 us; 16 lanes a block
// of 128), with each expert's peak; rows of no expert are zeroed in `rest`.  8192
// rows of 7168: 42 us, 5.6 TB/s (55 with a load at a time).
constexpr int kRowColumns = 1024;
__global__ void __launch_bounds__(256) split_kernel(Runs runs, Plan plan, const bf16* x, int64_t ld, int64_t H,
                                                    Pairs out, int64_t rows, Peaks* peaks, bool dy, bf16* rest,
                                                    int64_t ld_rest)
{
    next_may_start();
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t n_rows = (int64_t)*plan.n_tiles * kRows;
    const int64_t c0 = (int64_t)blockIdx.y * kRowColumns, c1 = min(c0 + kRowColumns, out.pitch);
    if (rest) {
        int64_t lo, hi;
        runs.get(runs.experts - 1, lo, hi);
        for (int64_t r = hi + warp; r < runs.tokens; r += (int64_t)gridDim.x * 8)
            for (int64_t c = c0 + lane * 8; c < min(c1, H); c += 256)
                *reinterpret_cast<uint4*>(rest + r * ld_rest + c) = make_uint4(0, 0, 0, 0);
    }
    if (warp >= n_rows) return;
    const Tile t = plan.tiles[warp / kRows];
    const int r = (int)(warp % kRows);
    if (r >= t.rows) return;
    const bf16* src = x + (int64_t)(t.token0 + r) * ld;
    constexpr int kLoads = kRowColumns / 256;  // all on their way before the first is needed
    uint4 v[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int64_t c = c0 + i * 256 + lane * 8;
        v[i] = make_uint4(0, 0, 0, 0);
        if (c < H) v[i] = __ldg(reinterpret_cast<const uint4*>(src + c));
    }
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int64_t c = c0 + i * 256 + lane * 8;
        const float2 f[4] = {bf16_pair(v[i].x), bf16_pair(v[i].y), bf16_pair(v[i].z), bf16_pair(v[i].w)};
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) amax = fmaxf(amax, fmaxf(fabsf(f[j].x), fabsf(f[j].y)));
        // the expert's peak is that of its finite numbers: an infinity stays one in FP16, the others keep their bits
        if (amax == INFINITY) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (fabsf(f[j].x) < INFINITY) top = fmaxf(top, fabsf(f[j].x));
                if (fabsf(f[j].y) < INFINITY) top = fmaxf(top, fabsf(f[j].y));
            }
        } else {
            top = fmaxf(top, amax);
        }
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if (c >= out.pitch) continue;
        const PairScale ps = pair_scale(amax);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) pair_encode<Lo::kE5M2>(f[j].x, f[j].y, ps.up, hi[j], lo[j]);
        *reinterpret_cast<uint2*>(out.hi + warp * out.pitch + c) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
        *reinterpret_cast<uint2*>(out.lo + warp * out.pitch + c) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
        if ((lane & 15) == 0) out.scale[c / kBlock * rows + warp] = ps.down;
    }
    if (peaks) {
        const uint32_t p = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
        if (lane == 0) atomicMax(dy ? &peaks[t.expert].dy : &peaks[t.expert].x, p);
    }
}

__device__ __forceinline__ uint32_t half_pair(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Rows of x and dy to FP16 in the tiles' order, each expert's at its power of two.
// Bound by memory: 8192 rows of 7168 take 78 us, 6.0 TB/s.
__global__ void __launch_bounds__(256) halves_kernel(Plan plan, const bf16* x, int64_t ld_x, const bf16* dy,
                                                     int64_t ld_dy, int64_t H, int64_t pitch, __half* x16,
                                                     __half* dy16, const Peaks* peaks)
{
    next_may_start();
    after_previous();
    const int lane = threadIdx.x & 31;
    const int64_t warp = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (warp >= (int64_t)*plan.n_tiles * kRows) return;
    const Tile t = plan.tiles[warp / kRows];
    const int r = (int)(warp % kRows);
    if (r >= (t.rows + 15) / 16 * 16) return;  // zeros to the next multiple of 16, which is what is multiplied
    const Peaks p = peaks[t.expert];
    const Pow2 fx = pow2(peak_shift(p.x)), fd = pow2(peak_shift(p.dy));
    const bf16* sx = x + (int64_t)(t.token0 + r) * ld_x;
    const bf16* sd = dy + (int64_t)(t.token0 + r) * ld_dy;
    const int64_t c0 = (int64_t)blockIdx.y * kRowColumns, c1 = min(c0 + kRowColumns, pitch);
#pragma unroll
    for (int64_t c = c0 + lane * 8; c < c1; c += 256) {
        uint4 vx = make_uint4(0, 0, 0, 0), vd = vx;
        if (r < t.rows && c < H) {
            vx = __ldg(reinterpret_cast<const uint4*>(sx + c));
            vd = __ldg(reinterpret_cast<const uint4*>(sd + c));
        }
        const uint32_t wx[4] = {vx.x, vx.y, vx.z, vx.w}, wd[4] = {vd.x, vd.y, vd.z, vd.w};
        uint32_t ox[4], od[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 a = bf16_pair(wx[i]), b = bf16_pair(wd[i]);
            ox[i] = half_pair(fx.times(a.x), fx.times(a.y));
            od[i] = half_pair(fd.times(b.x), fd.times(b.y));
        }
        *reinterpret_cast<uint4*>(x16 + warp * pitch + c) = make_uint4(ox[0], ox[1], ox[2], ox[3]);
        *reinterpret_cast<uint4*>(dy16 + warp * pitch + c) = make_uint4(od[0], od[1], od[2], od[3]);
    }
}

// v times f as two FP16 numbers, four at a time
__device__ __forceinline__ void store_halves(__half* hi, __half* lo, const float4& f, const float4& v)
{
    const float a = f.x * v.x, b = f.y * v.y, c = f.z * v.z, d = f.w * v.w;
    const __half2 h0 = __floats2half2_rn(a, b), h1 = __floats2half2_rn(c, d);
    *reinterpret_cast<uint2*>(hi) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&h0), *reinterpret_cast<const uint32_t*>(&h1));
    const float2 g0 = __half22float2(h0), g1 = __half22float2(h1);
    *reinterpret_cast<uint2*>(lo) = make_uint2(half_pair(a - g0.x, b - g0.y), half_pair(c - g1.x, d - g1.y));
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// dg, du and h of 32 rows x 128 columns: read with lanes along rows (as the
// products wrote them), turned in shared memory, written with lanes along
// columns: [dg | du] as FP8 pairs for dx and as FP16 pairs for d_gate_up, h as
// FP16 pairs for d_down.  The eight CTAs of two tiles are a cluster: a column's power
// of two is that of its largest number in all 256 rows.  Bound by memory, 28 bytes an
// element: 8192 rows of 2048 take 127 us, 3.7 TB/s (100 with one power of two for an
// expert, known beforehand).  The peaks go through 32-bit words: stores of bytes in the
// load loop kept later loads behind them (302 us for 215 at 2051 rows of 14336).
constexpr int kActPitch = 132;
constexpr int kActSmem = (3 * 32 * kActPitch + 3 * 128) * 4;
__global__ void __launch_bounds__(256) activation_kernel(Plan plan, const float* gu, const float* dh, int64_t F,
                                                         int64_t rows, Pairs pairs, __half* dgu_hi, __half* dgu_lo,
                                                         __half* h_hi, __half* h_lo, float* factors)
{
    extern __shared__ __align__(16) float act[];  // [3][32][kActPitch], then the columns' powers of two
    __shared__ uint32_t mine[3 * 128];                 // this CTA's largest numbers of the columns (bits)
    __shared__ __align__(16) uint8_t peaks[8][3 * 128];  // the exponents of every CTA's
    next_may_start();
    after_previous();
    const int64_t pair = blockIdx.x >> 3;
    if (pair >= *plan.n_pairs) return;  // with the whole cluster
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();  // this CTA has started: the others may write to it
    const int rank = (int)cluster.block_rank();
    const int second = blockIdx.x >> 2 & 1, quarter = blockIdx.x & 3, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int32_t first_tile = plan.pairs[pair];
    const int64_t tile = (first_tile >> 1) + second;
    // of this CTA's 32 rows; it may have none
    const int rows_here = second && !(first_tile & 1) ? 0 : min(plan.tiles[tile].rows - quarter * 32, 32);
    const bool there = lane < rows_here;
    const int64_t f0 = (int64_t)blockIdx.y * 128;
    const float* pg = gu + (tile * 2 * F + f0) * kRows + quarter * 32 + lane;
    const float* pu = pg + F * kRows;
    const float* pd = dh + (tile * F + f0) * kRows + quarter * 32 + lane;
#pragma unroll 8
    for (int i = 0; i < 16; ++i) {
        const int c = warp * 16 + i;
        float g = 0.0f, u = 0.0f, d = 0.0f;
        if (there) {
            g = __ldcs(pg + c * kRows);
            u = __ldcs(pu + c * kRows);
            d = __ldcs(pd + c * kRows);
        }
        // the sigmoid and its complement, by exp(-|g|) <= 1: neither overflows nor cancels
        const float e = expf(-fabsf(g)), big = __fdividef(1.0f, 1.0f + e), small = e * big;
        const float s = g < 0.0f ? small : big, rest = g < 0.0f ? big : small, a = g * s;
        float* o = act + lane * kActPitch + c;
        const float dg = d * u * s * (1.0f + g * rest), du = d * a, h = a * u;
        o[0] = dg;
        o[32 * kActPitch] = du;
        o[64 * kActPitch] = h;
        const uint32_t p0 = __reduce_max_sync(0xffffffffu, abs_bits(dg)), p1 = __reduce_max_sync(0xffffffffu, abs_bits(du)),
                       p2 = __reduce_max_sync(0xffffffffu, abs_bits(h));
        if (lane == 0) mine[c] = p0, mine[128 + c] = p1, mine[256 + c] = p2;
    }
    __syncwarp();
    cluster.barrier_wait();
    if (lane < 24) {  // the warp's 16 columns of one of the three, to one of the CTAs
        const int at = lane % 3 * 128 + warp * 16;
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) v[j] |= mine[at + 4 * j + k] >> 23 << (8 * k);
        }
        *reinterpret_cast<uint4*>(cluster.map_shared_rank(&peaks[rank][at], lane / 3)) = make_uint4(v[0], v[1], v[2], v[3]);
    }
    __syncwarp();
    cluster.sync();
    float* up = act + 3 * 32 * kActPitch;
    if (threadIdx.x < 96) {  // four columns of one of the three
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) m = __vmaxu4(m, *reinterpret_cast<const uint32_t*>(&peaks[q][threadIdx.x * 4]));
        const ColumnScale x = column_scale(m & 255), y = column_scale(m >> 8 & 255), z = column_scale(m >> 16 & 255),
                          w = column_scale(m >> 24);
        *reinterpret_cast<float4*>(up + threadIdx.x * 4) = make_float4(x.up, y.up, z.up, w.up);
        if (rank == 0)
            *reinterpret_cast<float4*>(factors + (pair * 3 + threadIdx.x / 32) * F + f0 + lane * 4) =
                make_float4(x.down, y.down, z.down, w.down);
    }
    __syncthreads();
    const float4 fg = *reinterpret_cast<const float4*>(up + lane * 4),
                 fu = *reinterpret_cast<const float4*>(up + 128 + lane * 4),
                 fh = *reinterpret_cast<const float4*>(up + 256 + lane * 4);
    // zeros to the next multiple of 16, which is what the weight gradients multiply
    for (int r = warp; r < (rows_here + 15) / 16 * 16; r += 8) {
        const int64_t at = tile * kRows + quarter * 32 + r;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const float4 v = *reinterpret_cast<const float4*>(act + (half * 32 + r) * kActPitch + lane * 4);
            const int64_t col = half * F + f0 + lane * 4;
            store_halves(dgu_hi + at * 2 * F + col, dgu_lo + at * 2 * F + col, half ? fu : fg, v);
            if (pairs.hi) {
                float amax = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
                amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
                const PairScale ps = pair_scale(amax);
                uint32_t h0, l0, h1, l1;
                pair_encode<Lo::kE4M3>(v.x, v.y, ps.up, h0, l0);
                pair_encode<Lo::kE4M3>(v.z, v.w, ps.up, h1, l1);
                *reinterpret_cast<uint32_t*>(pairs.hi + at * pairs.pitch + col) = h0 | h1 << 16;
                *reinterpret_cast<uint32_t*>(pairs.lo + at * pairs.pitch + col) = l0 | l1 << 16;
                if (lane == 0) pairs.scale[(half * F + f0) / kBlock * rows + at] = ps.down;
            }
        }
        const float4 v = *reinterpret_cast<const float4*>(act + (64 + r) * kActPitch + lane * 4);
        store_halves(h_hi + at * F + f0 + lane * 4, h_lo + at * F + f0 + lane * 4, fh, v);
    }
}

int check_dims(const fp8z1_ffn_dims* d)
{
    if (!d || d->tokens < 0 || d->tokens > kMaxRows || d->hidden < 16 || d->hidden % 16 ||
        d->hidden >= (int64_t)1 << 24 || d->inner < 128 || d->inner % 128 || d->inner >= (int64_t)1 << 23 ||
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

Dims dims_of(const fp8z1_ffn_dims* d) { return Dims{d->tokens, d->hidden, d->inner, d->experts}; }

}  // namespace

extern "C" int fp8z1_ffn_sizes(const fp8z1_ffn_dims* dims, int64_t* saved_bytes, int64_t* forward_bytes,
                               int64_t* backward_bytes)
{
    const int st = check_dims(dims);
    if (st != FP8Z1_OK) return st;
    if (!saved_bytes || !forward_bytes || !backward_bytes) return FP8Z1_EINVAL;
    const Dims d = dims_of(dims);
    Cut saved(nullptr), forward(nullptr), backward(nullptr);
    Saved().cut(saved, d);
    Forward().cut(forward, d);
    Backward().cut(backward, d);
    *saved_bytes = saved.at;
    *forward_bytes = forward.at;
    *backward_bytes = backward.at;
    return FP8Z1_OK;
}

extern "C" int fp8z1_ffn_forward(const fp8z1_ffn_dims* dims, const void* x, int64_t ld_x, const int32_t* d_offsets,
                                 const uint8_t* gate_up, const float* gate_up_scale, const uint8_t* down,
                                 const float* down_scale, void* y, int64_t ld_y, void* saved, void* workspace,
                                 void* stream)
{
    int st = check_dims(dims);
    if (st != FP8Z1_OK) return st;
    if ((st = check_weights(dims, d_offsets, gate_up, gate_up_scale, down, down_scale)) != FP8Z1_OK) return st;
    const Dims d = dims_of(dims);
    if (d.T == 0) return FP8Z1_OK;
    if ((st = check_rows(x, ld_x, d.H)) != FP8Z1_OK || (st = check_rows(y, ld_y, d.H)) != FP8Z1_OK) return st;
    if (!workspace) return FP8Z1_EINVAL;
    if (!aligned(saved, 256) || !aligned(workspace, 256)) return FP8Z1_EALIGN;
    NvtxRange range("fp8z1_ffn_forward");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const Runs runs{d_offsets, d.T, d.E};
    const Weight wgu{gate_up, gate_up_scale, d.H, 2 * d.F}, wd{down, down_scale, d.F, d.H};
    Cut cw(workspace), cs(saved);
    Forward f;
    f.cut(cw, d);
    if (few_tokens(d)) {  // y is the same whether the call saves or not
        st = launch_gemv(d, runs, static_cast<const bf16*>(x), ld_x, wgu, wd, f.part, static_cast<bf16*>(y), ld_y, s);
        if (st != FP8Z1_OK || !saved) return st;
    }
    Saved keep = {};
    if (saved) keep.cut(cs, d);
    const Plan plan = f.plan.plan();
    const dim3 row_ctas((unsigned)ceil_div(d.rows(), 8), (unsigned)ceil_div(d.Hp(), kRowColumns));
    count_launch();
    plan_kernel<<<1, 1024, 0, s>>>(runs, f.plan, d.tiles(), keep.peaks, nullptr);
    if ((st = launch_status()) != FP8Z1_OK ||
        (st = launch_after(split_kernel, row_ctas, 256, 0, s, runs, plan, static_cast<const bf16*>(x), ld_x, d.H, f.x,
                           d.rows(), keep.peaks, false, static_cast<bf16*>(y), ld_y)) != FP8Z1_OK ||
        (st = launch_gate_up(d, plan, f.x, wgu, f.h, keep.gu, f.part, s)) != FP8Z1_OK)
        return st;
    if (few_tokens(d)) return FP8Z1_OK;
    return launch_down(d, plan, f.h, wd, static_cast<bf16*>(y), ld_y, f.part, s);
}

extern "C" int fp8z1_ffn_backward(const fp8z1_ffn_dims* dims, const void* dy, int64_t ld_dy, const void* x,
                                  int64_t ld_x, const int32_t* d_offsets, const uint8_t* gate_up,
                                  const float* gate_up_scale, const uint8_t* down, const float* down_scale,
                                  const void* saved, void* dx, int64_t ld_dx, float* d_gate_up, float* d_down,
                                  void* workspace, void* stream)
{
    int st = check_dims(dims);
    if (st != FP8Z1_OK) return st;
    if ((st = check_weights(dims, d_offsets, gate_up, gate_up_scale, down, down_scale)) != FP8Z1_OK) return st;
    if (!d_gate_up || !d_down) return FP8Z1_EINVAL;
    if (!aligned(d_gate_up, 16) || !aligned(d_down, 16)) return FP8Z1_EALIGN;
    const Dims d = dims_of(dims);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (d.T == 0) {
        if (cudaMemsetAsync(d_gate_up, 0, (size_t)(d.E * d.H * 2 * d.F) * 4, s) != cudaSuccess ||
            cudaMemsetAsync(d_down, 0, (size_t)(d.E * d.F * d.H) * 4, s) != cudaSuccess)
            return FP8Z1_ECUDA;
        return FP8Z1_OK;
    }
    if ((st = check_rows(x, ld_x, d.H)) != FP8Z1_OK || (st = check_rows(dy, ld_dy, d.H)) != FP8Z1_OK ||
        (dx && (st = check_rows(dx, ld_dx, d.H)) != FP8Z1_OK))
        return st;
    if (!saved || !workspace) return FP8Z1_EINVAL;
    if (!aligned(saved, 256) || !aligned(workspace, 256)) return FP8Z1_EALIGN;
    NvtxRange range("fp8z1_ffn_backward");
    const Runs runs{d_offsets, d.T, d.E};
    const Weight wgu{gate_up, gate_up_scale, d.H, 2 * d.F}, wd{down, down_scale, d.F, d.H};
    Cut cw(workspace), cs(const_cast<void*>(saved));
    Backward b;
    b.cut(cw, d);
    Saved keep;
    keep.cut(cs, d);
    const Plan plan = b.plan.plan();
    const bf16 *xb = static_cast<const bf16*>(x), *dyb = static_cast<const bf16*>(dy);
    const dim3 row_ctas((unsigned)ceil_div(d.rows(), 8), (unsigned)ceil_div(d.Hp(), kRowColumns));
    count_launch();
    plan_kernel<<<1, 1024, 0, s>>>(runs, b.plan, d.tiles(), b.peaks, keep.peaks);
    if ((st = launch_status()) != FP8Z1_OK ||
        (st = launch_after(split_kernel, row_ctas, 256, 0, s, runs, plan, dyb, ld_dy, d.H, b.dy, d.rows(), b.peaks, true,
                           static_cast<bf16*>(dx), ld_dx)) != FP8Z1_OK ||
        (st = launch_dh(d, plan, b.dy, wd, b.dh, s)) != FP8Z1_OK)
        return st;
    Pairs pairs = b.dgu;
    if (!dx) pairs.hi = nullptr;
    if (!allow_smem<activation_kernel>(kActSmem)) return FP8Z1_ECUDA;
    if ((st = launch_after<8>(activation_kernel, dim3((unsigned)(d.pairs() * 8), (unsigned)(d.F / 128)), 256, kActSmem, s,
                              plan, keep.gu, b.dh, d.F, d.rows(), pairs, b.dgu_hi, b.dgu_lo, b.h_hi, b.h_lo,
                              b.factors)) != FP8Z1_OK ||
        (st = launch_after(halves_kernel, row_ctas, 256, 0, s, plan, xb, ld_x, dyb, ld_dy, d.H, d.Hp(), b.x16, b.dy16,
                           b.peaks)) != FP8Z1_OK)
        return st;
    if (dx && (st = launch_dx(d, plan, b.dgu, wgu, static_cast<bf16*>(dx), ld_dx, s)) != FP8Z1_OK) return st;
    if ((st = launch_d_gate_up(d, plan, b, d_gate_up, s)) != FP8Z1_OK) return st;
    return launch_d_down(d, plan, b, d_down, s);
}

extern "C" int fp8z1_ffn_timeouts(uint32_t* count)
{
    if (!count) return FP8Z1_EINVAL;
    // the devices' counters only grow, so that no count is lost between a read and a reset
    static std::mutex lock;
    static uint32_t seen[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return FP8Z1_ECUDA;
    std::lock_guard<std::mutex> hold(lock);
    unsigned a = 0, b = 0;
    int st = read_timeouts_gemm(&a);
    if (st == FP8Z1_OK) st = read_timeouts_wgrad(&b);
    if (st != FP8Z1_OK) {
        cudaGetLastError();
        return st;
    }
    *count = a + b - seen[dev];
    seen[dev] = a + b;
    return FP8Z1_OK;
}

extern "C" int fp8z1_checked_ffn_stall(uint32_t kernels)
{
#if FP8Z1_CHECKED
    const int st = stall_gemm(kernels & 31);
    return st == FP8Z1_OK ? stall_wgrad(kernels >> 5) : st;
#else
    (void)kernels;
    return FP8Z1_EINVAL;
#endif
}
