// Embedding lookup from an FP8 table, and the table's gradient.
//
//   out[t, d]     = alpha * e4m3(code[id_t, d]) * scale[id_t / 128, d / 128]
//   d_table[v, d] = alpha * sum over {t : id_t = v} of dy[t, d]
//
// Both are bound by memory.  The lookup reads a code and writes an element (16384
// tokens of 7168 to BF16: 49 us, 7.3 TB/s with repeated tokens from L2); the
// gradient reads dy once and writes the whole FP32 table, most of it zeros.
//
// The gradient sorts the tokens by id (stable, so equal ids stay in order of
// t), cuts the sorted list into chunks of 32 and gives a chunk and a slice of
// columns to a CTA, which adds up runs of equal ids in registers.  A run inside
// one chunk is written at once; one that crosses chunks leaves a partial sum in
// each, and a last kernel adds those up in order.  Nothing depends on the order
// in which CTAs run: no atomics on floating point.
//
// Nearly all of the time is the table's zeros.  Up to 16384 tokens one CTA sorts
// while the others clear as much as takes that long; what is left of a large table
// is cleared beside the sums, by CTAs that look up which of their rows have a
// token and leave those out.  131072 x 4096 with 16384 tokens: 360 us, 6.3 TB/s
// (412 with all of it cleared beside the sort); with 2000 tokens 322 (359); with
// 40000, sorted in passes, 503 (598).
#include <algorithm>
#include <type_traits>

#include "ops_common.cuh"

namespace {

using namespace fp8z1;

struct Ids {
    const void* p;
    int32_t bytes;
    __device__ __forceinline__ int64_t at(int64_t t) const
    {
        return bytes == 8 ? static_cast<const int64_t*>(p)[t] : static_cast<const int32_t*>(p)[t];
    }
};

// ---- lookup --------------------------------------------------------------------

constexpr int kEmbedThreads = 256;

// Eight columns a thread, kTokens tokens at once (their loads in flight
// together).
template <class T, int kTokens>
__global__ void __launch_bounds__(kEmbedThreads)
embed_kernel(int64_t vocab, int64_t dim, const uint8_t* __restrict__ codes, const float* __restrict__ scales, Ids ids,
             int64_t tokens, float alpha, T* __restrict__ out, int64_t ld)
{
    const int64_t d = ((int64_t)blockIdx.y * kEmbedThreads + threadIdx.x) * 8;
    if (d >= dim) return;
    const int64_t t0 = (int64_t)blockIdx.x * kTokens, sc = (dim + 127) / 128;
    uint2 c[kTokens];
    float s[kTokens];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        c[i] = make_uint2(0, 0);
        s[i] = 0.0f;
        if (t0 + i >= tokens) continue;
        const int64_t id = ids.at(t0 + i);
        if (id < 0 || id >= vocab) continue;
        c[i] = __ldg(reinterpret_cast<const uint2*>(codes + id * dim + d));
        s[i] = __ldg(scales + id / 128 * sc + d / 128);
    }
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
        if (t0 + i >= tokens) continue;
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = e4m3x2_decode((j < 2 ? c[i].x : c[i].y) >> (16 * (j & 1)) & 0xffffu);
            f[2 * j] = alpha * (v.x * s[i]);
            f[2 * j + 1] = alpha * (v.y * s[i]);
        }
        T* o = out + (t0 + i) * ld + d;
        if constexpr (sizeof(T) == 4) {
            __stcs(reinterpret_cast<float4*>(o), make_float4(f[0], f[1], f[2], f[3]));
            __stcs(reinterpret_cast<float4*>(o) + 1, make_float4(f[4], f[5], f[6], f[7]));
        } else {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 two = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&two);
            }
            __stcs(reinterpret_cast<uint4*>(o), make_uint4(w[0], w[1], w[2], w[3]));
        }
    }
}

// Any dim and alignment: a column a thread.
template <class T>
__global__ void __launch_bounds__(kEmbedThreads)
embed_any_kernel(int64_t vocab, int64_t dim, const uint8_t* __restrict__ codes, const float* __restrict__ scales,
                 Ids ids, float alpha, T* __restrict__ out, int64_t ld)
{
    const int64_t t = blockIdx.x, id = ids.at(t), sc = (dim + 127) / 128;
    const bool there = id >= 0 && id < vocab;
    for (int64_t d = (int64_t)blockIdx.y * kEmbedThreads + threadIdx.x; d < dim;
         d += (int64_t)gridDim.y * kEmbedThreads)
        out[t * ld + d] = from_float<T>(
            there ? alpha * (e4m3_value(__ldg(codes + id * dim + d)) * __ldg(scales + id / 128 * sc + d / 128)) : 0.0f);
}

template <class T>
int launch_embed(int64_t vocab, int64_t dim, const uint8_t* codes, const float* scales, Ids ids, int64_t tokens,
                 float alpha, T* out, int64_t ld, cudaStream_t s)
{
    count_launch();
    if (dim % 8 == 0 && aligned(codes, 8) && aligned(out, 16) && ld * sizeof(T) % 16 == 0 &&
        ceil_div(dim, 8 * kEmbedThreads) <= 65535) {
        const unsigned slices = (unsigned)ceil_div(dim, 8 * kEmbedThreads);
        // 4 tokens a thread once that still leaves several CTAs for every SM
        if (tokens * slices >= 4 * kSms * 8)
            embed_kernel<T, 4><<<dim3((unsigned)ceil_div(tokens, 4), slices), kEmbedThreads, 0, s>>>(
                vocab, dim, codes, scales, ids, tokens, alpha, out, ld);
        else
            embed_kernel<T, 1><<<dim3((unsigned)tokens, slices), kEmbedThreads, 0, s>>>(vocab, dim, codes, scales, ids,
                                                                                       tokens, alpha, out, ld);
    } else {
        const int64_t slices = ceil_div(dim, 4 * kEmbedThreads);
        embed_any_kernel<T><<<dim3((unsigned)tokens, (unsigned)(slices < 65535 ? slices : 65535)), kEmbedThreads, 0, s>>>(
            vocab, dim, codes, scales, ids, alpha, out, ld);
    }
    return launch_status();
}

// ---- sorting the tokens by id ------------------------------------------------------

constexpr int kSortThreads = 1024, kSortWarps = 32, kBins = 256;

// What the gradient needs of the sort: keys ascending (ids; `vocab` for no
// token, at the end), the tokens behind them, and how many are real.
struct Sorted {
    uint32_t* key;
    int32_t* token;
    int32_t* n_real;
};

__device__ __forceinline__ uint32_t key_of(Ids ids, int64_t t, int64_t vocab)
{
    const int64_t id = ids.at(t);
    return (uint32_t)(id >= 0 && id < vocab ? id : vocab);
}

// Clears `n` floats from CTA `cta` of `ctas`.
__device__ __forceinline__ void clear(float* p, int64_t n, int64_t cta, int64_t ctas)
{
    const int64_t head = min(n, (int64_t)((16 - reinterpret_cast<uintptr_t>(p) % 16) % 16 / 4));
    float4* v = reinterpret_cast<float4*>(p + head);
    const int64_t n4 = (n - head) / 4;
    for (int64_t i = cta * blockDim.x + threadIdx.x; i < n4; i += ctas * blockDim.x)
        __stcs(v + i, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
    if (cta == 0 && threadIdx.x < head) p[threadIdx.x] = 0.0f;
    if (cta == 0 && (int64_t)threadIdx.x < n - head - n4 * 4) p[head + n4 * 4 + threadIdx.x] = 0.0f;
}

// The stable order of one digit within a CTA: every warp holds kItems x 32
// consecutive keys; on return rank[j] is the key's place among the warp's keys of
// its digit, and counts[bin * kSortWarps + warp] how many of them there are.
template <int kItems>
__device__ __forceinline__ void rank_in_warp(const uint32_t (&key)[kItems], int shift, uint16_t* counts,
                                             uint16_t (&rank)[kItems])
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint16_t* mine = counts + warp;  // [bin * kSortWarps]
    for (int b = lane; b < kBins; b += 32) mine[b * kSortWarps] = 0;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const uint32_t digit = key[j] >> shift & (kBins - 1);
        const unsigned peers = __match_any_sync(0xffffffffu, digit);
        const int before = __popc(peers & ((1u << lane) - 1));
        const uint16_t base = mine[digit * kSortWarps];
        rank[j] = (uint16_t)(base + before);
        __syncwarp();
        if (before == 0) mine[digit * kSortWarps] = (uint16_t)(base + __popc(peers));
        __syncwarp();
    }
}

// Exclusive sums of the kBins x kSortWarps counts, in place as 16-bit (a CTA
// holds at most 16384 keys): thread i owns counts [8 i, 8 i + 8).
__device__ __forceinline__ void scan_counts(uint16_t* counts, uint32_t* warp_sums)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint4* p = reinterpret_cast<uint4*>(counts) + threadIdx.x;
    const uint4 v = *p;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = sum;
        sum += w[i >> 1] >> (16 * (i & 1)) & 0xffffu;
    }
    uint32_t inclusive = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, inclusive, o);
        if (lane >= o) inclusive += up;
    }
    if (lane == 31) warp_sums[warp] = inclusive;
    __syncthreads();
    uint32_t before = inclusive - sum;
    for (int i = 0; i < warp; ++i) before += warp_sums[i];
    uint32_t o4[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o4[i] = (before + c[2 * i]) | (before + c[2 * i + 1]) << 16;
    *p = make_uint4(o4[0], o4[1], o4[2], o4[3]);
    __syncthreads();
}

// Up to kItems x 1024 tokens: CTA 0 sorts in shared memory (8 bits a pass),
// the others clear the table.
template <int kItems>
__global__ void __launch_bounds__(kSortThreads)
sort_small_kernel(Ids ids, int32_t tokens, int64_t vocab, int passes, Sorted out, float* table, int64_t n_table)
{
    if (blockIdx.x > 0) {
        clear(table, n_table, blockIdx.x - 1, gridDim.x - 1);
        return;
    }
    extern __shared__ uint8_t smem[];
    uint16_t* counts = reinterpret_cast<uint16_t*>(smem);                           // [kBins][kSortWarps]
    uint32_t* keys = reinterpret_cast<uint32_t*>(smem + kBins * kSortWarps * 2);    // [kItems * 1024]
    uint16_t* place = reinterpret_cast<uint16_t*>(keys + kItems * kSortThreads);    // [kItems * 1024]
    __shared__ uint32_t warp_sums[kSortWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t key[kItems];
    uint16_t token[kItems], rank[kItems];
    int real = 0;
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const int t = (warp * kItems + j) * 32 + lane;
        // past the end: after every key
        key[j] = t < tokens ? key_of(ids, t, vocab) : 0xffffffffu;
        token[j] = (uint16_t)t;
        real += key[j] < vocab;
    }
    for (int pass = 0; pass < passes; ++pass) {
        rank_in_warp<kItems>(key, pass * 8, counts, rank);
        __syncthreads();
        scan_counts(counts, warp_sums);
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int at = counts[(key[j] >> (pass * 8) & (kBins - 1)) * kSortWarps + warp] + rank[j];
            keys[at] = key[j];
            place[at] = token[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int at = (warp * kItems + j) * 32 + lane;
            key[j] = keys[at];
            token[j] = place[at];
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const int at = (warp * kItems + j) * 32 + lane;
        if (at < tokens) {
            out.key[at] = key[j];
            out.token[at] = token[j];
        }
    }
    real = __reduce_add_sync(0xffffffffu, real);
    if (lane == 0) warp_sums[warp] = real;
    __syncthreads();
    if (threadIdx.x == 0) {
        int n = 0;
        for (int i = 0; i < kSortWarps; ++i) n += warp_sums[i];
        *out.n_real = n;
    }
}

// More tokens: three launches for each 8 bits, a CTA for every 8192 keys.
constexpr int kSortItems = 8, kSortTile = kSortItems * kSortThreads;

struct Pass {
    Ids ids;  // the first pass reads these
    const uint32_t* key_in;
    const int32_t* token_in;
    uint32_t* key_out;
    int32_t* token_out;
    int64_t tokens, vocab;
    uint32_t* counts;  // [kBins, tiles]
    int64_t tiles;
    int shift;
};

__device__ __forceinline__ uint32_t pass_key(const Pass& p, int64_t t)
{
    if (t >= p.tokens) return 0xffffffffu;
    return p.key_in ? p.key_in[t] : key_of(p.ids, t, p.vocab);
}

// CTAs from `tiles` on clear the table (the first pass alone has them).
__global__ void __launch_bounds__(kSortThreads) count_kernel(Pass p, float* table, int64_t n_table)
{
    if (blockIdx.x >= p.tiles) {
        clear(table, n_table, blockIdx.x - p.tiles, gridDim.x - p.tiles);
        return;
    }
    __shared__ uint32_t bins[kBins];
    if (threadIdx.x < kBins) bins[threadIdx.x] = 0;
    __syncthreads();
    for (int j = 0; j < kSortItems; ++j) {
        const int64_t t = blockIdx.x * (int64_t)kSortTile + j * kSortThreads + threadIdx.x;
        if (t < p.tokens) atomicAdd(&bins[pass_key(p, t) >> p.shift & (kBins - 1)], 1u);
    }
    __syncthreads();
    if (threadIdx.x < kBins) p.counts[threadIdx.x * p.tiles + blockIdx.x] = bins[threadIdx.x];
}

// Exclusive sums over all counts, in one CTA.
__global__ void __launch_bounds__(kSortThreads) scan_kernel(uint32_t* counts, int64_t n)
{
    __shared__ uint32_t sums[kSortWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t carry = 0;
    for (int64_t i0 = 0; i0 < n; i0 += kSortThreads) {
        const int64_t i = i0 + threadIdx.x;
        const uint32_t v = i < n ? counts[i] : 0;
        uint32_t inclusive = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, inclusive, o);
            if (lane >= o) inclusive += up;
        }
        if (lane == 31) sums[warp] = inclusive;
        __syncthreads();
        uint32_t before = carry, all = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            if (w < warp) before += sums[w];
            all += sums[w];
        }
        if (i < n) counts[i] = before + inclusive - v;
        carry += all;
        __syncthreads();
    }
}

__global__ void __launch_bounds__(kSortThreads) scatter_kernel(Pass p)
{
    __shared__ uint16_t counts[kBins * kSortWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t key[kSortItems];
    uint16_t rank[kSortItems];
#pragma unroll
    for (int j = 0; j < kSortItems; ++j)
        key[j] = pass_key(p, blockIdx.x * (int64_t)kSortTile + (warp * kSortItems + j) * 32 + lane);
    rank_in_warp<kSortItems>(key, p.shift, counts, rank);
    __syncthreads();
    if (threadIdx.x < kBins) {  // each digit's keys in the warps before
        uint32_t sum = 0;
        for (int w = 0; w < kSortWarps; ++w) {
            const uint16_t c = counts[threadIdx.x * kSortWarps + w];
            counts[threadIdx.x * kSortWarps + w] = (uint16_t)sum;
            sum += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortItems; ++j) {
        const int64_t t = blockIdx.x * (int64_t)kSortTile + (warp * kSortItems + j) * 32 + lane;
        if (t >= p.tokens) continue;
        const uint32_t digit = key[j] >> p.shift & (kBins - 1);
        const int64_t at = (int64_t)p.counts[digit * p.tiles + blockIdx.x] + counts[digit * kSortWarps + warp] + rank[j];
        p.key_out[at] = key[j];
        p.token_out[at] = p.token_in ? p.token_in[t] : (int32_t)t;
    }
}

// The number of keys below vocab in the sorted list.
__global__ void count_real_kernel(const uint32_t* key, int64_t n, int64_t vocab, int32_t* n_real)
{
    int64_t a = 0, b = n;
    while (a < b) {
        const int64_t m = (a + b) / 2;
        if (key[m] < vocab)
            a = m + 1;
        else
            b = m;
    }
    *n_real = (int32_t)a;
}

// ---- adding up --------------------------------------------------------------------

constexpr int kChunk = 32, kSumThreads = 256;

struct Runs {
    Sorted s;
    float* partial;  // [chunks][2][dim]: the chunk's first run when it began before, its last when it goes on
    float* table;
    int64_t dim;
    float alpha;
    int64_t chunks;
    // rows [uncleared, vocab) hold no zeros yet: CTAs behind the chunks' have rows_each of them and clear what has no token
    int64_t uncleared, vocab, rows_each;
};

constexpr int kMostRowsEach = 128;

__device__ __forceinline__ void clear_unnamed_rows(const Runs& r)
{
    __shared__ bool named[kMostRowsEach];
    const int64_t r0 = r.uncleared + ((blockIdx.x - r.chunks) * gridDim.y + blockIdx.y) * r.rows_each;
    const int n = (int)max(min(r.rows_each, r.vocab - r0), (int64_t)0);
    if ((int)threadIdx.x < n) {
        int64_t a = 0, b = *r.s.n_real, end = b;
        const uint32_t row = (uint32_t)(r0 + threadIdx.x);
        while (a < b) {
            const int64_t m = (a + b) / 2;
            if (r.s.key[m] < row)
                a = m + 1;
            else
                b = m;
        }
        named[threadIdx.x] = a < end && r.s.key[a] == row;
    }
    __syncthreads();
    for (int i = 0; i < n; ++i)
        if (!named[i])
            for (int64_t d = threadIdx.x * 4; d < r.dim; d += kSumThreads * 4)
                __stcs(reinterpret_cast<float4*>(r.table + (r0 + i) * r.dim + d), make_float4(0.0f, 0.0f, 0.0f, 0.0f));
}

// Columns of a thread: 8 of aligned rows, 1 of others.
template <class T, int kCols>
struct Row {
    float f[kCols];
    __device__ __forceinline__ void load(const T* p)
    {
        if constexpr (kCols == 1) {
            f[0] = to_float(__ldcs(p));
        } else if constexpr (sizeof(T) == 4) {
            const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
            f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
        } else {
            const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                f[2 * i] = __uint_as_float(w[i] << 16);
                f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
};

template <int kCols>
__device__ __forceinline__ void store_cols(float* p, const float (&f)[kCols], float by)
{
    if constexpr (kCols == 1) {
        p[0] = by * f[0];
    } else {
        __stcs(reinterpret_cast<float4*>(p), make_float4(by * f[0], by * f[1], by * f[2], by * f[3]));
        __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(by * f[4], by * f[5], by * f[6], by * f[7]));
    }
}

template <class T, int kCols>
__global__ void __launch_bounds__(kSumThreads) sum_kernel(Runs r, const T* __restrict__ dy, int64_t ld)
{
    __shared__ uint32_t key[kChunk + 2];
    __shared__ int32_t token[kChunk];
    if constexpr (kCols == 8)
        if (blockIdx.x >= r.chunks) return clear_unnamed_rows(r);
    const int64_t c = blockIdx.x, p0 = c * kChunk, real = *r.s.n_real;
    if (p0 >= real) return;
    const int n = (int)min((int64_t)kChunk, real - p0);
    if (threadIdx.x < kChunk + 2) {
        const int64_t p = p0 - 1 + threadIdx.x;  // key[i + 1] is position p0 + i's
        key[threadIdx.x] = p >= 0 && p < real ? r.s.key[p] : 0xffffffffu;
        if (threadIdx.x < n) token[threadIdx.x] = r.s.token[p0 + threadIdx.x];
    }
    __syncthreads();
    const int64_t d = ((int64_t)blockIdx.y * kSumThreads + threadIdx.x) * kCols;
    if (d >= r.dim) return;
    constexpr int kAhead = kCols == 1 ? 8 : 4;
    float sum[kCols] = {};
    int start = 0;
    for (int i0 = 0; i0 < n; i0 += kAhead) {
        Row<T, kCols> row[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i0 + i < n) row[i].load(dy + (int64_t)token[i0 + i] * ld + d);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int at = i0 + i;
            if (at >= n) break;
            const uint32_t v = key[at + 1];
#pragma unroll
            for (int j = 0; j < kCols; ++j) sum[j] += row[i].f[j];
            const bool goes_on = key[at + 2] == v;
            if (goes_on && at + 1 < n) continue;
            const bool began_before = start == 0 && key[0] == v;
            if (!goes_on && !began_before)
                store_cols<kCols>(r.table + (int64_t)v * r.dim + d, sum, r.alpha);
            else
                store_cols<kCols>(r.partial + (c * 2 + (began_before ? 0 : 1)) * r.dim + d, sum, 1.0f);
            start = at + 1;
#pragma unroll
            for (int j = 0; j < kCols; ++j) sum[j] = 0.0f;
        }
    }
}

// The runs that cross chunks, each by the CTAs of the chunk it begins in.
template <int kCols>
__global__ void __launch_bounds__(kSumThreads) join_kernel(Runs r)
{
    const int64_t c = blockIdx.x, real = *r.s.n_real, last = (c + 1) * kChunk - 1;
    if (last + 1 >= real) return;
    const uint32_t v = r.s.key[last];
    if (r.s.key[last + 1] != v) return;                                      // ends here
    if (c > 0 && r.s.key[c * kChunk - 1] == v) return;                        // began before
    // the chunk it ends in: the first after c whose last key is not followed by another v
    __shared__ int32_t stop;
    int64_t end = c + 1;
    for (;; end += kSumThreads) {
        if (threadIdx.x == 0) stop = kSumThreads;
        __syncthreads();
        const int64_t q = (end + threadIdx.x + 1) * kChunk;  // the position after that chunk
        if (q >= real || r.s.key[q] != v) atomicMin(&stop, (int32_t)threadIdx.x);
        __syncthreads();
        const int found = stop;
        __syncthreads();
        if (found < kSumThreads) {
            end += found;
            break;
        }
    }
    const int64_t d = ((int64_t)blockIdx.y * kSumThreads + threadIdx.x) * kCols;
    if (d >= r.dim) return;
    Row<float, kCols> sum;
    sum.load(r.partial + (c * 2 + 1) * r.dim + d);
    constexpr int kAhead = 4;
    for (int64_t k = c + 1; k <= end; k += kAhead) {
        Row<float, kCols> part[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (k + i <= end) part[i].load(r.partial + (k + i) * 2 * r.dim + d);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (k + i <= end)
#pragma unroll
                for (int j = 0; j < kCols; ++j) sum.f[j] += part[i].f[j];
    }
    store_cols<kCols>(r.table + (int64_t)v * r.dim + d, sum.f, r.alpha);
}

template <class T, int kCols>
int launch_sums(const Runs& r, const T* dy, int64_t ld, int64_t tokens, cudaStream_t s)
{
    const dim3 grid((unsigned)r.chunks, (unsigned)ceil_div(r.dim, kSumThreads * kCols));
    const int64_t clearing = ceil_div(ceil_div(r.vocab - r.uncleared, r.rows_each), grid.y);
    count_launch();
    sum_kernel<T, kCols><<<dim3((unsigned)(r.chunks + clearing), grid.y), kSumThreads, 0, s>>>(r, dy, ld);
    if (tokens > kChunk) {
        count_launch();
        join_kernel<kCols><<<grid, kSumThreads, 0, s>>>(r);
    }
    return launch_status();
}

// ---- entry points -----------------------------------------------------------------

int check_ids(int64_t vocab, int64_t dim, const void* ids, int32_t id_bytes, int64_t tokens, float alpha,
              const void* rows, int32_t type, int64_t ld)
{
    if (vocab < 1 || vocab >= (int64_t)1 << 31 || dim < 1 || dim > (int64_t)1 << 23 || tokens < 0 ||
        tokens > kMaxRows || (id_bytes != 4 && id_bytes != 8) || (type != FP8Z1_F32 && type != FP8Z1_BF16) ||
        ld < dim || !isfinite(alpha))
        return FP8Z1_EINVAL;
    if (tokens > 0 && (!ids || !rows)) return FP8Z1_EINVAL;
    if (!aligned(ids, id_bytes) || !aligned(rows, type == FP8Z1_F32 ? 4 : 2)) return FP8Z1_EALIGN;
    return FP8Z1_OK;
}

// The workspace: the sorted list, the other halves of the sort's passes, counts, partial sums.
struct Space {
    int32_t* n_real;
    uint32_t* key[2];
    int32_t* token[2];
    uint32_t* counts;
    float* partial;
    int64_t bytes;
    Space(void* base, int64_t dim, int64_t tokens)
    {
        char* p = static_cast<char*>(base);
        int64_t at = 0;
        auto take = [&](int64_t n) {
            char* q = p ? p + at : nullptr;
            at += align256(n);
            return q;
        };
        n_real = reinterpret_cast<int32_t*>(take(4));
        for (int i = 0; i < 2; ++i) {
            key[i] = reinterpret_cast<uint32_t*>(take(tokens * 4));
            token[i] = reinterpret_cast<int32_t*>(take(tokens * 4));
        }
        counts = reinterpret_cast<uint32_t*>(take(ceil_div(tokens, kSortTile) * kBins * 4));
        partial = reinterpret_cast<float*>(take(ceil_div(tokens, kChunk) * 2 * dim * 4));
        bytes = at;
    }
};

// Keys of a thread of the one sorting CTA: 2048 tokens take 10 to 15 us to sort (two
// and three passes), 4096 13 to 20, 8192 21 to 33, 16384 40 to 63; and the bytes that
// the other CTAs clear in about that time.
constexpr int sort_items(int64_t tokens)
{
    return tokens <= 2 * kSortThreads ? 2 : tokens <= 4 * kSortThreads ? 4 : tokens <= 8 * kSortThreads ? 8 : 16;
}
constexpr int64_t cleared_beside(int items) { return (int64_t)(64 + 21 * items) << 20; }

constexpr int sort_smem(int items) { return kBins * kSortWarps * 2 + items * kSortThreads * 6; }

template <int kItems>
int sort_small(Ids ids, int64_t tokens, int64_t vocab, int passes, const Sorted& out, float* table, int64_t n_table,
               unsigned clear_ctas, cudaStream_t s)
{
    if (!allow_smem<sort_small_kernel<kItems>>(sort_smem(kItems))) return FP8Z1_ECUDA;
    count_launch();
    sort_small_kernel<kItems><<<1 + clear_ctas, kSortThreads, sort_smem(kItems), s>>>(
        ids, (int32_t)tokens, vocab, passes, out, table, n_table);
    return launch_status();
}

}  // namespace

extern "C" int fp8z1_embed(int64_t vocab, int64_t dim, const uint8_t* codes, const float* scales, const void* ids,
                           int32_t id_bytes, int64_t tokens, float alpha, void* out, int32_t out_type,
                           int64_t ld_out, void* stream)
{
    if (!codes || !scales) return FP8Z1_EINVAL;
    const int st = check_ids(vocab, dim, ids, id_bytes, tokens, alpha, out, out_type, ld_out);
    if (st != FP8Z1_OK) return st;
    if (!aligned(scales, 4)) return FP8Z1_EALIGN;
    if (tokens == 0) return FP8Z1_OK;
    NvtxRange r("fp8z1_embed");
    const Ids i{ids, id_bytes};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (out_type == FP8Z1_F32)
        return launch_embed(vocab, dim, codes, scales, i, tokens, alpha, static_cast<float*>(out), ld_out, s);
    return launch_embed(vocab, dim, codes, scales, i, tokens, alpha, static_cast<__nv_bfloat16*>(out), ld_out, s);
}

extern "C" int fp8z1_embed_grad_workspace(int64_t vocab, int64_t dim, int64_t tokens, int64_t* bytes)
{
    if (!bytes || vocab < 1 || vocab >= (int64_t)1 << 31 || dim < 1 || dim > (int64_t)1 << 23 || tokens < 0 ||
        tokens > kMaxRows)
        return FP8Z1_EINVAL;
    *bytes = Space(nullptr, dim, tokens).bytes;
    return FP8Z1_OK;
}

extern "C" int fp8z1_embed_grad(int64_t vocab, int64_t dim, const void* ids, int32_t id_bytes, int64_t tokens,
                                float alpha, const void* dy, int32_t dy_type, int64_t ld_dy, float* d_table,
                                void* workspace, void* stream)
{
    if (!d_table || !workspace) return FP8Z1_EINVAL;
    int st = check_ids(vocab, dim, ids, id_bytes, tokens, alpha, dy, dy_type, ld_dy);
    if (st != FP8Z1_OK) return st;
    if (!aligned(d_table, 4) || !aligned(workspace, 256)) return FP8Z1_EALIGN;
    NvtxRange range("fp8z1_embed_grad");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t n_table = vocab * dim;
    if (tokens == 0)
        return cudaMemsetAsync(d_table, 0, (size_t)n_table * 4, s) == cudaSuccess ? FP8Z1_OK : FP8Z1_ECUDA;
    const Ids i{ids, id_bytes};
    Space w(workspace, dim, tokens);
    const int sms = sm_count_here();
    if (sms < 1) return FP8Z1_ECUDA;
    const int esz = dy_type == FP8Z1_F32 ? 4 : 2;
    const bool wide = dim % 8 == 0 && aligned(dy, 16) && ld_dy * esz % 16 == 0 && aligned(d_table, 16);
    // What is cleared while one CTA sorts (the passes of a larger sort are short launches that it would delay); the rest
    // beside the sums, where rows that get one are left out.
    int64_t first = vocab;
    if (wide) {
        const int64_t beside = tokens <= 16 * kSortThreads ? cleared_beside(sort_items(tokens)) : 0;
        if (beside / (dim * 4) < vocab) first = beside / (dim * 4);
    }
    // CTAs that clear: 64 KB each at least, two for every SM at most
    const int64_t n_first = first * dim, wanted = ceil_div(n_first, 16384);
    const unsigned clear_ctas = (unsigned)(wanted < 2 * sms ? wanted : 2 * sms);
    int bits = 1;  // of the keys 0 .. vocab
    while (vocab >> bits) ++bits;
    const int passes = (bits + 7) / 8;
    Sorted sorted{w.key[0], w.token[0], w.n_real};
    if (tokens <= 16 * kSortThreads) {
        const auto sort = [&](auto kItems) {
            return sort_small<decltype(kItems)::value>(i, tokens, vocab, passes, sorted, d_table, n_first, clear_ctas, s);
        };
        switch (sort_items(tokens)) {
            case 2: st = sort(std::integral_constant<int, 2>{}); break;
            case 4: st = sort(std::integral_constant<int, 4>{}); break;
            case 8: st = sort(std::integral_constant<int, 8>{}); break;
            default: st = sort(std::integral_constant<int, 16>{});
        }
    } else {
        const int64_t tiles = ceil_div(tokens, kSortTile);
        Pass p = {i, nullptr, nullptr, w.key[0], w.token[0], tokens, vocab, w.counts, tiles, 0};
        for (int k = 0; k < passes; ++k) {
            p.shift = 8 * k;
            p.key_out = w.key[k & 1];
            p.token_out = w.token[k & 1];
            count_launch();
            count_kernel<<<(unsigned)(tiles + (k == 0 ? clear_ctas : 0)), kSortThreads, 0, s>>>(p, d_table, n_table);
            count_launch();
            scan_kernel<<<1, kSortThreads, 0, s>>>(w.counts, tiles * kBins);
            count_launch();
            scatter_kernel<<<(unsigned)tiles, kSortThreads, 0, s>>>(p);
            p.key_in = p.key_out;
            p.token_in = p.token_out;
        }
        sorted.key = w.key[(passes - 1) & 1];
        sorted.token = w.token[(passes - 1) & 1];
        count_launch();
        count_real_kernel<<<1, 1, 0, s>>>(sorted.key, tokens, vocab, w.n_real);
        st = launch_status();
    }
    if (st != FP8Z1_OK) return st;
    // half a megabyte of rows for a clearing CTA
    const int64_t each = std::max<int64_t>(std::min<int64_t>((1 << 19) / (dim * 4), kMostRowsEach), 1);
    const Runs r{sorted, w.partial, d_table, dim, alpha, ceil_div(tokens, kChunk), first, vocab, each};
    if (dy_type == FP8Z1_F32) {
        const float* p = static_cast<const float*>(dy);
        return wide ? launch_sums<float, 8>(r, p, ld_dy, tokens, s) : launch_sums<float, 1>(r, p, ld_dy, tokens, s);
    }
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(dy);
    return wide ? launch_sums<__nv_bfloat16, 8>(r, p, ld_dy, tokens, s)
                : launch_sums<__nv_bfloat16, 1>(r, p, ld_dy, tokens, s);
}
