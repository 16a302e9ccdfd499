// Tokens sorted by expert, and back.
//
// A choice (t, j) of expert ids[t, j] gets a row: rows are grouped by expert, a group
// in the order of the choices.  offsets[e] is the first row of expert e, place[t, j]
// the choice's row (-1: no expert).
//
//   dispatch   rows[place[t, j]] = x[t], rows behind the last 0
//   combine    y[t] = r[t] + sum_j w[t, j] rows[place[t, j]]     (with w = 1 dispatch's gradient)
//   gradient   d_rows[place[t, j]] = w[t, j] dy[t],   d_w[t, j] = dy[t] . rows[place[t, j]]
//
// Sums are FP32 in the order of j (over columns: of the threads), without atomics.
// All four are bound by the rows moved: a token's row is read once for all its choices.
//
// 8192 tokens of 7168 BF16, 8 of 32 experts each: dispatch 156 us, 6.8 TB/s; combine 158 us, 6.7 TB/s, with a
// residual 180, 6.5; its gradient 300 us, 6.7 TB/s; the sort of 65536 choices 11 us.  61 tokens: 5, 4 and 4 us.
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "ops_common.cuh"

namespace fp8z1 {
namespace {

using bf16 = __nv_bfloat16;
namespace cg = cooperative_groups;

constexpr int kMostExperts = 1024, kMostTop = 64;

// ---- the sort -----------------------------------------------------------------------
//
// A cluster of CTAs, each warp a run of the choices: a choice's rank among those of its
// expert in the warp (by a match of the lanes, 32 choices a step, and the warp's counts in
// shared memory), the counts' sums over warps, CTAs and experts, and each choice's row is
// what lies before its warp's and its rank.  Bound by latency: the choices of a warp's
// first kHeld steps are on their way at once and stay in registers with their ranks, an
// expert's counts are added by a warp with a lane for each.

constexpr int kHeld = 16;

struct SortArgs {
    const void* ids;
    int64_t n;
    int32_t experts;
    int32_t per_warp;  // choices of a warp, a multiple of 32
    int32_t *offsets, *place;
};

template <class Id>
__device__ __forceinline__ int expert_of(const Id* ids, int64_t i, int64_t n, int experts)
{
    if (i >= n) return -1;
    const Id e = ids[i];
    return e >= 0 && e < (Id)experts ? (int)e : -1;
}

// The rank of each lane's choice among its expert's of the warp so far, which `mine` counts.
__device__ __forceinline__ int rank_of(int e, int32_t* mine, int lane)
{
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int rank = e < 0 ? 0 : mine[e] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
    return rank;
}

template <class Id>
__global__ void __launch_bounds__(1024) sort_kernel(const SortArgs a)
{
    extern __shared__ int32_t counts[];  // [warps][experts], then [experts] of the CTA
    __shared__ int32_t scan[32];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.experts;
    int32_t* mine = counts + warp * E;
    int32_t* total = counts + warps * E;
    const Id* ids = static_cast<const Id*>(a.ids);
    const int64_t i0 = ((int64_t)rank * warps + warp) * a.per_warp, i1 = min(i0 + a.per_warp, a.n);
    int held[kHeld], ranks[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
        held[k] = k * 32 < a.per_warp ? expert_of(ids, i0 + k * 32 + lane, a.n, E) : -1;
    for (int e = lane; e < E; e += 32) mine[e] = 0;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
        ranks[k] = 0;
        if (i0 + k * 32 < i1) ranks[k] = rank_of(held[k], mine, lane);
    }
    for (int64_t i = i0 + kHeld * 32; i < i1; i += 32) {  // these ranks wait in `place`
        const int rank_here = rank_of(expert_of(ids, i + lane, a.n, E), mine, lane);
        if (i + lane < a.n) a.place[i + lane] = rank_here;
    }
    __syncthreads();
    for (int e = warp; e < E; e += warps) {  // a lane a warp's counts: what lies before each of them
        const int32_t n = lane < warps ? counts[lane * E + e] : 0;
        int32_t sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += up;
        }
        if (lane < warps) counts[lane * E + e] = sum - n;
        if (lane == 31) total[e] = sum;
    }
    if (ctas > 1)
        cluster.sync();
    else
        __syncthreads();
    // a thread an expert: what lies before it, of the experts ahead and of its own in the CTAs ahead
    int32_t before = 0;  // of all experts up to this round's first
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        int32_t all = 0, ahead = 0;
        if (e < E)
#pragma unroll 8
            for (int c = 0; c < ctas; ++c) {
                const int32_t n = ctas > 1 ? cluster.map_shared_rank(total, c)[e] : total[e];
                if (c < rank) ahead += n;
                all += n;
            }
        int32_t sum = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int32_t n = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += n;
        }
        if (lane == 31) scan[warp] = sum;
        __syncthreads();
        const int32_t part = lane < warps ? scan[lane] : 0;
        const int32_t start = before + sum - all + (int32_t)__reduce_add_sync(0xffffffffu, lane < warp ? part : 0);
        before += (int32_t)__reduce_add_sync(0xffffffffu, part);
        if (e < E) {
            if (rank == 0) a.offsets[e] = start;
            if (rank == 0 && e == E - 1) a.offsets[E] = start + all;
        }
        if (ctas > 1)
            cluster.sync();  // the totals have been read
        else
            __syncthreads();
        if (e < E) total[e] = start + ahead;  // from here on the first row of the CTA's own
    }
    __syncthreads();
    auto place = [&](int64_t i, int e, int rank_here) {
        if (i < a.n) a.place[i] = e < 0 ? -1 : total[e] + mine[e] + rank_here;
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
        if (i0 + k * 32 < i1) place(i0 + k * 32 + lane, held[k], ranks[k]);
    for (int64_t i = i0 + kHeld * 32 + lane; i < i1; i += 32) place(i, expert_of(ids, i, a.n, E), a.place[i]);
}

// ---- rows ----------------------------------------------------------------------------

struct RowArgs {
    int64_t tokens, n;  // n: tokens * top
    int32_t top, experts;
    int64_t cols;       // of the element type, or of V
    const int32_t *offsets, *place;
    const float* weight;
    const void *x, *rows;
    void *y, *out;
    int64_t ld_x, ld_rows, ld_y, ld_out;
    float* d_weight;
};

// Rows behind the last expert's, cleared by the CTAs in turn.
template <class V>
__device__ __forceinline__ void clear_rest(const RowArgs& a, V* out, int64_t ld, int64_t cols)
{
    const int64_t last = min(max((int64_t)a.offsets[a.experts], (int64_t)0), a.n);
    for (int64_t r = last + blockIdx.x; r < a.n; r += gridDim.x)
        for (int64_t c = threadIdx.x; c < cols; c += blockDim.x) out[r * ld + c] = V{};
}

// A choice's row, or -1
__device__ __forceinline__ int64_t row_of(const RowArgs& a, int64_t choice)
{
    const int32_t p = __ldg(a.place + choice);
    return p >= 0 && p < a.n ? p : -1;
}

// A CTA a token; V: as many bytes of a row as its alignment lets be moved at a time.
template <class V>
__global__ void __launch_bounds__(256) dispatch_kernel(const RowArgs a)
{
    V* out = static_cast<V*>(a.out);
    const V* x = static_cast<const V*>(a.x) + (int64_t)blockIdx.x * a.ld_x;
    const int64_t first = (int64_t)blockIdx.x * a.top;
    for (int64_t c0 = 0; c0 < a.cols; c0 += 4 * blockDim.x) {
        V v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t c = c0 + i * blockDim.x + threadIdx.x;
            if (c < a.cols) v[i] = x[c];
        }
        for (int j = 0; j < a.top; ++j) {
            const int64_t r = row_of(a, first + j);
            if (r < 0) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t c = c0 + i * blockDim.x + threadIdx.x;
                if (c < a.cols) out[r * a.ld_out + c] = v[i];
            }
        }
    }
    clear_rest(a, out, a.ld_out, a.cols);
}

// What a thread takes of a row at a time: 16 bytes, or (rows that do not lie on them) four
// elements a CTA's width apart.  `left`: elements from its first to the row's end.
template <class T, bool kVec>
struct Piece;
template <class T>
struct Piece<T, false> {
    static constexpr int kN = 4;
    T raw[4];
    __device__ __forceinline__ void load(const T* p, int64_t left)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((int)blockDim.x * i < left) raw[i] = p[blockDim.x * i];
    }
    __device__ __forceinline__ void get(float (&v)[4]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = to_float(raw[i]);
    }
    static __device__ __forceinline__ void store(T* p, const float (&v)[4], int64_t left)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if ((int)blockDim.x * i < left) p[blockDim.x * i] = from_float<T>(v[i]);
    }
};
template <>
struct Piece<float, true> {
    static constexpr int kN = 4;
    float4 raw;
    __device__ __forceinline__ void load(const float* p, int64_t) { raw = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void get(float (&v)[4]) const { v[0] = raw.x, v[1] = raw.y, v[2] = raw.z, v[3] = raw.w; }
    static __device__ __forceinline__ void store(float* p, const float (&v)[4], int64_t)
    {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <>
struct Piece<bf16, true> {
    static constexpr int kN = 8;
    uint4 raw;
    __device__ __forceinline__ void load(const bf16* p, int64_t) { raw = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    static __device__ __forceinline__ void store(bf16* p, const float (&v)[8], int64_t)
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&two);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
// A thread's first element of a CTA's `part`-th width of pieces.
template <class T, bool kVec>
__device__ __forceinline__ int64_t first_of(int64_t part)
{
    return part * blockDim.x * Piece<T, kVec>::kN + threadIdx.x * (kVec ? Piece<T, kVec>::kN : 1);
}

// The choices of token t: rows and weights in shared memory.
struct Choices {
    int32_t row[kMostTop];  // -1: none
    float weight[kMostTop];
};
__device__ __forceinline__ void load_choices(Choices& c, const RowArgs& a, int64_t t)
{
    for (int j = threadIdx.x; j < a.top; j += blockDim.x) {
        const int64_t r = row_of(a, t * a.top + j);
        c.row[j] = (int32_t)r;
        c.weight[j] = r < 0 ? 0.0f : a.weight ? __ldg(a.weight + t * a.top + j) : 1.0f;
    }
    __syncthreads();
}

// Calls f<how many>(first) for `top` choices, kMost, then 4, 2 and 1 at a time: so many rows are on their way at
// once.  (Of single elements 4: 8 took 100 registers and 36 us for 3001 tokens' three rows of 1001 FP32.)
template <int kMost, class F>
__device__ __forceinline__ void by_parts(int top, F f)
{
    int j = 0;
    for (; j + kMost <= top; j += kMost) f(std::integral_constant<int, kMost>(), j);
    if (kMost > 4 && top & 4) f(std::integral_constant<int, 4>(), j), j += 4;
    if (top & 2) f(std::integral_constant<int, 2>(), j), j += 2;
    if (top & 1) f(std::integral_constant<int, 1>(), j);
}

// The pieces of kMany choices' rows from column c on.  The loads do not ask whether there is a row, so that
// they go together: a choice without one reads row 0, which is not used.
template <class T, bool kVec, int kMany>
__device__ __forceinline__ void load_rows(Piece<T, kVec> (&v)[kMany], const Choices& choices, int j0, const T* rows, int64_t ld,
                                          int64_t left)
{
#pragma unroll
    for (int j = 0; j < kMany; ++j) v[j].load(rows + (int64_t)max(choices.row[j0 + j], 0) * ld, left);
}

// Parts of a token's columns are neighbouring CTAs'.  A CTA waits for its choices, then for their rows: what its registers
// leave to other CTAs pays.  us with a residual, 8192 tokens: BF16, eight rows on their way and 4 CTAs an SM, 8 choices of
// 7168 180 (3 CTAs 193, 5 198); fewer choices four rows and 6, 2 of 5120 59 (63 with 4, 84 with eight rows).  FP32 8 CTAs, 2
// of 5120 100 (104 to 118 with four rows and 5 or 8).
template <class T, bool kVec, int kMost>
__global__ void __launch_bounds__(256, !kVec ? 4 : sizeof(T) == 4 ? 8 : kMost == 8 ? 4 : 6) combine_kernel(const RowArgs a, int parts)
{
    using P = Piece<T, kVec>;
    __shared__ Choices choices;
    const int64_t t = blockIdx.x / parts;
    load_choices(choices, a, t);
    int64_t part = blockIdx.x % parts;
    for (int64_t c = first_of<T, kVec>(part); c < a.cols; c = first_of<T, kVec>(part += parts)) {
        const T* rows = static_cast<const T*>(a.rows) + c;
        const int64_t left = a.cols - c;
        float sum[P::kN] = {};
        P add;
        if (a.x) add.load(static_cast<const T*>(a.x) + t * a.ld_x + c, left);
        by_parts<kMost>(a.top, [&](auto how_many, int j0) {
            constexpr int many = decltype(how_many)::value;
            P v[many];
            load_rows(v, choices, j0, rows, a.ld_rows, left);
#pragma unroll
            for (int j = 0; j < many; ++j) {
                if (choices.row[j0 + j] < 0) continue;
                float f[P::kN];
                v[j].get(f);
                const float w = choices.weight[j0 + j];
#pragma unroll
                for (int i = 0; i < P::kN; ++i) sum[i] = __fmaf_rn(w, f[i], sum[i]);
            }
        });
        if (a.x) {  // the residual joins last
            float f[P::kN];
            add.get(f);
#pragma unroll
            for (int i = 0; i < P::kN; ++i) sum[i] += f[i];
        }
        P::store(static_cast<T*>(a.y) + t * a.ld_y + c, sum, left);
    }
}

// A CTA a token.  As above: BF16, 8192 tokens, 8 choices of 7168 300 us with 3 CTAs an SM (2: 326, 4: 318), 2 of 5120
// 87 with four rows and 5 (96 with 4, 115 with eight rows and 3).
template <class T, bool kVec, int kMost>
__global__ void __launch_bounds__(256, !kVec ? 4 : kMost == 8 ? 3 : 5) combine_grad_kernel(const RowArgs a)
{
    using P = Piece<T, kVec>;
    __shared__ float sums[8][8];
    __shared__ Choices choices;
    const int64_t t = blockIdx.x;
    load_choices(choices, a, t);
    const T* dy = static_cast<const T*>(a.y) + t * a.ld_y;
    T* out = static_cast<T*>(a.out);
    by_parts<kMost>(a.top, [&](auto how_many, int j0) {
        constexpr int many = decltype(how_many)::value;
        float dot[many];
#pragma unroll
        for (int j = 0; j < many; ++j) dot[j] = 0.0f;
        int64_t part = 0;
        for (int64_t c = first_of<T, kVec>(0); c < a.cols; c = first_of<T, kVec>(++part)) {
            const int64_t left = a.cols - c;
            P v[many], raw;
            raw.load(dy + c, left);
            load_rows(v, choices, j0, static_cast<const T*>(a.rows) + c, a.ld_rows, left);
            float d[P::kN];
            raw.get(d);
#pragma unroll
            for (int j = 0; j < many; ++j) {
                const int32_t r = choices.row[j0 + j];
                if (r < 0) continue;
                const float w = choices.weight[j0 + j];
                float f[P::kN], g[P::kN];
                v[j].get(f);
#pragma unroll
                for (int i = 0; i < P::kN; ++i) {
                    if (kVec || (int)blockDim.x * i < left) dot[j] = __fmaf_rn(d[i], f[i], dot[j]);
                    g[i] = w * d[i];
                }
                P::store(out + r * a.ld_out + c, g, left);
            }
        }
#pragma unroll
        for (int j = 0; j < many; ++j)
#pragma unroll
            for (int o = 16; o; o >>= 1) dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
        __syncthreads();
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int j = 0; j < many; ++j) sums[threadIdx.x >> 5][j] = dot[j];
        __syncthreads();
        if (threadIdx.x < many) {
            float s = 0.0f;
            for (int q = 0; q < (int)(blockDim.x >> 5); ++q) s += sums[q][threadIdx.x];
            a.d_weight[t * a.top + j0 + threadIdx.x] = s;
        }
    });
    clear_rest(a, out, a.ld_out, a.cols);
}

int check(int64_t tokens, int64_t top, int64_t experts)
{
    if (tokens < 0 || top < 1 || top > kMostTop || experts < 1 || experts > kMostExperts || tokens > kMaxRows / top)
        return FP8Z1_EINVAL;
    return FP8Z1_OK;
}
int check(int64_t tokens, int64_t top, int64_t experts, int64_t dim, int32_t type)
{
    if (dim < 1 || dim > (int64_t)1 << 23 || (type != FP8Z1_F32 && type != FP8Z1_BF16)) return FP8Z1_EINVAL;
    return check(tokens, top, experts);
}

// As many as go round a row's vectors evenly, at most 256.
unsigned threads_for(int64_t vectors)
{
    const int64_t rounds = std::max<int64_t>(1, ceil_div(vectors, 256));
    return (unsigned)(std::max<int64_t>(1, ceil_div(vectors, rounds * 32)) * 32);
}

template <class V>
int launch_dispatch(RowArgs a, int64_t bytes, int64_t size, cudaStream_t s)
{
    const int64_t n = (int64_t)sizeof(V);
    a.cols = bytes / n;
    a.ld_x = a.ld_x * size / n;
    a.ld_out = a.ld_out * size / n;
    count_launch();
    dispatch_kernel<V><<<(unsigned)a.tokens, threads_for(ceil_div(a.cols, 4)), 0, s>>>(a);
    return launch_status();
}

template <class T, bool kVec, int kMost>
int launch_combine(const RowArgs& a, cudaStream_t s)
{
    constexpr int kN = Piece<T, kVec>::kN;
    const unsigned threads = threads_for(ceil_div(a.cols, kN));
    // few tokens: their columns over more CTAs
    const int64_t most = ceil_div(a.cols, (int64_t)threads * kN);
    const int parts = (int)std::max<int64_t>(1, std::min(most, 4 * kSms / a.tokens));
    count_launch();
    combine_kernel<T, kVec, kVec && sizeof(T) == 4 ? 8 : kMost><<<(unsigned)(a.tokens * parts), threads, 0, s>>>(a, parts);
    return launch_status();
}

template <class T, bool kVec, int kMost>
int launch_combine_grad(const RowArgs& a, cudaStream_t s)
{
    count_launch();
    combine_grad_kernel<T, kVec, kMost><<<(unsigned)a.tokens, threads_for(ceil_div(a.cols, Piece<T, kVec>::kN)), 0, s>>>(a);
    return launch_status();
}

// Calls f for a call's type, pieces and rows on their way at once.
template <class F>
int by_type(int32_t type, bool vec, int64_t top, F f)
{
    const auto of = [&](auto t) {
        using B = std::bool_constant<true>;
        if (!vec) return f(t, std::bool_constant<false>(), std::integral_constant<int, 4>());
        return top >= 8 ? f(t, B(), std::integral_constant<int, 8>()) : f(t, B(), std::integral_constant<int, 4>());
    };
    return type == FP8Z1_F32 ? of(float()) : of(bf16());
}

bool fits(const void* p, int64_t ld, int64_t size, int64_t bytes) { return !p || (aligned(p, bytes) && ld * size % bytes == 0); }

}  // namespace
}  // namespace fp8z1

using namespace fp8z1;

extern "C" int fp8z1_route(const void* ids, int32_t id_bytes, int64_t tokens, int64_t top, int64_t experts,
                           int32_t* offsets, int32_t* place, void* stream)
{
    int st = check(tokens, top, experts);
    if (st != FP8Z1_OK) return st;
    const int64_t n = tokens * top;
    if (!offsets || (n && (!ids || !place)) || (id_bytes != 4 && id_bytes != 8)) return FP8Z1_EINVAL;
    if (!aligned(ids, id_bytes) || !aligned(offsets, 4) || !aligned(place, 4)) return FP8Z1_EALIGN;
    {
        // long runs of choices are read twice, and ranks wait in `place` between
        const Area in = dense(n ? ids : nullptr, n * id_bytes), at = dense(n ? place : nullptr, n * 4), ends = dense(offsets, (experts + 1) * 4);
        if (overlap(in, at) || overlap(in, ends) || overlap(at, ends)) return FP8Z1_EINVAL;
    }
    NvtxRange range("fp8z1_route");
    // one CTA up to 4096 choices (a cluster's barriers cost as much as four steps), then up to 8 CTAs of 32 warps
    const int ctas = (int)std::min<int64_t>(8, std::max<int64_t>(1, ceil_div(n, 4096)));
    const int warps = ctas > 1 ? 32 : (int)std::min<int64_t>(32, std::max<int64_t>(4, ceil_div(n, 64)));
    SortArgs a = {ids, n, (int32_t)experts, 0, offsets, place};
    a.per_warp = (int32_t)(ceil_div(ceil_div(n, (int64_t)ctas * warps), 32) * 32);
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at[1] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    c.gridDim = dim3((unsigned)ctas);
    c.blockDim = dim3((unsigned)warps * 32);
    c.dynamicSmemBytes = (size_t)(warps + 1) * experts * 4;
    c.stream = static_cast<cudaStream_t>(stream);
    c.attrs = at;
    c.numAttrs = 1;
    constexpr int kMostSmem = 33 * kMostExperts * 4;
    if (!(id_bytes == 4 ? allow_smem<sort_kernel<int32_t>>(kMostSmem) : allow_smem<sort_kernel<int64_t>>(kMostSmem)))
        return FP8Z1_ECUDA;
    count_launch();
    if ((id_bytes == 4 ? cudaLaunchKernelEx(&c, sort_kernel<int32_t>, a) : cudaLaunchKernelEx(&c, sort_kernel<int64_t>, a)) !=
        cudaSuccess) {
        cudaGetLastError();
        return FP8Z1_ECUDA;
    }
    return launch_status();
}

extern "C" int fp8z1_dispatch(int64_t tokens, int64_t top, int64_t experts, int64_t dim, const void* x, int32_t type,
                              int64_t ld_x, const int32_t* offsets, const int32_t* place, void* rows, int64_t ld_rows,
                              void* stream)
{
    int st = check(tokens, top, experts, dim, type);
    if (st != FP8Z1_OK) return st;
    if (tokens == 0) return FP8Z1_OK;
    if (!x || !offsets || !place || !rows || ld_x < dim || ld_rows < dim) return FP8Z1_EINVAL;
    const int64_t size = type == FP8Z1_F32 ? 4 : 2, bytes = dim * size;
    if (!aligned(x, size) || !aligned(rows, size) || !aligned(offsets, 4) || !aligned(place, 4)) return FP8Z1_EALIGN;
    // tokens read what others have written
    const Area to = {rows, tokens * top, bytes, ld_rows * size};
    if (overlap(to, Area{x, tokens, bytes, ld_x * size}) || overlap(to, dense(offsets, (experts + 1) * 4)) ||
        overlap(to, dense(place, tokens * top * 4)))
        return FP8Z1_EINVAL;
    NvtxRange range("fp8z1_dispatch");
    RowArgs a = {};
    a.tokens = tokens;
    a.n = tokens * top;
    a.top = (int32_t)top;
    a.experts = (int32_t)experts;
    a.offsets = offsets;
    a.place = place;
    a.x = x;
    a.ld_x = ld_x;
    a.out = rows;
    a.ld_out = ld_rows;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto all = [&](int64_t b) { return bytes % b == 0 && fits(x, ld_x, size, b) && fits(rows, ld_rows, size, b); };
    if (all(16)) return launch_dispatch<uint4>(a, bytes, size, s);
    if (all(4)) return launch_dispatch<uint32_t>(a, bytes, size, s);
    return launch_dispatch<uint16_t>(a, bytes, size, s);
}

extern "C" int fp8z1_combine(int64_t tokens, int64_t top, int64_t dim, const void* rows, int32_t type, int64_t ld_rows,
                             const int32_t* place, const float* weight, const void* residual, int64_t ld_residual,
                             void* y, int64_t ld_y, void* stream)
{
    int st = check(tokens, top, 1, dim, type);
    if (st != FP8Z1_OK) return st;
    if (tokens == 0) return FP8Z1_OK;
    if (!rows || !place || !y || ld_rows < dim || (residual && ld_residual < dim) || ld_y < dim) return FP8Z1_EINVAL;
    const int64_t size = type == FP8Z1_F32 ? 4 : 2;
    if (!aligned(rows, size) || !aligned(residual, size) || !aligned(y, size) || !aligned(place, 4) || !aligned(weight, 4))
        return FP8Z1_EALIGN;
    // tokens read what others have written; a token its own residual
    const Area to = {y, tokens, dim * size, ld_y * size};
    if (overlap(to, Area{rows, tokens * top, dim * size, ld_rows * size}) || overlap(to, dense(place, tokens * top * 4)) ||
        overlap(to, dense(weight, tokens * top * 4)) || !same_or_apart(to, Area{residual, tokens, dim * size, ld_residual * size}))
        return FP8Z1_EINVAL;
    NvtxRange range("fp8z1_combine");
    RowArgs a = {};
    a.tokens = tokens;
    a.n = tokens * top;
    a.top = (int32_t)top;
    a.cols = dim;
    a.place = place;
    a.weight = weight;
    a.x = residual;
    a.ld_x = ld_residual;
    a.rows = rows;
    a.ld_rows = ld_rows;
    a.y = y;
    a.ld_y = ld_y;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec = dim * size % 16 == 0 && fits(rows, ld_rows, size, 16) && fits(residual, ld_residual, size, 16) &&
                     fits(y, ld_y, size, 16);
    return by_type(type, vec, top, [&](auto t, auto v, auto n) { return launch_combine<decltype(t), v(), n()>(a, s); });
}

extern "C" int fp8z1_combine_grad(int64_t tokens, int64_t top, int64_t experts, int64_t dim, const void* dy, int32_t type,
                                  int64_t ld_dy, const void* rows, int64_t ld_rows, const int32_t* offsets,
                                  const int32_t* place, const float* weight, void* d_rows, int64_t ld_d, float* d_weight,
                                  void* stream)
{
    int st = check(tokens, top, experts, dim, type);
    if (st != FP8Z1_OK) return st;
    if (tokens == 0) return FP8Z1_OK;
    if (!dy || !rows || !offsets || !place || !weight || !d_rows || !d_weight || ld_dy < dim || ld_rows < dim || ld_d < dim)
        return FP8Z1_EINVAL;
    const int64_t size = type == FP8Z1_F32 ? 4 : 2;
    if (!aligned(dy, size) || !aligned(rows, size) || !aligned(d_rows, size) || !aligned(offsets, 4) || !aligned(place, 4) ||
        !aligned(weight, 4) || !aligned(d_weight, 4))
        return FP8Z1_EALIGN;
    // tokens read what others have written; a choice its own row and weight
    const Area to = {d_rows, tokens * top, dim * size, ld_d * size}, got = {rows, tokens * top, dim * size, ld_rows * size},
               from = {dy, tokens, dim * size, ld_dy * size}, at = dense(place, tokens * top * 4), w = dense(weight, tokens * top * 4),
               to_w = dense(d_weight, tokens * top * 4), ends = dense(offsets, (experts + 1) * 4);
    if (overlap(to, from) || !same_or_apart(to, got) || overlap(to, at) || overlap(to, w) || overlap(to, to_w) || overlap(to, ends) ||
        overlap(to_w, from) || overlap(to_w, got) || overlap(to_w, at) || overlap(to_w, ends) || !same_or_apart(to_w, w))
        return FP8Z1_EINVAL;
    NvtxRange range("fp8z1_combine_grad");
    RowArgs a = {};
    a.tokens = tokens;
    a.n = tokens * top;
    a.top = (int32_t)top;
    a.experts = (int32_t)experts;
    a.cols = dim;
    a.offsets = offsets;
    a.place = place;
    a.weight = weight;
    a.rows = rows;
    a.ld_rows = ld_rows;
    a.y = const_cast<void*>(dy);
    a.ld_y = ld_dy;
    a.out = d_rows;
    a.ld_out = ld_d;
    a.d_weight = d_weight;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool vec = dim * size % 16 == 0 && fits(dy, ld_dy, size, 16) && fits(rows, ld_rows, size, 16) &&
                     fits(d_rows, ld_d, size, 16);
    return by_type(type, vec, top, [&](auto t, auto v, auto n) { return launch_combine_grad<decltype(t), v(), n()>(a, s); });
}
