// Distillation loss against a teacher's top logits, and its gradient.
//
//   q_j = exp2((z_j - m) k) / sum,  k = log2(e) / tau,  m the row's maximum,
//   loss = tau^2 sum_k p_k (log p_k - log q_{id_k}),
//   dz_j = w tau (q_j - sum of the p listed for j).
//
// Bound by memory: the logits are read from it once and the gradient written
// once.  A row is read twice, for its maximum and sum and, backwards, for the
// gradient; the second time it comes from L2, and a long row's first 92 KB from
// shared memory.  4096 rows of 131072 BF16 logits take 361 us with the gradient
// (5.9 TB/s) and 164 without (6.5).
//
// A row belongs to a CTA of 2 to 16 warps, or to a cluster of up to 8 of them,
// each with a slice.  A thread has eight vectors of 16 bytes on their way and
// joins them, four at a time, to a running maximum and the sum of exponentials in
// reference to it; the warps' pairs are joined through distributed shared memory
// in a fixed order, so results repeat bit for bit.  One warp of a CTA has the teacher's
// entries, a long chain of small steps beside the others' loads: the softmax,
// the student's logits behind the ids, repeated ids added up; then the loss and,
// over the dense gradient w tau q_j, the listed elements.
#include <cooperative_groups.h>

#include <algorithm>

#include "ops_common.cuh"

namespace {

using namespace fp8z1;
namespace cg = cooperative_groups;

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <class T>
struct Vec {
    static constexpr int n = 16 / sizeof(T);
    uint4 v;
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    // the largest element (NaN ignored)
    __device__ __forceinline__ float largest() const
    {
        if constexpr (sizeof(T) == 4) return fmaxf(fmaxf(get(0), get(1)), fmaxf(get(2), get(3)));
        const auto two = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
        const __nv_bfloat162 m = __hmax2(__hmax2(two(v.x), two(v.y)), __hmax2(two(v.z), two(v.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
};

template <class T>
__device__ __forceinline__ uint4 pack(const float (&f)[Vec<T>::n])
{
    if constexpr (sizeof(T) == 4)
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 two = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&two);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// 16 bytes of a row from element `at` (a multiple of the vector from the
// aligned address below the row's start, so `at` may be negative); elements
// outside [0, n) read as -inf and are not touched.
template <class T>
__device__ __forceinline__ uint4 load_vec(const T* z, int64_t at, int64_t n)
{
    constexpr int kN = Vec<T>::n;
    if (at >= 0 && at + kN <= n) return __ldcs(reinterpret_cast<const uint4*>(z + at));
    float f[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i) f[i] = at + i >= 0 && at + i < n ? to_float(z[at + i]) : -INFINITY;
    return pack<T>(f);
}

template <class T>
__device__ __forceinline__ void store_vec(T* z, int64_t at, int64_t n, bool whole, const float (&f)[Vec<T>::n])
{
    constexpr int kN = Vec<T>::n;
    if (whole && at >= 0 && at + kN <= n) {
        __stcs(reinterpret_cast<uint4*>(z + at), pack<T>(f));
        return;
    }
#pragma unroll
    for (int i = 0; i < kN; ++i)
        if (at + i >= 0 && at + i < n) z[at + i] = from_float<T>(f[i]);
}

// Exponents are taken in the log2 domain as fma(z, k, -mk), one rounding of the
// whole, with mk the rounded m k: the reference is mk / k, and what it differs from
// m by, rest() in the log2 domain, is the same for all that is added up and comes
// off the sum's logarithm at the end.  From |m k| = 2^22 on (a row, or a thread's part
// of one, of nothing but a mask's value) the rest could leave FP32's exponents, and
// (z - m) k is taken, whose reference is m itself.
struct Base {  // of a launch
    float k, limit;
    __device__ __forceinline__ explicit Base(float tau)
    {
        k = 1.4426950408889634f / tau;
        limit = 4194304.0f / k;
    }
};
struct Scale : Base {
    float m, mk;
    bool plain;
    __device__ __forceinline__ Scale(const Base& b, float top) : Base(b)
    {
        m = top == -INFINITY ? 0.0f : top;
        plain = fabsf(m) <= limit;
        mk = m * k;
    }
    __device__ __forceinline__ float of(float z) const
    {
        return exp2_fast(plain ? fmaf(z, k, -mk) : (z - m) * k);
    }
    __device__ __forceinline__ float rest() const { return plain ? fmaf(m, k, -mk) : 0.0f; }
};

// A maximum and the sum of the exponentials in reference to it.
struct __align__(8) Sum {
    float m, s;
};
// `part`'s sum in reference to another, no smaller maximum; 0 for an empty part
__device__ __forceinline__ float in_reference(const Sum& part, const Scale& to)
{
    if (to.plain && fabsf(part.m) <= to.limit) return part.s * exp2_fast(part.m * to.k - to.mk);
    if (part.m == -INFINITY) return part.s * 0.0f;
    const Scale from(to, part.m);
    return part.s * exp2_fast((part.m - to.m) * to.k + (to.rest() - from.rest()));
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v)
{
    float m;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

template <class T>
struct Args {
    const T* logits;
    int64_t ld, rows, vocab;
    const int32_t* ids;
    const float* teacher;
    int32_t top;
    float tau;
    const float* weight;
    float* loss;
    T* dlogits;
    int64_t ld_d;
    int64_t slice;     // vectors of a CTA
    int32_t kept;      // the first batches of a slice that stay in shared memory for the gradient
};

// A CTA's part of a row.  Vector v of the row holds elements v kN - shift ..;
// the CTA has vectors [rank slice, (rank + 1) slice), elements [first, end).
template <class T>
struct Slice {
    const T* z;
    T* dz;
    int64_t first, end;
    bool same;  // the gradient's row starts alike
    __device__ __forceinline__ Slice(const Args<T>& a, int64_t r, int rank)
    {
        z = a.logits + r * a.ld;
        dz = a.dlogits ? a.dlogits + r * a.ld_d : nullptr;
        const int shift = (int)(reinterpret_cast<uintptr_t>(z) % 16 / sizeof(T));
        same = dz && reinterpret_cast<uintptr_t>(dz) % 16 == reinterpret_cast<uintptr_t>(z) % 16;
        first = (int64_t)rank * a.slice * Vec<T>::n - shift;
        end = min(first + a.slice * Vec<T>::n, a.vocab);
    }
};

// The teacher's entries of one row, in shared memory.
struct Lists {
    // All of them: p (0: absent) and the student's logit.
    float *p, *zk;
    // Those of the CTA's slice (first all of them): id, p of all an id's repeats at the first one and -1 at the
    // others, the student's logit.
    int32_t* id;
    float *own_p, *own_z;
};
__host__ __device__ __forceinline__ int64_t list_entries(int64_t top) { return (top + 3) / 4 * 4; }
constexpr int kListBytes = 20;  // an entry
__device__ __forceinline__ Lists lists_at(uint8_t* smem, int top)
{
    const int n = (int)list_entries(top);
    float* f = reinterpret_cast<float*>(smem);
    return Lists{f, f + n, reinterpret_cast<int32_t*>(f + 2 * n), f + 3 * n, f + 4 * n};
}

struct Entries {
    float p_logp;  // the sum of p log p
    int32_t any;
    int32_t own;   // entries of the CTA's slice
};

// One warp fills the lists of row r, for the slice [first, end).
template <class T>
__device__ __forceinline__ Entries fill_lists(const Args<T>& a, int64_t r, const T* z, int64_t first, int64_t end,
                                              const Lists& l)
{
    const int lane = threadIdx.x & 31;
    constexpr float kLog2e = 1.4426950408889634f;
    float top = -INFINITY;
    bool any = false;
#pragma unroll 4
    for (int i = lane; i < a.top; i += 32) {
        const int32_t j = __ldg(a.ids + r * a.top + i);
        const float t = __ldg(a.teacher + r * a.top + i);
        const bool there = j >= 0 && j < a.vocab && t != -INFINITY;
        l.id[i] = there ? j : -1;
        l.p[i] = there ? t : -INFINITY;
        l.zk[i] = there ? to_float(z[j]) : 0.0f;
        any |= there;
        top = fmaxf(top, l.p[i]);
    }
    Entries e = {0.0f, __any_sync(0xffffffffu, any), 0};
    if (!e.any) return e;
    top = warp_max(top);
    float mass = 0.0f;
    for (int i = lane; i < a.top; i += 32)
        if (l.id[i] >= 0) {
            // the difference first: a mask's lowest value by a temperature below 1 would be -inf
            const float t = (l.p[i] - top) / a.tau;
            l.p[i] = t;
            mass += exp2_fast(t * kLog2e);
        }
    mass = warp_sum(mass);
    const float log_mass = logf(mass), by = 1.0f / mass;
    for (int i0 = 0; i0 < a.top; i0 += 32) {
        const int i = i0 + lane;
        int32_t j = -1;
        float p = 0.0f, zk = 0.0f;
        if (i < a.top && l.id[i] >= 0) {
            j = l.id[i];
            zk = l.zk[i];
            const float logp = l.p[i] - log_mass;
            p = exp2_fast(l.p[i] * kLog2e) * by;
            // an entry too small to count: 0 log 0 = 0, whatever the student's logit
            if (p != 0.0f) e.p_logp = fmaf(p, logp, e.p_logp);
        }
        if (i < a.top) l.p[i] = p;
        // the slice's entries move to the front of theirs
        const bool mine = j >= 0 && j >= first && j < end;
        const unsigned group = __ballot_sync(0xffffffffu, mine);
        if (mine) {
            const int at = e.own + __popc(group & ((1u << lane) - 1));
            l.id[at] = j;
            l.own_p[at] = p;
            l.own_z[at] = zk;
        }
        e.own += __popc(group);
        __syncwarp();
    }
    e.p_logp = warp_sum(e.p_logp);
    if (e.own + lane < list_entries(e.own)) l.id[e.own + lane] = -1;
    __syncwarp();
    // repeats of an id, at its first entry
    for (int i0 = 0; i0 < e.own; i0 += 32) {
        const int i = i0 + lane;
        const int32_t j = i < e.own ? l.id[i] : -2;
        int same = 0, before = 0;
        const int4* ids = reinterpret_cast<const int4*>(l.id);
#pragma unroll 2
        for (int o = 0; o < e.own; o += 4) {
            const int4 q = ids[o >> 2];
            const int hits = (q.x == j) + (q.y == j) + (q.z == j) + (q.w == j);
            same += hits;
            // entries before i: whole groups of 4, and i's own group up to i
            before += o + 4 <= i ? hits
                                 : o > i ? 0 : (q.x == j && o < i) + (q.y == j && o + 1 < i) + (q.z == j && o + 2 < i);
        }
        float sum = i < e.own ? l.own_p[i] : 0.0f;
        if (same > 1 && before == 0) {
            sum = 0.0f;
            for (int o = i; o < e.own; ++o)  // its repeats come later; their p is not read again after this group
                if (l.id[o] == j) sum += l.own_p[o];
        }
        __syncwarp();
        if (i < e.own) l.own_p[i] = before == 0 ? sum : -1.0f;
        __syncwarp();
    }
    return e;
}

// The loss of a row of reference `sc` and sum `total`, by one warp:
//   log p - log q = log p - (z - m) / tau + log (total / 2^rest), and the p add up to 1.
template <class T>
__device__ __forceinline__ void write_loss(const Args<T>& a, int64_t r, const Lists& l, const Entries& e, const Scale& sc,
                                           float total)
{
    float pz = 0.0f;
    if (e.any)
        for (int i = threadIdx.x & 31; i < a.top; i += 32)
            if (l.p[i] != 0.0f) pz = fmaf(l.p[i], l.zk[i] - sc.m, pz);
    pz = warp_sum(pz);
    // a row of -inf alone has q = 0: its log q is z = -inf, not -inf - -inf
    const float log_total = total == 0.0f ? 0.0f : fmaf(sc.rest(), -0.6931471805599453f, logf(total));
    if ((threadIdx.x & 31) == 0) a.loss[r] = e.any ? a.tau * (a.tau * (e.p_logp + log_total) - pz) : 0.0f;
}

// The listed elements of a slice, over its dense gradient, by one warp.
template <class T>
__device__ __forceinline__ void write_listed(const Lists& l, int own, T* dz, const Scale& sc, float q, float by)
{
    for (int i = threadIdx.x & 31; i < own; i += 32)
        if (!(l.own_p[i] < 0.0f)) dz[l.id[i]] = from_float<T>(sc.of(l.own_z[i]) * q - l.own_p[i] * by);
}

__device__ __forceinline__ float inverse(float total)
{
    return total > 0.0f ? 1.0f / total : total;  // 0 and NaN stay so
}

// Maximum and sum of kHold vectors, joined to `mine`.
template <class T, int kHold>
__device__ __forceinline__ void add_vecs(const Vec<T> (&x)[kHold], const Base& k, Sum& mine)
{
    float m = x[0].largest();
#pragma unroll
    for (int j = 1; j < kHold; ++j) m = fmaxf(m, x[j].largest());
    m = fmaxf(m, mine.m);
    const Scale sc(k, m);
    float s[2] = {in_reference(mine, sc), 0.0f};
    if (sc.plain) {
#pragma unroll
        for (int j = 0; j < kHold; ++j)
#pragma unroll
            for (int i = 0; i < Vec<T>::n; ++i) s[i & 1] += exp2_fast(fmaf(x[j].get(i), sc.k, -sc.mk));
    } else {
#pragma unroll
        for (int j = 0; j < kHold; ++j)
#pragma unroll
            for (int i = 0; i < Vec<T>::n; ++i) s[i & 1] += exp2_fast((x[j].get(i) - sc.m) * sc.k);
    }
    mine = Sum{m, s[0] + s[1]};
}

// One vector, any elements of it.
template <class T>
__device__ __forceinline__ void add_vec(const Vec<T>& x, const Base& k, Sum& mine)
{
    const float m = fmaxf(mine.m, x.largest());
    const Scale sc(k, m);
    float s = in_reference(mine, sc);
#pragma unroll
    for (int i = 0; i < Vec<T>::n; ++i) s += sc.of(x.get(i));
    mine = Sum{m, s};
}

// The sum over a warp's lanes.
__device__ __forceinline__ Sum warp_join(const Sum& mine, const Base& k)
{
    const float m = warp_max(mine.m);
    return Sum{m, warp_sum(in_reference(mine, Scale(k, m)))};
}
// The row's, from the `n` pairs its cluster's warps left; every lane gets it.
__device__ __forceinline__ Sum row_join(const Sum* parts, int n, const Base& k)
{
    const int lane = threadIdx.x & 31;
    float top = -INFINITY;
    for (int i = lane; i < n; i += 32) top = fmaxf(top, parts[i].m);
    const Scale sc(k, warp_max(top));
    float s = 0.0f;
    for (int i = lane; i < n; i += 32) s += in_reference(parts[i], sc);
    return Sum{sc.m, warp_sum(s)};
}

template <class T>
__device__ __forceinline__ void dense(const Vec<T>& x, const Scale& sc, float q, float (&f)[Vec<T>::n])
{
#pragma unroll
    for (int i = 0; i < Vec<T>::n; ++i) f[i] = sc.of(x.get(i)) * q;
}

constexpr int kHold = 4;  // vectors a thread joins at once

// kHold vectors a thread apart, from p on (or back, with a negative step).
template <class T, int kStep>
__device__ __forceinline__ void load_some(Vec<T> (&x)[kHold], const T* p)
{
#pragma unroll
    for (int j = 0; j < kHold; ++j) x[j].v = *reinterpret_cast<const uint4*>(p + j * kStep * Vec<T>::n);
}
template <class T, int kStep>
__device__ __forceinline__ void store_some(const Vec<T> (&x)[kHold], T* p, const Scale& sc, float q)
{
    constexpr int kN = Vec<T>::n;
#pragma unroll
    for (int j = 0; j < kHold; ++j) {
        float f[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) f[i] = exp2_fast(fmaf(x[j].get(i), sc.k, -sc.mk)) * q;
        __stcs(reinterpret_cast<uint4*>(p + j * kStep * kN), pack<T>(f));
    }
}

// kKeep: whether the first batches of a slice stay in shared memory.
template <class T, int kThreads, bool kKeep>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) row_kernel(const Args<T> a)
{
    constexpr int kN = Vec<T>::n, kReaders = kThreads - 32, kWarps = kReaders / 32;
    constexpr int64_t kBatch = (int64_t)kHold * kReaders * kN;  // elements
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ Sum parts[8 * kWarps];
    __shared__ Entries entries;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Base k(a.tau);
    const Lists l = lists_at(smem, a.top);
    const int64_t r = blockIdx.x / ranks;
    const Slice<T> s(a, r, rank);
    const float w = a.weight ? __ldg(a.weight + r) : 1.0f;
    auto clear = [&]() {
        const float zero[kN] = {};
        if (rank == 0 && tid == 0) a.loss[r] = 0.0f;
        if (s.dz)
            for (int64_t at = s.first + (int64_t)tid * kN; at < s.end; at += kThreads * kN)
                store_vec(s.dz, at, s.end, s.same, zero);
    };
    if (w == 0.0f) return clear();  // the same in every CTA of the cluster
    if (ranks > 1) cluster.sync();  // every CTA has started: the others may write to it
    // the slice's vectors [0, vecs), those inside the row whole [f0, f1): the others are the row's first and last
    const int vecs = s.end > s.first ? (int)((s.end - s.first + kN - 1) / kN) : 0;
    const int f0 = s.first < 0 ? 1 : 0, f1 = s.end > s.first ? (int)((s.end - s.first) / kN) : 0;
    const bool head = tid == 0 && f0 && vecs, tail = tid == 0 && f1 < vecs && (f1 || !f0);
    const int64_t tail_at = s.first + (int64_t)f1 * kN;
    // this thread's whole vectors: `share` of them, kReaders apart
    const int share = f1 - f0 > tid ? (f1 - f0 - 1 - tid) / kReaders + 1 : 0, batches = share / kHold;
    const T* const z0 = s.z + s.first + (int64_t)(f0 + tid) * kN;
    uint4* const kept = reinterpret_cast<uint4*>(smem + list_entries(a.top) * kListBytes) + tid;
    auto keep = [&](const Vec<T>(&v)[kHold], int b) {
        if constexpr (kKeep) {
            if (b >= a.kept) return;
#pragma unroll
            for (int j = 0; j < kHold; ++j) kept[(b * kHold + j) * kReaders] = v[j].v;
        }
    };
    auto again = [&](Vec<T>(&v)[kHold], int b, const T* p) {
        if constexpr (kKeep) {
            if (b < a.kept) {
#pragma unroll
                for (int j = 0; j < kHold; ++j) v[j].v = kept[(b * kHold + j) * kReaders];
                return;
            }
        }
        load_some<T, kReaders>(v, p);
    };
    if (warp == kWarps) {
        const Entries e = fill_lists(a, r, s.z, s.first, s.end, l);
        if (lane == 0) entries = e;
    } else {
        Sum mine = {-INFINITY, 0.0f};
        Vec<T> x[kHold], y[kHold];
        const T* p = z0;
        if (batches > 0) load_some<T, kReaders>(x, p);
        if (head) add_vec(Vec<T>{load_vec(s.z, s.first, s.end)}, k, mine);
        if (tail) add_vec(Vec<T>{load_vec(s.z, tail_at, s.end)}, k, mine);
        for (int b = 0; b < batches; b += 2, p += 2 * kBatch) {
            if (b + 1 < batches) load_some<T, kReaders>(y, p + kBatch);
            keep(x, b);
            add_vecs<T, kHold>(x, k, mine);
            if (b + 2 < batches) load_some<T, kReaders>(x, p + 2 * kBatch);
            if (b + 1 < batches) {
                keep(y, b + 1);
                add_vecs<T, kHold>(y, k, mine);
            }
        }
        // the last few
        p = z0 + batches * kBatch;
        const int left = share - batches * kHold;
#pragma unroll
        for (int j = 0; j < kHold - 1; ++j)
            if (j < left) x[j].v = *reinterpret_cast<const uint4*>(p + j * kReaders * kN);
#pragma unroll
        for (int j = 0; j < kHold - 1; ++j)
            if (j < left) add_vec(x[j], k, mine);
        mine = warp_join(mine, k);
        if (lane < ranks) *cluster.map_shared_rank(&parts[rank * kWarps + warp], lane) = mine;
    }
    // Every warp's pair is here, and every CTA has read the listed logits, which the gradient may overwrite.
    __syncwarp();
    cluster.sync();
    const Entries e = entries;
    if (!e.any) return clear();
    const Sum row = row_join(parts, ranks * kWarps, k);
    const Scale sc(k, row.m);
    const float q = inverse(row.s) * (w * a.tau);
    if (warp == kWarps && rank == 0) write_loss(a, r, l, e, sc, row.s);
    if (!s.dz) return;
    if (warp < kWarps) {
        float f[kN];
        if (s.same && sc.plain) {
            // backwards: the vectors read last are the likeliest to be in L2 still
            T* const d0 = s.dz + s.first + (int64_t)(f0 + tid) * kN;
            for (int v = share - 1; v >= batches * kHold; --v) {
                const Vec<T> x{*reinterpret_cast<const uint4*>(z0 + (int64_t)v * kReaders * kN)};
#pragma unroll
                for (int i = 0; i < kN; ++i) f[i] = exp2_fast(fmaf(x.get(i), sc.k, -sc.mk)) * q;
                __stcs(reinterpret_cast<uint4*>(d0 + (int64_t)v * kReaders * kN), pack<T>(f));
            }
            Vec<T> x[kHold], y[kHold];
            const T* p = z0 + (batches - 1) * kBatch;
            T* o = d0 + (batches - 1) * kBatch;
            if (batches > 0) again(x, batches - 1, p);
            for (int b = batches; b > 0; b -= 2, p -= 2 * kBatch, o -= 2 * kBatch) {
                if (b > 1) again(y, b - 2, p - kBatch);
                store_some<T, kReaders>(x, o, sc, q);
                if (b > 2) again(x, b - 3, p - 2 * kBatch);
                if (b > 1) store_some<T, kReaders>(y, o - kBatch, sc, q);
            }
        } else {
            for (int v = f0 + tid; v < f1; v += kReaders) {
                const int64_t at = s.first + (int64_t)v * kN;
                dense(Vec<T>{*reinterpret_cast<const uint4*>(s.z + at)}, sc, q, f);
                store_vec(s.dz, at, s.end, s.same, f);
            }
        }
        if (head) {
            dense(Vec<T>{load_vec(s.z, s.first, s.end)}, sc, q, f);
            store_vec(s.dz, s.first, s.end, false, f);
        }
        if (tail) {
            dense(Vec<T>{load_vec(s.z, tail_at, s.end)}, sc, q, f);
            store_vec(s.dz, tail_at, s.end, false, f);
        }
    }
    __syncthreads();  // the dense gradient, before the listed elements of the slice
    if (warp == kWarps) write_listed(l, e.own, s.dz, sc, q, w * a.tau);
}

constexpr int kMostSmem = 112 * 1024;  // two CTAs of 512 threads an SM

template <auto kKernel, class T>
int launch_clusters(const Args<T>& a, int64_t clusters, int ranks, int threads, int64_t smem, cudaStream_t s)
{
    cudaLaunchConfig_t c = {};
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)ranks;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.gridDim = dim3((unsigned)(clusters * ranks));
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = (size_t)smem;
    c.stream = s;
    c.attrs = &at;
    c.numAttrs = ranks > 1;
    if (smem > 40 * 1024 && !allow_smem<kKernel>(kMostSmem)) return FP8Z1_ECUDA;
    count_launch();
    if (cudaLaunchKernelEx(&c, kKernel, a) != cudaSuccess) {
        cudaGetLastError();
        return FP8Z1_ECUDA;
    }
    return launch_status();
}

template <class T, int kThreads, bool kKeep = false>
int launch_rows(Args<T> a, int ranks, cudaStream_t s)
{
    constexpr int64_t kBatchBytes = (int64_t)kHold * (kThreads - 32) * 16;
    const int64_t lists = list_entries(a.top) * kListBytes;
    a.kept = kKeep ? (int32_t)std::min<int64_t>((kMostSmem - lists) / kBatchBytes, a.slice * 16 / kBatchBytes) : 0;
    // rows beyond the grid's reach go in further launches
    const int64_t most = (int64_t)1 << 24;
    const Args<T> all = a;
    for (int64_t r = 0; r < all.rows; r += most) {
        a.rows = all.rows - r < most ? all.rows - r : most;
        a.logits = all.logits + r * all.ld;
        a.ids = all.ids + r * all.top;
        a.teacher = all.teacher + r * all.top;
        a.weight = all.weight ? all.weight + r : nullptr;
        a.loss = all.loss + r;
        a.dlogits = all.dlogits ? all.dlogits + r * all.ld_d : nullptr;
        const int st = launch_clusters<row_kernel<T, kThreads, kKeep>>(a, a.rows, ranks, kThreads, lists + a.kept * kBatchBytes, s);
        if (st != FP8Z1_OK) return st;
    }
    return FP8Z1_OK;
}

template <class T>
int launch(Args<T> a, cudaStream_t s)
{
    constexpr int kN = Vec<T>::n;
    // the most vectors a row spans, whatever its alignment
    const int64_t vecs = ceil_div(a.vocab + kN - 1, kN);
    // few rows are spread over more CTAs, down to 16 KB slices, while that still leaves SMs idle
    int ranks = 1;
    while (ranks < 8 && a.rows * ranks * 2 <= kSms && vecs > ranks * 2 * 1024) ranks *= 2;
    a.slice = ceil_div(vecs, ranks);
    // A CTA's fixed chain of steps is about 7 us: short rows go to small CTAs, of which an SM holds many.  Long ones
    // to few: they are read again from L2, where eight 256 KB rows an SM would not fit.  At two, four and eight rows an
    // SM (CTAs of 512, 256 and 128 threads, nothing kept), BF16, 64 entries: 4096 rows of 131072 take 408, 450 and 479
    // us, of 65536 188, 204 and 230, of 32768 116, 100 and 108; 8192 rows of 16384 240, 154 and 118.  Rows of a few KB
    // are that chain alone: 65536 of 2048 take 470 us in CTAs of 128 threads, 331 in 64; 16384 of 8192 161 and 140 (120
    // and 132 with 8 entries).  The loss alone reads once, and four rows an SM do best (164 us for 131072, 173 at two).
    const int64_t bytes = a.slice * 16;
    if (bytes <= 24 * 1024 && a.rows * ranks > kSms * 8) return launch_rows<T, 64>(a, ranks, s);
    if (bytes <= 48 * 1024) return launch_rows<T, 128>(a, ranks, s);
    if (bytes <= 128 * 1024 || (!a.dlogits && bytes <= 1024 * 1024)) return launch_rows<T, 256>(a, ranks, s);
    // Long rows keep the first of their batches in shared memory, as many as leave room for the SM's other CTA: the
    // gradient reads them last, when a row's worth of every CTA and the gradient's lines have passed through L2.  Kept
    // and not, 4000 rows of BF16 logits took 223 and 221 us at 160 KB a row, 246 and 258 at 184, 286 and 319 at 216, 353
    // and 399 at 256; 1000 of FP32 64 and 62, 72 and 72, 80 and 87, 98 and 104.
    if (a.dlogits && bytes > 176 * 1024) return launch_rows<T, 512, true>(a, ranks, s);
    return launch_rows<T, 512>(a, ranks, s);
}

}  // namespace

extern "C" int fp8z1_distill(const void* logits, int32_t type, int64_t ld, int64_t rows, int64_t vocab,
                             const int32_t* teacher_ids, const float* teacher_logits, int64_t top,
                             float temperature, const float* row_weight, float* loss, void* dlogits, int64_t ld_d,
                             void* stream)
{
    if (rows < 0 || rows > kMaxRows || vocab < 1 || vocab >= (int64_t)1 << 31 || top < 1 ||
        top > FP8Z1_DISTILL_MAX_TOP || (type != FP8Z1_F32 && type != FP8Z1_BF16) || ld < vocab ||
        (dlogits && ld_d < vocab) || (dlogits && dlogits == logits && ld_d != ld) || !isfinite(temperature) ||
        temperature <= 0.0f)
        return FP8Z1_EINVAL;
    if (rows > 0 && (!logits || !teacher_ids || !teacher_logits || !loss)) return FP8Z1_EINVAL;
    const int esz = type == FP8Z1_F32 ? 4 : 2;
    if (!aligned(logits, esz) || !aligned(dlogits, esz) || !aligned(teacher_ids, 4) || !aligned(teacher_logits, 4) ||
        !aligned(row_weight, 4) || !aligned(loss, 4))
        return FP8Z1_EALIGN;
    if (rows == 0) return FP8Z1_OK;
    NvtxRange range("fp8z1_distill");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (type == FP8Z1_F32)
        return launch<float>({static_cast<const float*>(logits), ld, rows, vocab, teacher_ids, teacher_logits,
                              (int32_t)top, temperature, row_weight, loss, static_cast<float*>(dlogits), ld_d, 0}, s);
    return launch<__nv_bfloat16>({static_cast<const __nv_bfloat16*>(logits), ld, rows, vocab, teacher_ids,
                                  teacher_logits, (int32_t)top, temperature, row_weight, loss,
                                  static_cast<__nv_bfloat16*>(dlogits), ld_d, 0}, s);
}
