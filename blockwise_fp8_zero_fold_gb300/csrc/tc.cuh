// The sm_103a pieces the operators are built from: mbarriers,
// TMA tile copies, tcgen05 matrix products and tensor memory.
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace fp8z1 {
namespace tc {

__device__ __forceinline__ uint32_t smem_addr(const void* p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---- mbarriers -------------------------------------------------------------

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// how long one try may suspend its thread before it returns
constexpr uint32_t kSuspendNs = 20000;

__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity), "r"(kSuspendNs)
                 : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint64_t now_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

// Every wait ends: after kWaitNs, and kWaitTries of up to kSuspendNs each (the clock
// goes on while a process is paused or its context switched out, the tries do not), it
// gives up and returns false.  A warp that adds up then stores NaN for what it could
// not finish; the others drain their own copies, free tensor memory and return.
#if FP8Z1_CHECKED
constexpr uint64_t kWaitNs = 200000000ull;
constexpr int kWaitTries = 5000;
#else
constexpr uint64_t kWaitNs = 4000000000ull;
constexpr int kWaitTries = 100000;
#endif

__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity)
{
    if (bar_try(bar, parity)) return true;
    const uint64_t t0 = now_ns();
    for (int tries = 1;; ++tries) {
        if (bar_try(bar, parity)) return true;
        if (tries >= kWaitTries && tries % 64 == 0 && now_ns() - t0 > kWaitNs) return false;
    }
}

// The cluster address of this CTA's address `a` in the first CTA of its pair.
__device__ __forceinline__ uint32_t first_of_pair(uint32_t a)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
    return r;
}
// An arrival on a barrier at a cluster address, after this thread's tensor memory
// loads.  Its writes are not released (a release to the cluster would wait for
// every global store in flight).
__device__ __forceinline__ void bar_arrive_pair(uint32_t bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Every thread of the cluster's CTAs.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
    return r;
}

// The next of kSlots slots used in turn, and the parity of its use: a consumer
// waits for `phase` of "full", a producer for `phase ^ 1` of "empty" (which a new
// barrier has behind it).
template <int kSlots>
struct Turn {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next()
    {
        if (++slot == kSlots) {
            slot = 0;
            phase ^= 1;
        }
    }
};

// ---- TMA ----------------------------------------------------------------------

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// Tiles to this CTA's shared memory.
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

// To this CTA's shared memory, counted on a barrier of either CTA of a pair
// (`bar` is a cluster address, of first_of_pair).
__device__ __forceinline__ void load_3d_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            dst),
        "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void store_3d(const CUtensorMap* map, uint32_t src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

__device__ __forceinline__ void store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void store_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void store_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// this thread's shared memory writes, before a TMA copy reads them
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- tcgen05 -----------------------------------------------------------------------
//
// kGroup 1: a CTA multiplies 128 rows by up to 256 columns by itself.  kGroup 2:
// a pair of CTAs 256 rows by up to 256 columns; each holds 128 rows of the first
// operand, half the columns of the second and the sums of its rows, and the
// first CTA's thread issues for both.

// By one warp of the CTA (of each CTA).
template <int kGroup, int kCols>
__device__ __forceinline__ void tmem_alloc(uint32_t smem_out)
{
    if constexpr (kGroup == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_out), "n"(kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_out), "n"(kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}
template <int kGroup, int kCols>
__device__ __forceinline__ void tmem_free(uint32_t taddr)
{
    if constexpr (kGroup == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(kCols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "n"(kCols) : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrives on `bar` once every product this thread issued has finished.
__device__ __forceinline__ void commit(uint32_t bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// The same, of a pair's products, on the barriers at this offset of both its CTAs.
__device__ __forceinline__ void commit_pair(uint32_t bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
}

// Shared memory operand (of a pair: at the same offset in both CTAs), 128-byte
// swizzle (atoms of 8 rows x 128 bytes).
//   K-major (a row is 128 bytes of k): group_stride = bytes between groups of
//     8 rows of the M or N index; chunk_stride unused.
//   M/N-major (a row is 128 bytes of the M or N index): group_stride = bytes
//     between groups of 8 k; chunk_stride = bytes between 128-byte runs of it.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t group_stride, uint32_t chunk_stride)
{
    return (uint64_t)((addr & 0x3FFFF) >> 4) | (uint64_t)(chunk_stride >> 4) << 16 |
           (uint64_t)(group_stride >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction descriptor of m rows x n columns: FP32 sums, operand formats E4M3
// (f8f6f4) or F16 (f16), both encoded 0, the first operand E5M2 instead with
// `a_e5m2`; `mn_major` bits say which operands are M/N-major.
__host__ __device__ constexpr uint32_t instruction(int m, int n, bool a_mn_major, bool b_mn_major, bool a_e5m2 = false)
{
    return 1u << 4 | (a_e5m2 ? 1u << 7 : 0u) | (a_mn_major ? 1u << 15 : 0u) | (b_mn_major ? 1u << 16 : 0u) |
           (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

// By one CTA.
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}
// By a pair.
__device__ __forceinline__ void mma_f16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add)
{
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

// 16 columns of this warp's 32 lanes: r[i] = tensor memory (lane, column + i).
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
// The loads before this are done; `r` is one of them, so that no use of it moves up.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(r[i]));
}

template <int kRegs>
__device__ __forceinline__ void regs_less()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_more()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Two FP32 numbers in one register pair, and their multiply-add in one
// instruction.
__device__ __forceinline__ uint64_t pair(uint32_t a, uint32_t b)
{
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(a), "r"(b));
    return p;
}
__device__ __forceinline__ uint64_t pair(float a, float b) { return pair(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ float2 unpair(uint64_t p)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
    return f;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

}  // namespace tc
}  // namespace fp8z1
