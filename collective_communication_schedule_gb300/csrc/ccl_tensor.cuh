// Device-side building blocks of the tensor products: shared-memory barriers
// with bounded waits, TMA tile loads, tcgen05 matrix instructions on tensor
// memory, and the descriptors they take.  sm_103a only.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

namespace ccl {
namespace tensor {

__device__ __forceinline__ uint32_t smem_addr(const void* p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ unsigned long long now_ns()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Every kernel here may be launched before the one ahead of it on the stream
// has ended: each lets the next one in early, and touches no global memory
// before the previous one is complete.
__device__ __forceinline__ void let_next_in() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ------------------------------------------------------------- barriers
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
// the same shared-memory address in another threadblock of the cluster
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// arrive on a barrier of any threadblock of the cluster (address from cluster_addr)
__device__ __forceinline__ void bar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void store_cluster(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
// CLUSTER: also acquire what other threadblocks of the cluster released (dearer)
template <bool CLUSTER>
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    if (CLUSTER)
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.b32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(bar), "r"(parity)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.b32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok)
                     : "r"(bar), "r"(parity)
                     : "memory");
    return ok != 0;
}

// Limit of every wait: no step of a product takes anywhere near this long,
// so a wait that reaches it means a lost signal.
constexpr unsigned long long kWaitNs = 4000000000ull;
constexpr int kWaitSpins = 1 << 26;

template <bool CLUSTER>
__device__ __noinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, volatile int* failed)
{
    if (*failed) return false;
    // reading the timer is slow: not before the wait has proved long
    unsigned long long t0 = 0;
    for (int i = 1; i < kWaitSpins; ++i) {
        if (bar_try<CLUSTER>(bar, parity)) return true;
        if ((i & 255) == 0) {
            if (*failed) return false;
            const unsigned long long t = now_ns();
            if (!t0) t0 = t;
            if (t - t0 > kWaitNs) break;
        }
    }
    *failed = 1;
    return false;
}
// Bounded wait for the completion of the phase with this parity.  Gives up
// when the limit passes or another warp of the threadblock has given up.
template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* failed)
{
    if (bar_try<CLUSTER>(bar, parity)) return true;
    return bar_wait_long<CLUSTER>(bar, parity, failed);
}

// One lane of a converged warp.  The loops that issue copies and matrix
// instructions are run by the whole warp, so that the compiler keeps their
// addresses in uniform registers, and only the issue is left to one lane.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// ------------------------------------------------------------------ TMA
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];"
                 ::"r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// into this threadblock's memory, signalling a barrier of either threadblock of the pair
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
                 "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
                 "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// a tile from shared memory to global; parts outside the matrix are not written
__device__ __forceinline__ void tma_store(const CUtensorMap* map, uint32_t src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int LEFT>
__device__ __forceinline__ void tma_stores_read()   // all but the last LEFT stores of this thread have read their source
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void tma_prefetch(const CUtensorMap* map)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ------------------------------------------------------- tensor memory
// CG: threadblocks that work on one tile (1, or a pair on neighbouring SMs)
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols)
{
    if (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols)
{
    if (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void fence_after()
{
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_before()
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
// 32 lanes x 32 columns of 32-bit accumulators, one lane per thread
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t r[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void tmem_load16(uint32_t addr, uint32_t r[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15])
                 : "r"(addr)
                 : "memory");
}

// ------------------------------------------------- matrix instructions
// Shared-memory operand descriptor, 128-byte swizzle.  Operand tiles are
// stacks of 1024-byte atoms (8 rows of 128 bytes):
//   reduction-major (rows of 64 reduction elements): `stride` is the step
//     between atoms of 8 rows; `lead` is not used;
//   row-major (rows of 64 consecutive M or N elements, one row per reduction
//     index): `stride` is the step between atoms of 8 reduction indexes,
//     `lead` the step to the next 64 M or N elements.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, uint32_t lead, uint32_t stride)
{
    return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(stride >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// Instruction descriptor: f32 accumulators, both operands bf16 or both f16.
__host__ __device__ constexpr uint32_t mma_desc(bool bf16, bool a_mn, bool b_mn, int m, int n)
{
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
           ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    if (CG == 1)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
                     : "memory");
}
// the barrier (of both threadblocks of a pair) is arrived on once every matrix
// instruction this thread issued so far has finished
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar)
{
    if (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     ::"r"(bar), "h"((uint16_t)3)
                     : "memory");
}

// ------------------------------------------------------- named barriers
__device__ __forceinline__ void named_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void named_arrive(int id, int threads)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ------------------------------------------------------- element types
template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t u)
{
    if (BF) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if (BF)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float load1(const uint16_t* p, bool bf)
{
    const uint16_t u = *p;
    return bf ? __uint_as_float((uint32_t)u << 16) : __half2float(*reinterpret_cast<const __half*>(&u));
}
__device__ __forceinline__ void store1(uint16_t* p, float v, bool bf)
{
    if (bf) {
        const __nv_bfloat16 h = __float2bfloat16_rn(v);
        *p = *reinterpret_cast<const uint16_t*>(&h);
    } else {
        const __half h = __float2half_rn(v);
        *p = *reinterpret_cast<const uint16_t*>(&h);
    }
}
__device__ __forceinline__ void unpack8(const uint4& u, bool bf, float v[8])
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf ? unpack2<true>(w[i]) : unpack2<false>(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}
// the first n of 8 consecutive elements at a multiple of 16 bytes; the others
// read as 0 and are not touched
__device__ __forceinline__ void load8(const uint16_t* p, bool bf, int n, float v[8])
{
    if (n >= 8) {
        unpack8(*reinterpret_cast<const uint4*>(p), bf, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? load1(p + i, bf) : 0.f;
    }
}
__device__ __forceinline__ void store8(uint16_t* p, bool bf, int n, const float v[8])
{
    if (n >= 8) {
        uint4 u;
        if (bf)
            u = make_uint4(pack2<true>(v[0], v[1]), pack2<true>(v[2], v[3]), pack2<true>(v[4], v[5]),
                           pack2<true>(v[6], v[7]));
        else
            u = make_uint4(pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3]), pack2<false>(v[4], v[5]),
                           pack2<false>(v[6], v[7]));
        *reinterpret_cast<uint4*>(p) = u;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) store1(p + i, v[i], bf);
    }
}

// ---------------------------------------------------------- activations
// gelu is the tanh form, 0.5 z (1 + tanh u) = z sigmoid(2 u),
// u = sqrt(2/pi) (z + 0.044715 z^3); silu is z sigmoid(z).  In 32 bits.
enum { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_SILU = 3 };

// 1 / (1 + 2^(-x log2 e)): two approximate instructions, the exponential within 2^-22 and the reciprocal within 2^-23
__device__ __forceinline__ float sigmoid(float x)
{
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

__device__ __forceinline__ float activate(float z, int act)
{
    if (act == ACT_RELU) return z < 0.f ? 0.f : z;   // keeps NaN
    if (act == ACT_SILU) return z * sigmoid(z);
    if (act == ACT_GELU) return z * sigmoid(1.5957691216057308f * (z + 0.044715f * z * z * z));
    return z;
}
__device__ __forceinline__ float activate_grad(float z, int act)
{
    if (act == ACT_RELU) return z > 0.f ? 1.f : 0.f;
    // both slopes are 0 or 1 in 32 bits beyond 100; limiting z there (NaN passes) keeps
    // 0 x Inf out of the terms below: z z overflows from 1.8e19 on, a kept z may be Inf
    z = z > 100.f ? 100.f : z < -100.f ? -100.f : z;
    if (act == ACT_SILU) {
        const float s = sigmoid(z);
        return s * (1.f + z * (1.f - s));
    }
    if (act == ACT_GELU) {
        const float s = sigmoid(1.5957691216057308f * (z + 0.044715f * z * z * z));
        return s + z * s * (1.f - s) * 1.5957691216057308f * (1.f + 0.134145f * z * z);
    }
    return 1.f;
}

}  // namespace tensor
}  // namespace ccl
