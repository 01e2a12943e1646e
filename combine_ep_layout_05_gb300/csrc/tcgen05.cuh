// The 5th-generation tensor core's instructions that the expert products use:
// tensor memory, FP8 matrix products, tiled copies and their tensor maps.
#pragma once

#include <cuda.h>

#include "dispatch_device.cuh"
#include "moe_internal.cuh"

namespace ep {

namespace {

// Whether a phase is over: asked at once (SLEEP false), or after sleeping until
// it is, or for as long as the hardware lets a thread sleep.  CLUSTER: for
// arrivals of the other CTA's threads; orders no memory by itself.
template <bool SLEEP, bool CLUSTER>
__device__ __forceinline__ bool mbar_over(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
#define EP_MBAR_OVER(WAIT)                                                                                        \
    asm volatile("{ .reg .pred p; mbarrier." WAIT ".shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"          \
                 : "=r"(ok)                                                                                       \
                 : "r"(smem_addr(bar)), "r"(parity)                                                               \
                 : "memory")
    if (SLEEP && CLUSTER) EP_MBAR_OVER("try_wait.parity.relaxed.cluster");
    else if (SLEEP) EP_MBAR_OVER("try_wait.parity");
    else if (CLUSTER) EP_MBAR_OVER("test_wait.parity.relaxed.cluster");
    else EP_MBAR_OVER("test_wait.parity");
#undef EP_MBAR_OVER
    return ok != 0;
}

// How long a thread waits: until `clocks` cycles have passed, or another
// thread of the CTA has set the flag because they had.
struct Patience {
    volatile int *gave_up;
    long long clocks;
};

// Waits for a phase of an mbarrier; false if patience ran out.  The caller then
// leaves, and what it has in flight is drained at the end.
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, const Patience &p) {
    if (mbar_over<false, CLUSTER>(bar, parity)) return true;
    const long long t0 = clock64();
    do {
        if (clock64() - t0 > p.clocks) {
            *p.gave_up = 1;
            return false;
        }
        if (mbar_over<true, CLUSTER>(bar, parity)) return true;
    } while (!*p.gave_up);
    return false;
}

// The same for a whole warp; every lane polls (one lane's poll and a shuffle
// of its result took 1.1 to 1.2 times as long in the expert products).
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const Patience &p) {
    return __all_sync(kFull, mbar_wait<CLUSTER>(bar, parity, p));
}

// Waits for the phases of steps [max(0, n - S), n) of a ring of S barriers:
// of copies and products that have been issued and so end by themselves.
// Every CTA does, so that nothing is in flight when it leaves, whether it gave
// up or not.  All steps together get a second (2^31 cycles).
__device__ __forceinline__ void drain(uint64_t *bars, int S, int n) {
    const long long t0 = clock64();
    for (int i = n > S ? n - S : 0; i < n; ++i)
        while (!mbar_try_wait(&bars[i % S], i / S & 1))
            if (clock64() - t0 > (1ll << 31)) return;
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Address of the same shared-memory object in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
    return r;
}
// Shared memory of a CTA, handed to a thread of the other CTA of its pair: the
// release, of what this thread has written and seen in its own CTA's shared
// memory, before a relaxed arrival, and the acquire after a relaxed wait.
// Restricted to shared memory, the only kind that crosses: a release of all
// memory at cluster scope takes 1900 to 2700 cycles (8192 tokens' SwiGLU over
// 32 experts 3.4 ms with one for each step, 1.75 so).
__device__ __forceinline__ void release_shared_to_cluster() {
    asm volatile("fence.release.sync_restrict::shared::cta.cluster;" ::: "memory");
}
__device__ __forceinline__ void acquire_shared_of_cluster() {
    asm volatile("fence.acquire.sync_restrict::shared::cluster.cluster;" ::: "memory");
}
// Arrival on a barrier of either CTA that orders no memory by itself: after
// the release above, or for word of tensor memory's accumulators, which tcgen05's
// own fences on both sides order.
__device__ __forceinline__ void mbar_arrive_relaxed_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// one lane of a converged warp, always the same
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}
// a word of the shared memory of either CTA
__device__ __forceinline__ void store_cluster(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One box of a tensor map -> this CTA's shared memory; its bytes are counted on bar.
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

// 16 bytes global -> shared, by the thread itself (not kept in L1)
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 4 bytes global -> shared
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// arrives on bar once the copies that this thread has issued so far have landed
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// writes to shared memory that this thread has waited for become visible to the tensor core
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory descriptor of a K-major operand, rows of 128 bytes in the
// 128-byte swizzle (8-row atoms of 1024 bytes): start address and stride
// between atoms in 16-byte units, descriptor version 1, swizzle mode 2.
// The 32-byte steps along a row are added to the start address.
__device__ __forceinline__ uint64_t smem_desc(const void *p) {
    return (uint64_t)((smem_addr(p) & 0x3FFFF) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction descriptor: fp32 accumulators, e4m3 operands, both K-major.
__host__ __device__ constexpr uint32_t mma_idesc(int M, int N) {
    return 1u << 4 | (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24;
}

// D[M x N] (+)= A[M x 32] B[N x 32]^T, e4m3, fp32 accumulators in tensor
// memory; issued by one thread.  On a CTA pair (CG = 2) each CTA holds half of
// A's rows, half of B's rows (at the same shared-memory offsets) and the
// accumulators of its rows of A; a thread of the first CTA issues.
template <int CG>
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    if (CG == 2)
        asm volatile(
            "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(
                d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p; }" ::"r"(
                d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
}

// arrives on bar (of a pair: in both CTAs) once the products issued so far by this thread are done
template <int CG>
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    if (CG == 2)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_addr(bar)),
            "h"((uint16_t)3)
            : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         smem_addr(bar))
                     : "memory");
}

// all 512 columns of tensor memory, by one warp (of each CTA of a pair); the base goes to shared memory
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t *base) {
    if (CG == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(base)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(base)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t base) {
    if (CG == 2) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(base));
    else asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(base));
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 64 columns of the warp's 32 lanes (lane in the address's high half), waited
// for: the registers are the instruction's own, with no copies behind it
__device__ __forceinline__ void tmem_ld64(uint32_t addr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
        "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
        "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, "
        "%38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, "
        "%56, %57, %58, %59, %60, %61, %62, %63"
        "}, [%64]; tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]),
          "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]),
          "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
          "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]),
          "=r"(r[63])
        : "r"(addr)
        : "memory");
}

// 16 columns, started only
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
// waits for the loads started before; no use of the N registers moves ahead of the wait
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

__device__ __forceinline__ uint64_t pair2(uint32_t lo, uint32_t hi) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
    return v;
}
// acc += d * s on two neighbouring columns
__device__ __forceinline__ void fma2(uint64_t &acc, uint64_t d, uint64_t s) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(d), "l"(s));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float lo2(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi2(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// x / (1 + exp(-x)) * y; the reciprocal is within one unit in the last place
__device__ __forceinline__ float swiglu(float x, float y) {
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + expf(-x)));
    return x * r * y;
}

// Tensor map of a byte tensor with rows of dims[0] bytes in the 128-byte
// swizzle; strides in bytes of dimensions 1 and up.  The encoder is a host
// function of the driver, found once through the runtime.
inline cudaError_t encode_map(CUtensorMap *map, int rank, const void *base, const cuuint64_t *dims,
                              const cuuint64_t *strides, const cuuint32_t *box) {
    typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static std::atomic<EncodeFn> fn{nullptr};
    EncodeFn f = fn.load(std::memory_order_acquire);
    if (!f) {
        void *q = nullptr;
        cudaDriverEntryPointQueryResult found;
        const cudaError_t e =
            cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault, &found);
        if (e != cudaSuccess) return e;
        if (found != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
        f = (EncodeFn)q;
        fn.store(f, std::memory_order_release);
    }
    const cuuint32_t ones[3] = {1, 1, 1};
    const CUresult r = f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void *>(base), dims, strides,
                         box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

}  // namespace ep
