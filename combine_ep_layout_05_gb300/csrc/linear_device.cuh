// What the dense products' kernels share: their arguments on the device, the
// activations and the rows of an epilogue.
#pragma once

#include "launch_order.cuh"
#include "tcgen05.cuh"
#include "vec8.cuh"

namespace ep {

namespace {

constexpr int kStep = 64;                       // contraction of a step: 128 bytes of bf16
constexpr int kPart = 128;                      // rows of an operand that a CTA holds
constexpr int kPartBytes = kPart * kStep * 2;

constexpr float kGeluA = 0.7978845608028654f, kGeluB = 0.044715f;   // sqrt(2 / pi), and the cubic's factor

// Instruction descriptor: fp32 accumulators, bf16 operands; A and B along the
// contraction (K-major) or along their rows (MN-major).
__host__ __device__ constexpr uint32_t mma_idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (uint32_t)a_mn << 15 | (uint32_t)b_mn << 16 | (uint32_t)(N >> 3) << 17 |
           (uint32_t)(M >> 4) << 24;
}

// Shared-memory descriptor of an MN-major operand in the 128-byte swizzle: 64
// rows of the operand lie side by side in 128 bytes, one line for each index of
// the contraction, atoms of 8 lines (1024 bytes) one after the other; the next
// 64 rows are group_bytes further on.
__device__ __forceinline__ uint64_t smem_desc_mn(const void *p, int group_bytes) {
    return (uint64_t)((smem_addr(p) & 0x3FFFF) >> 4) | (uint64_t)(group_bytes >> 4) << 16 |
           (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// D[M x N] (+)= A[M x 16] B[N x 16]^T, bf16, fp32 accumulators in tensor memory; as mma_f8
template <int CG>
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    if (CG == 2)
        asm volatile(
            "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(
                d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(
                d_tmem),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
            : "memory");
}

// One box of a tensor map -> this CTA's shared memory; its bytes are counted on
// a barrier of either CTA of the pair (bar: its address in the cluster).
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
        "[%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// One box of this CTA's shared memory -> a tensor; parts beyond its ends are not written
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, int x, int y, int z, const void *src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
                 "r"(y), "r"(z), "r"(smem_addr(src))
                 : "memory");
}

__device__ __forceinline__ float sigmoid_fast(float x) {   // the reciprocal is within one unit in the last place
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.f + expf(-x)));
    return r;
}

// the activation of one pre-activation (SwiGLU: swiglu())
__device__ __forceinline__ float activate(float z, int act) {
    switch (act) {
        case EP_ACT_RELU: return z < 0.f ? 0.f : z;        // (NaN stays)
        case EP_ACT_SILU: return z * sigmoid_fast(z);
        case EP_ACT_GELU: return z * sigmoid_fast(2.f * kGeluA * (z + kGeluB * z * z * z));
        default: return z;
    }
}

// N (a multiple of 16) consecutive outputs of a row, of which n (if positive,
// possibly more than N) exist, in the widest stores that the row's alignment
// allows: align 32 or 16 bytes at every 16th column, or none.
template <int N>
__device__ __forceinline__ void store_bf16(uint16_t *p, const float (&v)[N], int n, int align) {
#pragma unroll
    for (int i = 0; i < N; i += 16) {
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = pack_bf16x2(v[i + 2 * j], v[i + 2 * j + 1]);
        if (n - i >= 16 && align == 32) {
            st_v8(p + i, o);
        } else if (n - i >= 16 && align == 16) {
            st_v4(p + i, make_uint4(o[0], o[1], o[2], o[3]));
            st_v4(p + i + 8, make_uint4(o[4], o[5], o[6], o[7]));
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (i + j < n) p[i + j] = (uint16_t)(o[j / 2] >> (j & 1) * 16);
        }
    }
}
template <int N>
__device__ __forceinline__ void store_fp32(float *p, const float (&v)[N], int n, int align) {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(v[i + j]);
        if (n - i >= 8 && align == 32) {
            st_v8(p + i, o);
        } else if (n - i >= 8 && align == 16) {
            st_v4(p + i, make_uint4(o[0], o[1], o[2], o[3]));
            st_v4(p + i + 4, make_uint4(o[4], o[5], o[6], o[7]));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (i + j < n) p[i + j] = v[i + j];
        }
    }
}
// N consecutive bf16 of a row, as far as they exist (the rest are 0), two in a word
template <int N>
__device__ __forceinline__ void load_bf16(const uint16_t *p, uint32_t (&o)[N / 2], int n, int align) {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        if (n - i >= 8 && align >= 16) {
            const uint4 a = *reinterpret_cast<const uint4 *>(p + i);   // (may be what the same thread overwrites later)
            o[i / 2] = a.x;
            o[i / 2 + 1] = a.y;
            o[i / 2 + 2] = a.z;
            o[i / 2 + 3] = a.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; j += 2)
                o[(i + j) / 2] = (i + j < n ? p[i + j] : 0u) | (i + j + 1 < n ? (uint32_t)p[i + j + 1] << 16 : 0u);
        }
    }
}
template <int N>
__device__ __forceinline__ void add_bf16(const uint32_t (&o)[N / 2], float (&v)[N]) {
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
        v[2 * j] += bf16_lo(o[j]);
        v[2 * j + 1] += bf16_hi(o[j]);
    }
}
// v += N consecutive numbers of a vector (the same for every lane), as far as they exist
template <int N>
__device__ __forceinline__ void add_vector(const float *p, float (&v)[N], int n) {
    if (n >= N && ((uintptr_t)p & 15) == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 b = __ldg(reinterpret_cast<const float4 *>(p + i));
            v[i] += b.x;
            v[i + 1] += b.y;
            v[i + 2] += b.z;
            v[i + 3] += b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) v[i] += __ldg(p + i);
    }
}

}  // namespace

}  // namespace ep
