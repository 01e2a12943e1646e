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
constexpr int kMostChain = 128;                 // steps that one accumulator sums, where the result is bf16

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

__device__ __forceinline__ float gelu(float z) { return z * sigmoid_fast(2.f * kGeluA * (z + kGeluB * z * z * z)); }

// the activation of N pre-activations (SwiGLU: swiglu()).  One branch for all: one for each took three times the arithmetic
// (a tile of 256 x 256 outputs with silu 12.8 us).
template <int N>
__device__ __forceinline__ void activate(float (&z)[N], int act) {
    if (act == EP_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] *= sigmoid_fast(z[i]);
    } else if (act == EP_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = gelu(z[i]);
    } else if (act == EP_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = z[i] < 0.f ? 0.f : z[i];        // (NaN stays)
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
// Rows that start anywhere, through 32 rows of 128 bytes of shared memory whose 16-byte pieces are swizzled: a thread owns
// row `lane` there, in global memory the warp goes along one row after the other (two at a time in words, if rows start at
// multiples of 4 bytes).  A thread going along its own row would touch a line of its own for each number: 7619 rows of
// 1806, with pre-activations, took 344 us.  By whole warps; rows: how many exist, n: columns that exist.
__device__ __forceinline__ unsigned char *row_byte(unsigned char *buf, int row, int byte) {
    return buf + row * 128 + ((byte >> 4 ^ (row & 7)) << 4) + (byte & 15);
}
__device__ __forceinline__ void put_row(unsigned char *buf, const float (&z)[32]) {       // as bf16
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(row_byte(buf, lane, i * 16)) =
            make_uint4(pack_bf16x2(z[8 * i], z[8 * i + 1]), pack_bf16x2(z[8 * i + 2], z[8 * i + 3]),
                       pack_bf16x2(z[8 * i + 4], z[8 * i + 5]), pack_bf16x2(z[8 * i + 6], z[8 * i + 7]));
}
__device__ __forceinline__ void put_row_fp32(unsigned char *buf, const float (&z)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        *reinterpret_cast<float4 *>(row_byte(buf, lane, i * 16)) = make_float4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]);
}
// 32 columns of bf16, from the shared rows to p (row 0, column 0)
__device__ __forceinline__ void copy_out(unsigned char *buf, uint16_t *p, int64_t stride, int rows, int n) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
    if ((((uintptr_t)p | (uintptr_t)(stride * 2)) & 3) == 0) {
        const int c = (lane & 15) * 2;
#pragma unroll 4
        for (int r = lane >> 4; r < rows; r += 2) {
            const uint32_t v = *reinterpret_cast<const uint32_t *>(row_byte(buf, r, c * 2));
            if (c + 1 < n) *reinterpret_cast<uint32_t *>(p + r * stride + c) = v;
            else if (c < n) p[r * stride + c] = (uint16_t)v;
        }
    } else if (lane < n) {
#pragma unroll 4
        for (int r = 0; r < rows; ++r) p[r * stride + lane] = *reinterpret_cast<const uint16_t *>(row_byte(buf, r, lane * 2));
    }
    __syncwarp();
}
__device__ __forceinline__ void copy_out_fp32(unsigned char *buf, float *p, int64_t stride, int rows, int n) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
    if (lane < n)
#pragma unroll 4
        for (int r = 0; r < rows; ++r) p[r * stride + lane] = *reinterpret_cast<const float *>(row_byte(buf, r, lane * 4));
    __syncwarp();
}
// 32 columns of bf16 to the thread that owns the row (the rest are 0); all loads are under way together
__device__ __forceinline__ void copy_in(unsigned char *buf, const uint16_t *p, int64_t stride, int rows, int n,
                                        uint32_t (&o)[16]) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
    if ((((uintptr_t)p | (uintptr_t)(stride * 2)) & 3) == 0) {
        const int c = (lane & 15) * 2, r0 = lane >> 4;
        uint32_t v[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint16_t *q = p + (r0 + 2 * i) * stride + c;
            v[i] = 0;
            if (r0 + 2 * i < rows && c + 1 < n) v[i] = *reinterpret_cast<const uint32_t *>(q);
            else if (r0 + 2 * i < rows && c < n) v[i] = *q;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) *reinterpret_cast<uint32_t *>(row_byte(buf, r0 + 2 * i, c * 2)) = v[i];
    } else {
        uint16_t v[32];
#pragma unroll
        for (int r = 0; r < 32; ++r) v[r] = lane < n && r < rows ? p[r * stride + lane] : (uint16_t)0;
#pragma unroll
        for (int r = 0; r < 32; ++r) *reinterpret_cast<uint16_t *>(row_byte(buf, r, lane * 2)) = v[r];
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 v = *reinterpret_cast<const uint4 *>(row_byte(buf, lane, i * 16));
        o[4 * i] = v.x;
        o[4 * i + 1] = v.y;
        o[4 * i + 2] = v.z;
        o[4 * i + 3] = v.w;
    }
    __syncwarp();
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
