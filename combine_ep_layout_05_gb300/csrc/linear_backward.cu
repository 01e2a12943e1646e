// What the gradients of a dense product need besides its two products: the
// gradient of the pre-activations (and its column sums, the bias's gradient),
// and the sum of the parts of a split contraction.
//
// G = grad_out * act'(pre) is bound by memory: one pass, a thread has 8 columns
// of every 8th row of its block, in 16-byte loads and stores where rows allow
// them.  G is rounded to bf16 once, because the tensor core's operands are bf16;
// the column sums take the numbers before that rounding.  Sums are fp32, in an
// order that depends on the sizes only.  8192 rows of 2 x 2048 (SwiGLU, bf16 gradient)
// take 33 us with a cold L2 (168 MB, 5.1 TB/s), the sum of 4 parts of 256 x 7168 10 us.
#include <algorithm>

#include "linear_device.cuh"

namespace ep {

namespace {

constexpr int kGradThreads = 256;
constexpr int kLanes = 8;                       // rows a block works on at once
constexpr int kCols = kGradThreads / kLanes * 8;

// d act(z) / dz, of silu and gelu
__device__ __forceinline__ float act_slope(float z, int act) {
    if (act == EP_ACT_SILU) {
        const float s = sigmoid_fast(z);
        return s * (1.f + z * (1.f - s));
    }
    const float s = sigmoid_fast(2.f * kGeluA * (z + kGeluB * z * z * z));
    const float d = s * (1.f + z * (1.f - s) * 2.f * kGeluA * (1.f + 3.f * kGeluB * z * z));
    // (from 30 on s is 0 or 1, and z^2 may overflow)
    return fabsf(z) > 30.f ? (z > 0.f ? 1.f : 0.f) : d;
}

// 8 consecutive numbers of a row, of which n exist (the rest read as 0)
__device__ __forceinline__ void load8(const uint16_t *p, int n, bool vec, float (&v)[8]) {
    if (vec && n >= 8) {
        const uint4 u = ld_stream(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = bf16_lo(w[i]);
            v[2 * i + 1] = bf16_hi(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? __uint_as_float((uint32_t)p[i] << 16) : 0.f;
    }
}
__device__ __forceinline__ void load8(const float *p, int n, bool vec, float (&v)[8]) {
    if (vec && n >= 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 u = ld_stream(p + 4 * h);
            v[4 * h] = __uint_as_float(u.x);
            v[4 * h + 1] = __uint_as_float(u.y);
            v[4 * h + 2] = __uint_as_float(u.z);
            v[4 * h + 3] = __uint_as_float(u.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
    }
}
__device__ __forceinline__ void store8(uint16_t *p, int n, bool vec, const float (&v)[8]) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    if (vec && n >= 8) {
        st_v4(p, make_uint4(o[0], o[1], o[2], o[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = (uint16_t)(o[i / 2] >> (i & 1) * 16);
    }
}

// L: type of grad_out.  vec bits: rows of grad_out (1), pre (2), its up half (4), G (8) and its up half (16) are
// aligned to 16 bytes at every 8th column.
template <typename L, bool SWIGLU>
__global__ void __launch_bounds__(kGradThreads) act_grad_kernel(const ActGradArgs a, int vec) {
    let_next_launch_begin();
    constexpr int P = SWIGLU ? 2 : 1;
    __shared__ float part[kLanes][P][kCols];
    const int group = threadIdx.x & 31, row_lane = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * kCols + group * 8;
    const int n = (int)min((int64_t)8, a.N - c);
    float sum[P][8] = {};
    if (n > 0) {
        const int64_t per = (a.M + a.blocks - 1) / a.blocks;
        const int64_t first = blockIdx.y * per, last = min(a.M, first + per);
        for (int64_t m = first + row_lane; m < last; m += kLanes) {
            float g[8], z[8], up[8];
            load8(reinterpret_cast<const L *>(a.grad) + m * a.grad_stride + c, n, vec & 1, g);
            if (SWIGLU) {
                const uint16_t *pre = a.pre + m * 2 * a.N + c;
                load8(pre, n, vec & 2, z);
                load8(pre + a.N, n, vec & 4, up);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float s = sigmoid_fast(z[i]), gi = g[i];
                    // (the slope first: far out it is 0, and products of the others may overflow)
                    g[i] = gi * (s * (1.f + z[i] * (1.f - s)) * up[i]);
                    up[i] = gi * (z[i] * s);
                    sum[0][i] += g[i];
                    sum[P - 1][i] += up[i];
                }
            } else {
                if (a.act != EP_ACT_NONE) {
                    load8(a.pre + m * a.N + c, n, vec & 2, z);
                    // (relu chooses, so that a gradient of infinity beside a slope of 0 leaves 0; a NaN stays)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        g[i] = a.act == EP_ACT_RELU ? (z[i] > 0.f ? g[i] : z[i] <= 0.f ? 0.f : z[i])
                                                    : g[i] * act_slope(z[i], a.act);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[0][i] += g[i];
            }
            if (a.G) {
                uint16_t *o = a.G + m * a.G_stride + c;
                store8(o, n, vec & 8, g);
                if (SWIGLU) store8(o + a.N, n, vec & 16, up);
            }
        }
    }
    if (!a.sums) return;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) part[row_lane][p][group * 8 + i] = sum[p][i];
    __syncthreads();
    for (int i = threadIdx.x; i < P * kCols; i += kGradThreads) {
        const int p = i / kCols, x = i % kCols;
        const int64_t col = (int64_t)blockIdx.x * kCols + x;
        if (col >= a.N) continue;
        float t = 0.f;
#pragma unroll
        for (int l = 0; l < kLanes; ++l) t += part[l][p][x];
        a.sums[blockIdx.y * P * a.N + p * a.N + col] = t;
    }
}

// bias[c] = sum over the blocks of sums[block][c]: 8 threads a column
__global__ void __launch_bounds__(kGradThreads) sum_blocks_kernel(const float *sums, int blocks, int64_t cols, float *bias) {
    wait_for_launch_before();
    let_next_launch_begin();
    __shared__ float part[kLanes][32];
    const int x = threadIdx.x & 31, l = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + x;
    float t = 0.f;
    if (c < cols)
        for (int b = l; b < blocks; b += kLanes) t += sums[b * cols + c];
    part[l][x] = t;
    __syncthreads();
    if (l == 0 && c < cols) {
        t = 0.f;
#pragma unroll
        for (int i = 0; i < kLanes; ++i) t += part[i][x];
        bias[c] = t;
    }
}

// out[r, c] = sum over the parts of parts[part][r, c], 8 columns (which divide a row) a thread
__global__ void __launch_bounds__(kGradThreads) sum_parts_kernel(const SumPartsArgs a) {
    wait_for_launch_before();
    let_next_launch_begin();
    const int64_t i = ((int64_t)blockIdx.x * kGradThreads + threadIdx.x) * 8;
    if (i >= a.rows * a.cols) return;
    float v[8] = {};
    for (int s = 0; s < a.parts; ++s) {
        float x[8];
        load8(a.p + s * a.rows * a.cols + i, 8, true, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += x[j];
    }
    const int64_t r = i / a.cols, c = i - r * a.cols;
    if (a.out32) {
        float *o = reinterpret_cast<float *>(a.out) + r * a.stride + c;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            st_v4(o + 4 * h, make_uint4(__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                                        __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])));
    } else {
        store8(reinterpret_cast<uint16_t *>(a.out) + r * a.stride + c, 8, a.vec, v);
    }
}

bool aligned16(const void *p, int64_t stride_bytes) { return (((uintptr_t)p | (uintptr_t)stride_bytes) & 15) == 0; }

}  // namespace

int act_grad_blocks(int64_t M, int64_t N) {
    // enough blocks for 8 on each of 152 SMs, of at least 8 rows
    const int64_t cols = (N + kCols - 1) / kCols, want = (1216 + cols - 1) / cols, most = (M + kLanes - 1) / kLanes;
    return (int)std::max<int64_t>(1, std::min(want, most));
}

cudaError_t launch_act_grad(const ActGradArgs &a, cudaStream_t st) {
    const bool swiglu = a.act == EP_ACT_SWIGLU;
    const int64_t wide = swiglu ? 2 * a.N : a.N;
    const dim3 grid((unsigned)((a.N + kCols - 1) / kCols), (unsigned)a.blocks);
    const int vec = (aligned16(a.grad, a.grad_stride * (a.grad32 ? 4 : 2)) ? 1 : 0) |
                    (aligned16(a.pre, wide * 2) ? 2 : 0) | (aligned16(a.pre + (swiglu ? a.N : 0), wide * 2) ? 4 : 0) |
                    (aligned16(a.G, a.G_stride * 2) ? 8 : 0) | (aligned16(a.G + (swiglu ? a.N : 0), a.G_stride * 2) ? 16 : 0);
    if (a.grad32) {
        if (swiglu) act_grad_kernel<float, true><<<grid, kGradThreads, 0, st>>>(a, vec);
        else act_grad_kernel<float, false><<<grid, kGradThreads, 0, st>>>(a, vec);
    } else {
        if (swiglu) act_grad_kernel<uint16_t, true><<<grid, kGradThreads, 0, st>>>(a, vec);
        else act_grad_kernel<uint16_t, false><<<grid, kGradThreads, 0, st>>>(a, vec);
    }
    if (cudaError_t e = cudaGetLastError()) return e;
    if (!a.sums) return cudaSuccess;
    return launch_in_order(kAfter, sum_blocks_kernel, dim3((unsigned)((wide + 31) / 32)), kGradThreads, 0, 0, st, a.sums,
                           a.blocks, wide, a.bias);
}

cudaError_t launch_sum_parts(SumPartsArgs a, cudaStream_t st) {
    a.vec = aligned16(a.out, a.stride * 2);
    const int64_t n = (a.rows * a.cols / 8 + kGradThreads - 1) / kGradThreads;
    return launch_in_order(kAfter, sum_parts_kernel, dim3((unsigned)n), kGradThreads, 0, 0, st, a);
}

}  // namespace ep
