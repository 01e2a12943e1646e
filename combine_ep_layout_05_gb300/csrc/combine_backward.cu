// Combine, backward: the gradients of the expert rows and of the weights.
//   grad_y[row(t, j)] = w_tj * grad_out[t]          (weights of a shared row summed)
//   grad_w[t, j]      = <grad_out[t], y[row(t, j)]>
// A CTA owns one token: a lane reads a 16-byte chunk of grad_out once, the
// same chunk of up to 8 rows of y, adds to its part of each row's dot
// product, and writes the scaled chunk to each row of grad_y.  The parts meet
// in a fixed order (lanes by halving, then warps in order): no atomics.
//
// Bound by memory: each row of y is read once and each row of grad_y written
// once.  32768 tokens rank-major, hidden 7168: 800 us, 6.8 TB/s, the copy rate;
// 1024 tokens expert-major: 47 us, 5.3 TB/s (the launch and three dependent
// loads before the rows are known are 9 us of it).
#include "combine_device.cuh"
#include "moe_internal.cuh"

namespace ep {

namespace {

constexpr int kBackRows = 8;   // rows a pass keeps in flight
// Tokens an SM below which a token gets eight warps.  Measured (hidden 7168,
// top-8, expert-major): 256 tokens 13.1 us with eight warps and 16.8 with four,
// 512 tokens 25.0 and 21.5, 1024 tokens 47.4 and 45.9 (seven blocks of four
// warps fit an SM, so that 1024 tokens are one wave).
#ifndef EP_COMBINE_BACK_TOKENS
#define EP_COMBINE_BACK_TOKENS 3
#endif

// The row of entry j = lane among the rows that resolve_sources kept, -1 if
// it has none (called by a whole warp).
template <int LAYOUT>
__device__ __forceinline__ int entry_row(const CombineArgs &a, int64_t t, const RouteRegs &g, const int64_t *rows, int nd) {
    const Dims &d = a.d;
    const bool in_range = g.e >= 0 && g.e < d.E;
    const unsigned same = __match_any_sync(kFull, in_range ? (int)g.e : -2 - (int)(threadIdx.x & 31));
    const bool kept = in_range && !(same & lanemask_lt());       // the first of repeated ids
    const uint32_t r = kept ? rank_of(d, (uint32_t)g.e) : 0;
    int64_t slot = g.s0, block = g.e;
    if (LAYOUT == EP_RANK_MAJOR) {
        const int32_t g0 = __shfl_sync(kFull, g.s0, r & 31), g1 = __shfl_sync(kFull, g.s1, r & 31);
        slot = r < 32 ? g0 : g1;
        block = r;
    }
    if (!kept || slot < 0 || slot >= d.Tr) return -1;
    const int64_t row = (block * d.R + t / d.Tr) * d.Tr + slot;
    for (int i = 0; i < nd; ++i)
        if (rows[i] == row) return i;
    return -1;
}

template <int LAYOUT, int W>
__global__ void __launch_bounds__(W * 32) combine_backward_kernel(CombineArgs a, const uint16_t *grad_out,
                                                                 uint16_t *grad_y, float *grad_weights) {
    __shared__ int64_t s_rows[kMaxTopk];
    __shared__ float s_wts[kMaxTopk], s_dot[W][kMaxTopk];
    __shared__ int s_nd, s_entry[kMaxTopk];
    const Dims &d = a.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t = blockIdx.x, hc = d.H / 8;
    if (warp == 0) {
        const RouteRegs g = load_route<LAYOUT>(a, t);
        const int nd = resolve_sources<LAYOUT>(a, t, t / d.Tr, g, s_rows, s_wts);
        s_entry[lane] = entry_row<LAYOUT>(a, t, g, s_rows, nd);
        if (lane == 0) s_nd = nd;
    }
    __syncthreads();
    const int nd = s_nd;
    const uint4 *go = reinterpret_cast<const uint4 *>(grad_out) + t * hc;
    const uint4 *y = reinterpret_cast<const uint4 *>(a.y);
    uint4 *gy = reinterpret_cast<uint4 *>(grad_y);
    for (int g0 = 0; g0 < nd; g0 += kBackRows) {
        float dot[kBackRows] = {};
        for (int64_t c = threadIdx.x; c < hc; c += W * 32) {
            uint4 v[kBackRows];
            if (grad_weights) {
#pragma unroll
                for (int i = 0; i < kBackRows; ++i)
                    if (g0 + i < nd) v[i] = ld_stream(y + s_rows[g0 + i] * hc + c);
            }
            const uint4 o4 = go[c];
            const uint32_t ow[4] = {o4.x, o4.y, o4.z, o4.w};
            float o[8];
#pragma unroll
            for (int h = 0; h < 4; ++h) { o[2 * h] = bf16_lo(ow[h]); o[2 * h + 1] = bf16_hi(ow[h]); }
#pragma unroll
            for (int i = 0; i < kBackRows; ++i) {
                if (g0 + i >= nd) continue;
                if (grad_weights) {
                    const uint32_t q[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        dot[i] = __fmaf_rn(o[2 * h], bf16_lo(q[h]), dot[i]);
                        dot[i] = __fmaf_rn(o[2 * h + 1], bf16_hi(q[h]), dot[i]);
                    }
                }
                if (grad_y) {
                    const float w = s_wts[g0 + i];
                    st_v4(gy + s_rows[g0 + i] * hc + c,
                          make_uint4(pack_bf16x2(w * o[0], w * o[1]), pack_bf16x2(w * o[2], w * o[3]),
                                     pack_bf16x2(w * o[4], w * o[5]), pack_bf16x2(w * o[6], w * o[7])));
                }
            }
        }
        if (grad_weights) {
#pragma unroll
            for (int i = 0; i < kBackRows; ++i) {
                float v = dot[i];
#pragma unroll
                for (int s = 16; s; s >>= 1) v += __shfl_xor_sync(kFull, v, s);
                if (lane == 0 && g0 + i < kMaxTopk) s_dot[warp][g0 + i] = v;
            }
        }
    }
    if (!grad_weights) return;
    __syncthreads();
    if (threadIdx.x < d.k) {
        const int i = s_entry[threadIdx.x];
        float v = 0.f;
        if (i >= 0)
            for (int w = 0; w < W; ++w) v += s_dot[w][i];
        grad_weights[t * d.k + threadIdx.x] = v;
    }
}

}  // namespace

cudaError_t launch_combine_backward(int layout, const CombineArgs &a, const uint16_t *grad_out, uint16_t *grad_y,
                                    float *grad_weights, cudaStream_t st) {
    const unsigned grid = (unsigned)a.d.T;
    const bool few = a.d.T < (int64_t)num_sms() * EP_COMBINE_BACK_TOKENS;
    if (layout == EP_RANK_MAJOR) {
        if (few) combine_backward_kernel<EP_RANK_MAJOR, 8><<<grid, 256, 0, st>>>(a, grad_out, grad_y, grad_weights);
        else combine_backward_kernel<EP_RANK_MAJOR, 4><<<grid, 128, 0, st>>>(a, grad_out, grad_y, grad_weights);
    } else {
        if (few) combine_backward_kernel<EP_EXPERT_MAJOR, 8><<<grid, 256, 0, st>>>(a, grad_out, grad_y, grad_weights);
        else combine_backward_kernel<EP_EXPERT_MAJOR, 4><<<grid, 128, 0, st>>>(a, grad_out, grad_y, grad_weights);
    }
    return cudaGetLastError();
}

}  // namespace ep
