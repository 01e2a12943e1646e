// Expert products over the expert-major receive buffer: FP8 operands with a
// scale for each block of 128 channels (1 x 128 for the rows, 128 x 128 for
// the matrices), fp32 accumulation, bf16 output or SwiGLU with an FP8 cast.
//
// A CTA owns 128 output channels of one expert (with SwiGLU 128 gate and the
// 128 up channels that go with them) and walks the expert's rows in tiles of
// 16; a thread owns one channel and 8 rows.
#include "combine_device.cuh"

namespace ep {

namespace {

constexpr int kTileRows = 16, kTileCols = 128;

template <bool SWIGLU>
__global__ void __launch_bounds__(256) expert_kernel(ExpertArgs a) {
    __shared__ float s_a[kTileRows][128];
    __shared__ int64_t s_row[kTileRows];
    __shared__ int s_first[kMaxRanks + 1];
    __shared__ unsigned s_amax[kTileRows];
    const Dims &d = a.d;
    const int64_t e = blockIdx.y, nb = blockIdx.x, K = a.K, kb_n = K / 128;
    if (threadIdx.x == 0) {
        int sum = 0;
        for (int r = 0; r < d.R; ++r) {
            s_first[r] = sum;
            int64_t c = a.tokens_per_expert[r * d.E + e];
            if (c < 0 || c > d.Tr) {
                raise_status(a.dev_status, EP_STATUS_BAD_SLOT);
                c = c < 0 ? 0 : d.Tr;
            }
            sum += (int)c;
        }
        s_first[d.R] = sum;
    }
    __syncthreads();
    const int rows = s_first[d.R];
    const int half = threadIdx.x / kTileCols, col = threadIdx.x % kTileCols;
    const int64_t n = nb * kTileCols + col, n_blocks = (a.N + 127) / 128;
    const bool live = SWIGLU || n < a.N;
    const uint8_t *wg = a.w + (e * a.N + (live ? n : 0)) * K;
    const float *sg = a.w_scales + (e * n_blocks + nb) * kb_n;
    const uint8_t *wu = SWIGLU ? wg + a.N / 2 * K : wg;
    const float *su = SWIGLU ? sg + a.N / 256 * kb_n : sg;
    for (int m0 = 0; m0 < rows; m0 += kTileRows) {
        __syncthreads();
        if (threadIdx.x < kTileRows) {
            const int m = min(m0 + (int)threadIdx.x, rows - 1);
            int r = 0;
            while (s_first[r + 1] <= m) ++r;
            s_row[threadIdx.x] = (e * d.R + r) * d.Tr + (m - s_first[r]);
            s_amax[threadIdx.x] = 0;
        }
        float acc[8] = {}, acc2[8] = {};
        for (int64_t kb = 0; kb < kb_n; ++kb) {
            __syncthreads();
            for (int i = threadIdx.x; i < kTileRows * 8; i += 256) {
                const int64_t row = s_row[i / 8];
                const uint4 v = *reinterpret_cast<const uint4 *>(a.a + row * K + kb * 128 + (i % 8) * 16);
                const float s = a.a_scales[row * kb_n + kb];
                const uint32_t q[4] = {v.x, v.y, v.z, v.w};
                for (int h = 0; h < 8; ++h) {
                    const float2 f = e4m3x2_to_f32x2((uint16_t)(q[h / 2] >> (16 * (h & 1))));
                    s_a[i / 8][(i % 8) * 16 + 2 * h] = f.x * s;
                    s_a[i / 8][(i % 8) * 16 + 2 * h + 1] = f.y * s;
                }
            }
            __syncthreads();
            const float s1 = sg[kb], s2 = su[kb];
            float p[8] = {}, p2[8] = {};
            for (int c = 0; c < 128; c += 4) {
                const uint32_t g4 = *reinterpret_cast<const uint32_t *>(wg + kb * 128 + c);
                const float2 g0 = e4m3x2_to_f32x2((uint16_t)g4), g1 = e4m3x2_to_f32x2((uint16_t)(g4 >> 16));
                float2 u0, u1;
                if (SWIGLU) {
                    const uint32_t u4 = *reinterpret_cast<const uint32_t *>(wu + kb * 128 + c);
                    u0 = e4m3x2_to_f32x2((uint16_t)u4);
                    u1 = e4m3x2_to_f32x2((uint16_t)(u4 >> 16));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 v = *reinterpret_cast<const float4 *>(&s_a[half * 8 + i][c]);
                    p[i] += v.x * g0.x + v.y * g0.y + v.z * g1.x + v.w * g1.y;
                    if (SWIGLU) p2[i] += v.x * u0.x + v.y * u0.y + v.z * u1.x + v.w * u1.y;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[i] = fmaf(p[i], s1, acc[i]);
                acc2[i] = fmaf(p2[i], s2, acc2[i]);
            }
        }
        if (SWIGLU) {
            const int64_t I = a.N / 2;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                acc[i] = acc[i] / (1.f + expf(-acc[i])) * acc2[i];
                atomicMax(&s_amax[half * 8 + i], __float_as_uint(fabsf(acc[i])));
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int m = half * 8 + i;
                if (m0 + m >= rows) continue;
                const float amax = __uint_as_float(s_amax[m]);
                const float inv = amax > 0.f ? fminf(448.f / amax, 3.402823466e38f) : 0.f;
                a.q[s_row[m] * I + n] = (uint8_t)pack_e4m3x2(acc[i] * inv, 0.f);
                if (col == 0) a.q_scales[s_row[m] * (I / 128) + nb] = amax / 448.f;
            }
        } else if (live) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (m0 + half * 8 + i < rows)
                    a.y[s_row[half * 8 + i] * a.N + n] = (uint16_t)pack_bf16x2(acc[i], 0.f);
        }
    }
}

}  // namespace

cudaError_t launch_expert(const ExpertArgs &a, cudaStream_t st) {
    const int64_t cols = a.q ? a.N / 2 : a.N;
    const dim3 grid((unsigned)((cols + kTileCols - 1) / kTileCols), (unsigned)a.d.E);
    if (a.q) expert_kernel<true><<<grid, 256, 0, st>>>(a);
    else expert_kernel<false><<<grid, 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace ep
