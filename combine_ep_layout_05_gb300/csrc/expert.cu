// Expert products over the expert-major receive buffer: FP8 operands with a
// scale for each block of 128 channels (1 x 128 for the rows, 128 x 128 for
// the matrices), fp32 accumulation, bf16 output or SwiGLU with an FP8 cast.
//
//   c[row, n] = sum_b as[row, b] ws[n / 128, b] sum_{i in b} a[row, i] w[n, i]
//
// The inner sums are tensor-core products of 128 rows x 128 NB matrix rows x
// 128 channels into tensor memory; the scales are plain fp32 numbers (not
// powers of two), so every block's product is taken out of tensor memory and
// added, times its scale, to fp32 registers.  Two accumulators in tensor
// memory alternate: one is filled while the other is taken out.
//
// A persistent CTA walks (expert, row tile, column tile) triples.  An
// expert's rows lie in R segments, so the row operand is gathered row by row
// with tiled copies of four rows; the matrix operand comes in boxes of 128
// rows.  Warp 0 issues the copies, warp 1 the products, eight warps (two
// warpgroups, one for each half of the columns) scale, accumulate and store;
// a thread owns a row, so its scale is one number a block.
#include "tcgen05.cuh"
#include "vec8.cuh"

namespace ep {

namespace {

constexpr int kBlock = 128;                     // channels, and matrix rows, of a scale; rows of a tile
constexpr int kOperand = kBlock * kBlock;       // bytes of 128 rows x 128 channels
constexpr int kExpertThreads = 384;             // warpgroup 0: copies and products; 1, 2: accumulation
constexpr int kIssueRegs = 72, kAccRegs = 216;  // 72 + 2 * 216 = 3 * 168, the launch's registers
constexpr int kTmemCols = 512;

template <int NB>
constexpr int kStages = NB == 2 ? 4 : 6;        // operand buffers: 192 KB

template <int NB>
struct ExpertShared {
    unsigned char buf[kStages<NB>][(1 + NB) * kOperand];   // rows, then matrix blocks
    uint64_t full[kStages<NB>], empty[kStages<NB>];        // operand buffers
    uint64_t tfull[2], tempty[2];                          // accumulators
    uint64_t joined;                                       // maxima of a unit are written
    float amax[2][2][kBlock];                              // [unit parity][warpgroup][row]
    int first[kMaxExperts + 1];                            // row tiles of the experts before
    int rows[kMaxExperts];
    uint32_t tmem;
    int abort;
};

// One unit of work
struct Unit {
    int e, rows;      // expert, its rows from m0 on (at most 128)
    int m0;           // first row
    int nb;           // column tile
};

template <int NB>
__device__ __forceinline__ Unit find_unit(const ExpertShared<NB> &s, int E, int col_tiles, int64_t u) {
    // the last e with first[e] * col_tiles <= u
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)s.first[mid] * col_tiles <= u) lo = mid;
        else hi = mid;
    }
    // experts without rows share their successor's first tile: the search ends at the last of equals
    const int tiles = s.first[lo + 1] - s.first[lo];
    const int r = (int)(u - (int64_t)s.first[lo] * col_tiles);
    Unit v;
    v.e = lo;
    v.nb = r / tiles;                 // row tiles fastest: they share the matrix rows
    v.m0 = (r % tiles) * kBlock;
    v.rows = min(kBlock, s.rows[lo] - v.m0);
    return v;
}

// Receive row of each lane's m-th row of expert e (called by whole warps;
// counts outside [0, Tr] are clamped).
__device__ __forceinline__ int receive_row(const ExpertArgs &a, int e, int m) {
    const Dims &d = a.d;
    const int lane = threadIdx.x & 31, R = (int)d.R, Tr = (int)d.Tr;
    int c[2], before = 0;
    int src = 0, start = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        if (h * 32 >= R) break;
        const int r = h * 32 + lane;
        c[h] = r < R ? min(max(a.tokens_per_expert[(int64_t)r * d.E + e], 0), Tr) : 0;
        int sum = c[h];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, sum, o);
            if (lane >= o) sum += v;
        }
        sum += before;                // rows up to and with source r
        for (int i = 0; i < min(32, R - h * 32); ++i) {
            const int end = __shfl_sync(kFull, sum, i);
            if (end <= m) {
                src = h * 32 + i + 1;
                start = end;
            }
        }
        before = __shfl_sync(kFull, sum, 31);
    }
    return (e * R + src) * Tr + (m - start);
}

template <bool SWIGLU, int NB>
__global__ void __launch_bounds__(kExpertThreads, 1)
    expert_kernel(const __grid_constant__ ExpertArgs a, const __grid_constant__ CUtensorMap map_a,
                  const __grid_constant__ CUtensorMap map_w) {
    extern __shared__ unsigned char raw[];
    ExpertShared<NB> &s = *reinterpret_cast<ExpertShared<NB> *>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
    constexpr int S = kStages<NB>;
    const Dims &d = a.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = (int)d.E;
    const int kb_n = (int)(a.K / kBlock);
    const int n_cols = (int)(SWIGLU ? a.N / 2 : a.N);               // output columns
    const int tile_cols = SWIGLU ? kBlock : NB * kBlock;
    const int col_tiles = (n_cols + tile_cols - 1) / tile_cols;

    // rows of every expert
    bool bad = false;
    for (int e = threadIdx.x; e < E; e += kExpertThreads) {
        int n = 0;
        for (int r = 0; r < d.R; ++r) {
            const int c = a.tokens_per_expert[(int64_t)r * E + e];
            const int ok = min(max(c, 0), (int)d.Tr);
            bad |= ok != c;
            n += ok;
        }
        s.rows[e] = n;
    }
    if (bad && blockIdx.x == 0) raise_status(a.dev_status, EP_STATUS_BAD_SLOT);
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], 8);
        }
        mbar_init(&s.joined, 8);
        s.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s.tmem)),
                     "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    __syncthreads();
    if (warp == 0) {   // tiles of the experts before each
        int sum = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int t = e0 + lane < E ? (s.rows[e0 + lane] + kBlock - 1) / kBlock : 0;
            int inc = t;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, inc, o);
                if (lane >= o) inc += v;
            }
            if (e0 + lane < E) s.first[e0 + lane] = sum + inc - t;
            sum += __shfl_sync(kFull, inc, 31);
        }
        if (lane == 0) s.first[E] = sum;
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = s.tmem;
    const int64_t units = (int64_t)s.first[E] * col_tiles;
    volatile int *abort = &s.abort;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 0) {
            // ---- copies ----
            int it = 0;
            bool ok = true;
            for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Unit v = find_unit(s, E, col_tiles, u);
                int row[4];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    row[i] = receive_row(a, v.e, v.m0 + min(lane * 4 + i, v.rows - 1));
                const int groups = (v.rows + 3) / 4;
                const uint32_t bytes = groups * 4 * kBlock + NB * kOperand;
                for (int kb = 0; kb < kb_n; ++kb, ++it) {
                    const int st = it % S;
                    ok = mbar_wait_or_abort(&s.empty[st], ((it / S) & 1) ^ 1, abort);
                    if (!__all_sync(kFull, ok)) { ok = false; break; }
                    unsigned char *buf = s.buf[st];
                    if (lane == 0) {
                        mbar_expect_tx(&s.full[st], bytes);
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            tma_load_3d(buf + (1 + b) * kOperand, &map_w, kb * kBlock,
                                        SWIGLU ? v.nb * kBlock + b * n_cols : v.nb * tile_cols + b * kBlock, v.e,
                                        &s.full[st]);
                    }
                    __syncwarp();
                    if (lane < groups)
                        tma_gather4(buf + lane * 4 * kBlock, &map_a, kb * kBlock, row[0], row[1], row[2], row[3],
                                    &s.full[st]);
                }
            }
            // no copy may land after the CTA has left (only where the products gave up is one still in flight)
            if (!ok)
                for (int i = it > S ? it - S : 0; i < it; ++i) mbar_wait_bounded(&s.full[i % S], (i / S) & 1);
        } else if (warp == 1) {
            // ---- products ----
            if (lane == 0) {
                constexpr uint32_t idesc = mma_idesc(kBlock, NB * kBlock);
                int it = 0;
                bool ok = true;
                for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x) {
                    for (int kb = 0; kb < kb_n && ok; ++kb, ++it) {
                        const int st = it % S, acc = it & 1;
                        ok = mbar_wait_or_abort(&s.tempty[acc], ((it >> 1) & 1) ^ 1, abort) &&
                             mbar_wait_or_abort(&s.full[st], (it / S) & 1, abort);
                        if (!ok) break;
                        tmem_fence_after();
                        const uint64_t da = smem_desc(s.buf[st]), db = smem_desc(s.buf[st] + kOperand);
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32 channels a step
                            mma_f8(tmem + acc * 256, da + k * 2, db + k * 2, idesc, k > 0);
                        mma_commit(&s.empty[st]);
                        mma_commit(&s.tfull[acc]);
                    }
                }
                if (!ok && it > 0) mbar_wait_bounded(&s.tfull[(it - 1) & 1], ((it - 1) >> 1) & 1);
            }
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAccRegs));
        // ---- accumulation: thread = row, warpgroup = 64 of each block's 128 columns ----
        const int half = (warp - 4) >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const uint32_t tm = tmem + (uint32_t)(quarter * 32) * 65536 + half * 64;
        const int64_t n_blocks = (a.N + kBlock - 1) / kBlock;
        int it = 0, unit = 0;
        bool ok = true;
        for (int64_t u = blockIdx.x; u < units && ok; u += gridDim.x, ++unit) {
            const Unit v = find_unit(s, E, col_tiles, u);
            const bool some = quarter * 32 < v.rows;     // rows in this warp's lanes
            const bool live = r < v.rows;
            const int64_t row = receive_row(a, v.e, v.m0 + min(r, v.rows - 1));
            const float *as = a.a_scales + row * kb_n;
            const float *ws[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                int64_t blk = SWIGLU ? v.nb + b * (n_blocks / 2) : (int64_t)v.nb * NB + b;
                if (blk >= n_blocks) blk = n_blocks - 1;  // columns beyond N: computed from zeros, not stored
                ws[b] = a.w_scales + ((int64_t)v.e * n_blocks + blk) * kb_n;
            }
            uint64_t acc[NB][32];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < 32; ++c) acc[b][c] = 0;
            float sa_n[4], sw_n[NB][4];
            auto load_scales = [&](int kb0) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int kb = min(kb0 + j, kb_n - 1);
                    sa_n[j] = as[kb];
#pragma unroll
                    for (int b = 0; b < NB; ++b) sw_n[b][j] = ws[b][kb];
                }
            };
            load_scales(0);
            for (int kb0 = 0; kb0 < kb_n && ok; kb0 += 4) {
                float sc[NB][4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int b = 0; b < NB; ++b) sc[b][j] = sa_n[j] * sw_n[b][j];
                if (kb0 + 4 < kb_n) load_scales(kb0 + 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (kb0 + j >= kb_n) break;
                    const int p = it & 1;
                    ok = mbar_wait_or_abort(&s.tfull[p], (it >> 1) & 1, abort);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    ++it;
                    if (!some) {
                        if (lane == 0) mbar_arrive(&s.tempty[p]);
                        continue;
                    }
                    tmem_fence_after();
                    uint32_t t[2][32];
                    const uint32_t at = tm + p * 256;
                    tmem_ld32(at, t[0]);
#pragma unroll
                    for (int q = 0; q < 2 * NB; ++q) {
                        tmem_wait_ld(t[q & 1]);
                        if (q + 1 < 2 * NB) {
                            tmem_ld32(at + ((q + 1) >> 1) * kBlock + ((q + 1) & 1) * 32, t[(q + 1) & 1]);
                        } else {
                            tmem_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&s.tempty[p]);
                        }
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            fma2(acc[q >> 1][(q & 1) * 16 + c], t[q & 1][2 * c], t[q & 1][2 * c + 1], sc[q >> 1][j]);
                    }
                }
            }
            if (!ok) break;
            if (SWIGLU) {
                // gate in acc[0], up in acc[NB - 1]; the cast's maximum over 128 channels joins the two warpgroups
                float amax = 0.f;
                bool nan = false;
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    float h[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float g = x ? hi2(acc[0][c]) : lo2(acc[0][c]);
                        const float up = x ? hi2(acc[NB - 1][c]) : lo2(acc[NB - 1][c]);
                        h[x] = g / (1.f + expf(-g)) * up;
                        amax = fmaxf(amax, fabsf(h[x]));
                        nan |= h[x] != h[x];
                    }
                    acc[0][c] = (uint64_t)__float_as_uint(h[1]) << 32 | __float_as_uint(h[0]);
                }
                if (nan) amax = __uint_as_float(0x7fffffffu);
                s.amax[unit & 1][half][r] = amax;
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.joined);
                ok = __all_sync(kFull, mbar_wait_or_abort(&s.joined, unit & 1, abort));
                if (!ok) break;
                const float other = s.amax[unit & 1][half ^ 1][r];
                amax = amax != amax || other != other ? __uint_as_float(0x7fffffffu) : fmaxf(amax, other);
                if (live) {
                    const float inv = amax > 0.f ? fminf(448.f / amax, 3.402823466e38f) : 0.f;
                    uint8_t *q = a.q + row * n_cols + v.nb * kBlock + half * 64;
                    uint32_t o[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        o[c] = (uint32_t)pack_e4m3x2(lo2(acc[0][2 * c]) * inv, hi2(acc[0][2 * c]) * inv) |
                               (uint32_t)pack_e4m3x2(lo2(acc[0][2 * c + 1]) * inv, hi2(acc[0][2 * c + 1]) * inv) << 16;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        st_v4(q + 16 * c, make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]));
                    if (half == 0) a.q_scales[row * (n_cols / kBlock) + v.nb] = amax / 448.f;
                }
            } else if (live) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int n0 = v.nb * tile_cols + b * kBlock + half * 64;
                    uint16_t *y = a.y + row * a.N + n0;
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        if (n0 + 8 * c < n_cols)
                            st_v4(y + 8 * c,
                                  make_uint4(pack_bf16x2(lo2(acc[b][4 * c]), hi2(acc[b][4 * c])),
                                             pack_bf16x2(lo2(acc[b][4 * c + 1]), hi2(acc[b][4 * c + 1])),
                                             pack_bf16x2(lo2(acc[b][4 * c + 2]), hi2(acc[b][4 * c + 2])),
                                             pack_bf16x2(lo2(acc[b][4 * c + 3]), hi2(acc[b][4 * c + 3]))));
                }
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 1) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
    }
    if (threadIdx.x == 0 && s.abort) raise_status(a.dev_status, EP_STATUS_TIMEOUT);
}

template <bool SWIGLU, int NB>
cudaError_t launch(const ExpertArgs &a, const CUtensorMap &map_a, const CUtensorMap &map_w, cudaStream_t st) {
    constexpr int bytes = sizeof(ExpertShared<NB>) + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory");
    static std::atomic<int> ready[kCacheDevices];
    cudaError_t e = cudaSuccess;
    cached_per_device(ready, [&](int) {
        e = cudaFuncSetAttribute(expert_kernel<SWIGLU, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        // the warpgroups' register shares are drawn from what the block was launched with
        cudaFuncAttributes f{};
        if (!e) e = cudaFuncGetAttributes(&f, expert_kernel<SWIGLU, NB>);
        if (!e && f.numRegs * 3 < kIssueRegs + 2 * kAccRegs) e = cudaErrorInvalidDeviceFunction;
        return e == cudaSuccess ? 1 : 0;
    });
    if (e) return e;
    expert_kernel<SWIGLU, NB><<<num_sms(), kExpertThreads, bytes, st>>>(a, map_a, map_w);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert(const ExpertArgs &a, cudaStream_t st) {
    CUtensorMap map_a, map_w;
    const cuuint64_t da[2] = {(cuuint64_t)a.K, (cuuint64_t)(a.d.E * a.d.T)}, sa[1] = {(cuuint64_t)a.K};
    const cuuint32_t ba[2] = {kBlock, 1};
    cudaError_t e = encode_map(&map_a, 2, a.a, da, sa, ba);
    if (e) return e;
    const cuuint64_t dw[3] = {(cuuint64_t)a.K, (cuuint64_t)a.N, (cuuint64_t)a.d.E};
    const cuuint64_t sw[2] = {(cuuint64_t)a.K, (cuuint64_t)(a.N * a.K)};
    const cuuint32_t bw[3] = {kBlock, kBlock, 1};
    e = encode_map(&map_w, 3, a.w, dw, sw, bw);
    if (e) return e;
    return a.q ? launch<true, 2>(a, map_a, map_w, st) : launch<false, 2>(a, map_a, map_w, st);
}

}  // namespace ep
