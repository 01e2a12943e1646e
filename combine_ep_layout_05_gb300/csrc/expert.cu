// Expert products over the expert-major receive buffer: FP8 operands with a
// scale for each block of 128 channels (1 x 128 for the rows, 128 x 128 for
// the matrices), fp32 accumulation, bf16 output or SwiGLU with an FP8 cast.
//
//   c[row, n] = sum_b as[row, b] ws[n / 128, b] sum_{i in b} a[row, i] w[n, i]
//
// The inner sums are tensor-core products of 256 rows x 256 matrix rows x 128
// channels on a CTA pair, into tensor memory; the scales are plain fp32
// numbers (not powers of two), so every block's product is taken out of
// tensor memory and added, times its scale, to fp32 registers.  Two
// accumulators in tensor memory alternate: one is filled while the other is
// taken out.
//
// A persistent pair walks (expert, row tile, column tile) triples; each CTA
// holds 128 of the tile's rows and 128 of its matrix rows.  An expert's rows
// lie in R segments: the part of a segment that falls in the tile is copied
// in boxes of 128, 64, .. 1 rows (one box where the segment covers the tile).
// Warp 0 issues the copies, warp 1 of the first CTA the products, eight warps
// of each CTA (two warpgroups, one for each half of the columns) scale,
// accumulate and store; a thread owns a row, so its scale is one number a
// block.
#include "tcgen05.cuh"
#include "vec8.cuh"

namespace ep {

namespace {

constexpr int kBlock = 128;                     // channels, and matrix rows, of a scale; rows of a tile
constexpr int kOperand = kBlock * kBlock;       // bytes of 128 rows x 128 channels
constexpr int kExpertThreads = 384;             // warpgroup 0: copies and products; 1, 2: accumulation
constexpr int kIssueRegs = 56, kAccRegs = 224;  // 56 + 2 * 224 = 3 * 168, the launch's registers
constexpr int kLdBufs = 2;
constexpr int kTmemCols = 512;

constexpr int kStages = 6;                      // operand buffers: 192 KB
constexpr int kPairRows = 2 * kBlock;           // rows of a pair's tile

struct ExpertMaps {
    CUtensorMap a[8];     // the rows, in boxes of 2^i rows
    CUtensorMap w;        // the matrices, in boxes of 128 rows
};

struct ExpertShared {
    unsigned char buf[kStages][2 * kOperand];              // rows, then matrix rows
    uint64_t full[kStages], empty[kStages];                // operand buffers
    uint64_t tfull[2], tempty[2];                          // accumulators
    uint64_t joined;                                       // maxima of a unit are written
    float amax[2][2][kBlock];                              // [unit parity][warpgroup][row]
    int2 box[kBlock];                                      // copies of a tile: first row; place and log2 height
    int first[kMaxExperts + 1];                            // row tiles of the experts before
    int rows[kMaxExperts];
    uint32_t tmem;
    int abort;
};

// One unit of work: the pair's tile
struct Unit {
    int e, m0;        // expert and its first row
    int rows;         // rows from m0 on (at most 256)
    int nb;           // column tile
};

__device__ __forceinline__ Unit find_unit(const ExpertShared &s, int E, int col_tiles, int u) {
    // the last e with first[e] * col_tiles <= u (experts without rows share their successor's first tile)
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.first[mid] * col_tiles <= u) lo = mid;
        else hi = mid;
    }
    const int tiles = s.first[lo + 1] - s.first[lo];
    const int r = u - s.first[lo] * col_tiles;
    Unit v;
    v.e = lo;
    v.nb = r / tiles;                 // row tiles fastest: they share the matrix rows
    v.m0 = (r % tiles) * kPairRows;
    v.rows = min(kPairRows, s.rows[lo] - v.m0);
    return v;
}

// Lists the copies that bring rows [m0, m0 + n) of expert e (n <= 128) into a
// tile; returns their number.  Called by a whole warp.
__device__ __forceinline__ int list_boxes(ExpertShared &s, const ExpertArgs &a, int e, int m0, int n) {
    const Dims &d = a.d;
    const int lane = threadIdx.x & 31, R = (int)d.R, Tr = (int)d.Tr;
    int before = 0, boxes = 0;
    __syncwarp();
    for (int r0 = 0; r0 < R; r0 += 32) {
        const int r = r0 + lane;
        const int c = r < R ? min(max(a.tokens_per_expert[(int64_t)r * d.E + e], 0), Tr) : 0;
        int end = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, end, o);
            if (lane >= o) end += v;
        }
        end += before;
        before = __shfl_sync(kFull, end, 31);
        const int lo = max(end - c, m0), hi = min(end, m0 + n);
        const int len = max(hi - lo, 0);
        int at = __popc(len);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, at, o);
            if (lane >= o) at += v;
        }
        const int last = __shfl_sync(kFull, at, 31);
        at += boxes - __popc(len);
        boxes += last;
        int row = (e * R + r) * Tr + lo - (end - c), place = lo - m0;
        for (int left = len; left;) {
            const int lg = 31 - __clz(left);
            s.box[at++] = make_int2(row, place | lg << 8);
            row += 1 << lg;
            place += 1 << lg;
            left -= 1 << lg;
        }
    }
    __syncwarp();
    return boxes;
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

template <bool SWIGLU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kExpertThreads, 1)
    expert_kernel(const __grid_constant__ ExpertArgs a, const __grid_constant__ ExpertMaps maps) {
    extern __shared__ unsigned char raw[];
    ExpertShared &s = *reinterpret_cast<ExpertShared *>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
    constexpr int S = kStages, NB = 2;
    const Dims &d = a.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = (int)d.E;
    const int rank = (int)cluster_rank();                           // place in the pair
    const int kb_n = (int)(a.K / kBlock);
    const int n_cols = (int)(SWIGLU ? a.N / 2 : a.N);               // output columns
    const int tile_cols = SWIGLU ? kBlock : NB * kBlock;
    const int col_tiles = (n_cols + tile_cols - 1) / tile_cols;
    const int first_unit = blockIdx.x >> 1, step = gridDim.x >> 1;

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
            mbar_init(&s.full[i], 1);      // the first CTA's counts both CTAs' bytes
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.tfull[i], 1);
            mbar_init(&s.tempty[i], 16);   // the first CTA's: the accumulating warps of both
        }
        mbar_init(&s.joined, 8);
        s.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s.tmem)),
                     "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    __syncthreads();
    if (warp == 0) {   // tiles of the experts before each
        int sum = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int t = e0 + lane < E ? (s.rows[e0 + lane] + kPairRows - 1) / kPairRows : 0;
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
    cluster_sync();    // the other CTA's barriers are there too
    tmem_fence_after();
    const uint32_t tmem = s.tmem;
    const int units = s.first[E] * col_tiles;   // below 2^31: checked on the host
    volatile int *abort = &s.abort;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 0) {
            // ---- copies ----
            int it = 0;
            bool ok = true;
            for (int u = first_unit; u < units && ok; u += step) {
                const Unit v = find_unit(s, E, col_tiles, u);
                const int m = v.m0 + rank * kBlock, n = min(max(v.rows - rank * kBlock, 0), kBlock);
                const int boxes = list_boxes(s, a, v.e, m, n);
                const int w_row = SWIGLU ? v.nb * kBlock + rank * n_cols : v.nb * tile_cols + rank * kBlock;
                const uint32_t bytes = v.rows * kBlock + 2 * kOperand;   // of both CTAs
                for (int kb = 0; kb < kb_n; ++kb, ++it) {
                    const int st = it % S;
                    ok = mbar_wait_or_abort(&s.empty[st], ((it / S) & 1) ^ 1, abort);
                    if (!__all_sync(kFull, ok)) { ok = false; break; }
                    unsigned char *buf = s.buf[st];
                    const uint32_t bar = cluster_addr(&s.full[st], 0);
                    if (lane == 0) {
                        if (rank == 0) mbar_expect_tx(&s.full[st], bytes);
                        tma_load_3d(buf + kOperand, &maps.w, kb * kBlock, w_row, v.e, bar);
                    }
                    for (int b = lane; b < boxes; b += 32) {
                        const int2 x = s.box[b];
                        tma_load_2d(buf + (x.y & 255) * kBlock, &maps.a[x.y >> 8], kb * kBlock, x.x, bar);
                    }
                    __syncwarp();
                }
            }
            // No copy may land after the pair has left.  Only where something gave up is one still in flight then:
            // the first CTA's barriers count all of them; the second gives its own a millisecond.
            if (!ok) {
                if (rank == 0) {
                    for (int i = it > S ? it - S : 0; i < it; ++i) mbar_wait_bounded(&s.full[i % S], (i / S) & 1);
                } else {
                    const long long t0 = clock64();
                    while (clock64() - t0 < (1 << 21)) {}
                }
            }
        } else if (warp == 1 && rank == 0) {
            // ---- products ----
            if (lane == 0) {
                constexpr uint32_t idesc = mma_idesc(kPairRows, NB * kBlock);
                int it = 0;
                bool ok = true;
                for (int u = first_unit; u < units && ok; u += step) {
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
        const int n_blocks = (int)((a.N + kBlock - 1) / kBlock);
        int it = 0, unit = 0;
        bool ok = true;
        uint32_t tempty[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) tempty[i] = cluster_addr(&s.tempty[i], 0);
        for (int u = first_unit; u < units && ok; u += step, ++unit) {
            const Unit v = find_unit(s, E, col_tiles, u);
            const bool some = rank * kBlock + quarter * 32 < v.rows;     // rows in this warp's lanes
            const bool live = rank * kBlock + r < v.rows;
            const int row = receive_row(a, v.e, v.m0 + min(rank * kBlock + r, v.rows - 1));
            // offsets of the row's and of the first block's scales (below 2^32: an operand in memory has 128 bytes a
            // scale); to the second block's: none beyond N, where the products are zeros and not stored
            const uint32_t as = (uint32_t)row * kb_n;
            const int blk = SWIGLU ? v.nb : v.nb * NB;
            const uint32_t ws = (uint32_t)(v.e * n_blocks + blk) * kb_n;
            const uint32_t ws2 = SWIGLU ? n_blocks / 2 * kb_n : blk + 1 < n_blocks ? kb_n : 0;
            uint64_t acc[NB][32];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < 32; ++c) acc[b][c] = 0;
            // scales of the next two blocks are on their way while two blocks are accumulated
            float sa_n[2], sw_n[NB][2];
            auto load_scales = [&](int kb0) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int kb = min(kb0 + j, kb_n - 1);
                    sa_n[j] = a.a_scales[as + kb];
#pragma unroll
                    for (int b = 0; b < NB; ++b) sw_n[b][j] = a.w_scales[ws + b * ws2 + kb];
                }
            };
            load_scales(0);
            for (int kb0 = 0; kb0 < kb_n && ok; kb0 += 2) {
                float sc[NB][2];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int b = 0; b < NB; ++b) sc[b][j] = sa_n[j] * sw_n[b][j];
                load_scales(kb0 + 2);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    if (kb0 + j >= kb_n) break;
                    const int p = it & 1;
                    ok = mbar_wait_or_abort(&s.tfull[p], (it >> 1) & 1, abort);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    ++it;
                    if (!some) {
                        if (lane == 0) mbar_arrive_cluster(tempty[p]);
                        continue;
                    }
                    tmem_fence_after();
                    constexpr int LB = kLdBufs;
                    uint32_t t[LB][32];
                    const uint32_t at = tm + p * 256;
                    if (LB == 2) tmem_ld32(at, t[0]);
#pragma unroll
                    for (int q = 0; q < 2 * NB; ++q) {
                        if (LB == 1) tmem_ld32(at + (q >> 1) * kBlock + (q & 1) * 32, t[0]);
                        tmem_wait_ld(t[q % LB]);
                        if (q + 1 == 2 * NB) {
                            tmem_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster(tempty[p]);
                        } else if (LB == 2) {
                            tmem_ld32(at + ((q + 1) >> 1) * kBlock + ((q + 1) & 1) * 32, t[(q + 1) % LB]);
                        }
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            fma2(acc[q >> 1][(q & 1) * 16 + c], t[q % LB][2 * c], t[q % LB][2 * c + 1], sc[q >> 1][j]);
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
                    uint8_t *q = a.q + (int64_t)row * n_cols + v.nb * kBlock + half * 64;
                    uint32_t o[16];
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        o[c] = (uint32_t)pack_e4m3x2(lo2(acc[0][2 * c]) * inv, hi2(acc[0][2 * c]) * inv) |
                               (uint32_t)pack_e4m3x2(lo2(acc[0][2 * c + 1]) * inv, hi2(acc[0][2 * c + 1]) * inv) << 16;
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        st_v4(q + 16 * c, make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]));
                    if (half == 0) a.q_scales[(int64_t)row * (n_cols / kBlock) + v.nb] = amax / 448.f;
                }
            } else if (live) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int n0 = v.nb * tile_cols + b * kBlock + half * 64;
                    uint16_t *y = a.y + (int64_t)row * a.N + n0;
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
    cluster_sync();    // nothing of the other CTA arrives here, or reads from here, any more
    if (warp == 1) {
        tmem_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
    }
    if (threadIdx.x == 0 && s.abort) raise_status(a.dev_status, EP_STATUS_TIMEOUT);
}

template <bool SWIGLU>
cudaError_t launch(const ExpertArgs &a, const ExpertMaps &maps, cudaStream_t st) {
    constexpr int bytes = sizeof(ExpertShared) + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory");
    static std::atomic<int> ready[kCacheDevices];
    cudaError_t e = cudaSuccess;
    cached_per_device(ready, [&](int) {
        e = cudaFuncSetAttribute(expert_kernel<SWIGLU>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        // the warpgroups' register shares are drawn from what the block was launched with
        cudaFuncAttributes f{};
        if (!e) e = cudaFuncGetAttributes(&f, expert_kernel<SWIGLU>);
        if (!e && f.numRegs * 3 < kIssueRegs + 2 * kAccRegs) e = cudaErrorInvalidDeviceFunction;
        return e == cudaSuccess ? 1 : 0;
    });
    if (e) return e;
    expert_kernel<SWIGLU><<<num_sms() & ~1, kExpertThreads, bytes, st>>>(a, maps);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert(const ExpertArgs &a, cudaStream_t st) {
    ExpertMaps maps;
    const cuuint64_t da[2] = {(cuuint64_t)a.K, (cuuint64_t)(a.d.E * a.d.T)}, sa[1] = {(cuuint64_t)a.K};
    for (int i = 0; i < 8; ++i) {
        const cuuint32_t box[2] = {kBlock, 1u << i};
        if (cudaError_t e = encode_map(&maps.a[i], 2, a.a, da, sa, box)) return e;
    }
    const cuuint64_t dw[3] = {(cuuint64_t)a.K, (cuuint64_t)a.N, (cuuint64_t)a.d.E};
    const cuuint64_t sw[2] = {(cuuint64_t)a.K, (cuuint64_t)(a.N * a.K)};
    const cuuint32_t bw[3] = {kBlock, kBlock, 1};
    if (cudaError_t e = encode_map(&maps.w, 3, a.w, dw, sw, bw)) return e;
    return a.q ? launch<true>(a, maps, st) : launch<false>(a, maps, st);
}

}  // namespace ep
