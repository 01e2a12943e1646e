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
// taken out.  A pair, because shared memory bounds these products: a CTA
// alone (128 x 256) would write and read 96 KB of it for a block, 768 cycles
// at 128 bytes each for 512 cycles of products; a CTA of a pair holds half of
// the matrix rows, 64 KB.
//
// A persistent pair walks (expert, row tile, column tile) triples; each CTA
// holds 128 of the tile's rows and 128 of its matrix rows.  Warps: warp 0
// copies boxes of 128 matrix rows (TMA), warp 1 of the first CTA issues the
// products, warps 4-7 copy the rows, which lie in R segments of any length,
// with 16-byte asynchronous copies in the swizzle that the products expect,
// and the scales (warp 2 passes on that they are there); eight warps (two warpgroups, one for each half of the
// columns) scale, accumulate and store: a thread owns a row.
#include <cstddef>

#include "expert_device.cuh"

namespace ep {

namespace {

constexpr int kExpertThreads = 512;             // warpgroup 0: boxes and products; 1: rows; 2, 3: accumulation
constexpr int kIssueRegs = 24, kCopyRegs = 56, kAccRegs = 216;   // 24 + 56 + 2 * 216 = 4 * 128, the launch's registers
constexpr int kStages = 6;                      // operand buffers: 192 KB
constexpr int kPairRows = 2 * kBlock;           // rows of a pair's tile
constexpr int kCopyWarps = 4;                   // warps that copy rows
// Steps whose scales are kept.  The copies of a step wait until the products
// kStages steps before are done, which waited for the accumulation two steps
// before those: its scales may be overwritten from kStages + 2 steps on.
constexpr int kScaleRing = 16;
static_assert(kScaleRing > kStages + 2, "scales are still in use when they are overwritten");

struct ExpertShared {
    unsigned char buf[kStages][2 * kOperand];              // rows, then matrix rows
    uint64_t rows_full[kStages], full[kStages];            // this CTA's rows and scales; all operands of both CTAs
    uint64_t done[kStages];                                // a step's products: its buffers are free, its sums ready
    uint64_t tempty[2];                                    // accumulators taken out
    uint64_t joined;                                       // maxima of a unit are written
    float row_scale[kScaleRing][kBlock], w_scale[kScaleRing][2];
    float amax[2][2][kBlock];                              // [unit parity][warpgroup][row]
    WorkList list;
    uint32_t tmem;
    int abort;
};

template <bool SWIGLU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kExpertThreads, 1)
    expert_kernel(const __grid_constant__ ExpertArgs a, const __grid_constant__ CUtensorMap map_w) {
    extern __shared__ unsigned char raw[];
    ExpertShared &s = *reinterpret_cast<ExpertShared *>(raw + ((1024 - (smem_addr(raw) & 1023)) & 1023));
    constexpr int S = kStages, NB = 2;
    static_assert(offsetof(ExpertShared, rows_full) % 8 == 0 && offsetof(ExpertShared, w_scale) % 8 == 0, "");
    const Dims &d = a.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = (int)d.E;
    const int rank = (int)cluster_rank();                           // place in the pair
    const int kb_n = (int)(a.K / kBlock);
    const int n_cols = (int)(SWIGLU ? a.N / 2 : a.N);               // output columns
    const int tile_cols = SWIGLU ? kBlock : NB * kBlock;
    const int col_tiles = (n_cols + tile_cols - 1) / tile_cols;
    const int first_unit = blockIdx.x >> 1, step = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&s.rows_full[i], kCopyWarps * 32);
            mbar_init(&s.full[i], 3);      // (the first CTA's) the bytes of both boxes, word of both CTAs' rows
            mbar_init(&s.done[i], 1);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&s.tempty[i], 16);   // (the first CTA's) the accumulating warps of both
        mbar_init(&s.joined, 8);
        s.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<2>(&s.tmem);
    make_list(s.list, a, kPairRows, kExpertThreads);
    tmem_fence_before();
    __syncthreads();
    cluster_sync();    // the other CTA's barriers are there too
    tmem_fence_after();
    const uint32_t tmem = s.tmem;
    const int units = s.list.first[E] * col_tiles;   // below 2^31: checked on the host
    volatile int *abort = &s.abort;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 0) {
            // ---- matrix rows ----
            if (lane == 0) {
                int st = 0, ph = 1, it = 0;
                bool ok = true;
                for (int u = first_unit; u < units && ok; u += step) {
                    const Unit v = find_unit(s.list, E, kPairRows, col_tiles, u);
                    const int w_row = SWIGLU ? v.nb * kBlock + rank * n_cols : v.nb * tile_cols + rank * kBlock;
                    for (int kb = 0; kb < kb_n; ++kb, ++it) {
                        ok = mbar_wait_or_abort(&s.done[st], ph, abort);
                        if (!ok) break;
                        if (rank == 0) mbar_expect_tx(&s.full[st], 2 * kOperand);
                        tma_load_3d<2>(s.buf[st] + kOperand, &map_w, kb * kBlock, w_row, v.e, cluster_addr(&s.full[st], 0));
                        if (++st == S) { st = 0; ph ^= 1; }
                    }
                }
                // No copy may land after the pair has left.  Only where something gave up is one still in flight
                // then: the first CTA's barriers count both boxes; the second gives its own a millisecond.
                if (!ok) {
                    if (rank == 0) {
                        for (int i = it > S ? it - S : 0; i < it; ++i) mbar_wait_bounded(&s.full[i % S], (i / S) & 1);
                    } else {
                        const long long t0 = clock64();
                        while (clock64() - t0 < (1 << 21)) {}
                    }
                }
            }
            __syncwarp();
        } else if (warp == 1 && rank == 0) {
            // ---- products (the loop is the whole warp's, so that its values are uniform; one lane issues) ----
            constexpr uint32_t idesc = mma_idesc(kPairRows, NB * kBlock);
            const bool issue = elect_one();
            const uint64_t desc = smem_desc(s.buf[0]);
            int st = 0, ph = 0, acc = 0, aph = 1, last = -1;
            bool ok = true;
            for (int u = first_unit; u < units && ok; u += step) {
                for (int kb = 0; kb < kb_n; ++kb) {
                    ok = mbar_wait_or_abort(&s.tempty[acc], aph, abort) && mbar_wait_or_abort(&s.full[st], ph, abort);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    tmem_fence_after();
                    if (issue) {
                        const uint64_t da = desc + (uint32_t)(st * (2 * kOperand >> 4)), db = da + (kOperand >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32 channels a step
                            mma_f8<2>(tmem + acc * 256, da + k * 2, db + k * 2, idesc, k > 0);
                        mma_commit<2>(&s.done[st]);
                    }
                    last = st | ph << 8;
                    if (++st == S) { st = 0; ph ^= 1; }
                    acc ^= 1;
                    aph ^= acc == 0;
                }
            }
            if (!ok && last >= 0) mbar_wait_bounded(&s.done[last & 255], last >> 8);
            __syncwarp();
        } else if (warp == 2) {
            // ---- word of this CTA's rows to the first CTA ----
            if (lane == 0) {
                const uint32_t full = cluster_addr(&s.full[0], 0);
                int st = 0, ph = 0;
                bool ok = true;
                for (int u = first_unit; u < units && ok; u += step) {
                    for (int kb = 0; kb < kb_n; ++kb) {
                        ok = mbar_wait_or_abort(&s.rows_full[st], ph, abort);
                        if (!ok) break;
                        fence_async_shared();
                        mbar_arrive_cluster(full + st * 8);
                        if (++st == S) { st = 0; ph ^= 1; }
                    }
                }
            }
            __syncwarp();
        }
    } else if (warp < 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
        // ---- rows and scales: eight lanes copy a row's 128 bytes, warp w rows 4 w .. 4 w + 3 of every 16 ----
        constexpr int kStep = kCopyWarps * 4, kMine = kBlock / kStep;
        static_assert(kMine == 8, "32 rows a warp: one scale a lane");
        const int part = (warp - 4) * 4 + (lane >> 3), piece = lane & 7;
        const int place = (lane >> 2) * kStep + (warp - 4) * 4 + (lane & 3);      // the row whose scale this lane copies
        const int n_blocks = (int)((a.N + kBlock - 1) / kBlock);
        int st = 0, ph = 1, ring = 0;
        bool ok = true;
        for (int u = first_unit; u < units && ok; u += step) {
            const Unit v = find_unit(s.list, E, kPairRows, col_tiles, u);
            // offsets in blocks of 128 channels, of the rows and so of their scales (below 2^32)
            int m[kMine + 1], row[kMine + 1];
#pragma unroll
            for (int i = 0; i < kMine; ++i) m[i] = v.m0 + rank * kBlock + i * kStep + part;
            m[kMine] = v.m0 + rank * kBlock + place;
            const int n = v.rows - rank * kBlock;     // this CTA's rows (128 or fewer, or none)
            receive_rows(a, v.e, m, row);
#pragma unroll
            for (int i = 0; i <= kMine; ++i) row[i] *= kb_n;
            const int blk = SWIGLU ? v.nb : v.nb * NB;
            uint32_t ws = (uint32_t)(v.e * n_blocks + blk) * kb_n;
            if (lane == 1) ws += SWIGLU ? n_blocks / 2 * kb_n : blk + 1 < n_blocks ? kb_n : 0;   // (zeros beyond N)
            for (int kb = 0; kb < kb_n; ++kb) {
                ok = __all_sync(kFull, mbar_wait_or_abort(&s.done[st], ph, abort));
                if (!ok) break;
                const uint32_t dst = smem_addr(s.buf[st]) + part * kBlock + ((piece ^ (part & 7)) << 4);
                const uint8_t *src = a.a + kb * kBlock + piece * 16;
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    if (i * kStep < n - part)
                        cp_async16(dst + i * kStep * kBlock, src + (uint64_t)(uint32_t)row[i] * kBlock);
                if (place < n)
                    cp_async4(smem_addr(&s.row_scale[ring][place]), a.a_scales + (uint32_t)(row[kMine] + kb));
                if (warp == 4 && lane < 2) cp_async4(smem_addr(&s.w_scale[ring][lane]), a.w_scales + (ws + kb));
                cp_async_arrive(&s.rows_full[st]);
                if (++st == S) { st = 0; ph ^= 1; }
                ring = (ring + 1) % kScaleRing;
            }
        }
        cp_async_wait_all();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAccRegs));
        // ---- accumulation: thread = row, warpgroup = 64 of each block's 128 columns ----
        const int half = (warp - 8) >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const uint32_t tm = tmem + (uint32_t)(quarter * 32) * 65536 + half * 64;
        const uint32_t tempty = cluster_addr(&s.tempty[0], 0);
        int st = 0, ph = 0, p = 0, ring = 0, unit = 0;
        bool ok = true;
        for (int u = first_unit; u < units && ok; u += step, ++unit) {
            const Unit v = find_unit(s.list, E, kPairRows, col_tiles, u);
            const bool some = rank * kBlock + quarter * 32 < v.rows;     // rows in this warp's lanes
            const bool live = rank * kBlock + r < v.rows;
            const int m[1] = {v.m0 + min(rank * kBlock + r, v.rows - 1)};
            int rows[1];
            receive_rows(a, v.e, m, rows);
            const int row = rows[0];
            uint64_t acc[NB][32];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < 32; ++c) acc[b][c] = 0;
            for (int kb = 0; kb < kb_n; ++kb) {
                ok = __all_sync(kFull, mbar_wait_or_abort(&s.done[st], ph, abort));
                if (!ok) break;
                if (some) {
                    tmem_fence_after();
                    const float sr = s.row_scale[ring][r];
                    const float2 sw = *reinterpret_cast<const float2 *>(s.w_scale[ring]);
                    const uint32_t s0 = __float_as_uint(sr * sw.x), s1 = __float_as_uint(sr * sw.y);
                    const uint64_t sc[2] = {pair2(s0, s0), pair2(s1, s1)};
#pragma unroll
                    for (int b = 0; b < NB; ++b) {
                        uint32_t t[64];
                        tmem_ld64(tm + p * 256 + b * kBlock, t);
                        if (b == NB - 1) {
                            tmem_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_cluster(tempty + p * 8);
                        }
#pragma unroll
                        for (int c = 0; c < 32; ++c) fma2(acc[b][c], pair2(t[2 * c], t[2 * c + 1]), sc[b]);
                    }
                } else if (lane == 0) {
                    mbar_arrive_cluster(tempty + p * 8);
                }
                if (++st == S) { st = 0; ph ^= 1; }
                p ^= 1;
                ring = (ring + 1) % kScaleRing;
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
                        h[x] = swiglu(g, up);
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
        tmem_free<2>(tmem);
    }
    if (threadIdx.x == 0 && s.abort) raise_status(a.dev_status, EP_STATUS_TIMEOUT);
}

template <bool SWIGLU>
cudaError_t launch(const ExpertArgs &a, const CUtensorMap &map_w, cudaStream_t st) {
    constexpr int bytes = sizeof(ExpertShared) + 1024;
    static_assert(bytes <= 227 * 1024, "shared memory");
    static std::atomic<int> ready[kCacheDevices];
    cudaError_t e = cudaSuccess;
    cached_per_device(ready, [&](int) {
        e = cudaFuncSetAttribute(expert_kernel<SWIGLU>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        // the warpgroups' register shares are drawn from what the block was launched with
        cudaFuncAttributes f{};
        if (!e) e = cudaFuncGetAttributes(&f, expert_kernel<SWIGLU>);
        if (!e && f.numRegs * 4 < kIssueRegs + kCopyRegs + 2 * kAccRegs) e = cudaErrorInvalidDeviceFunction;
        return e == cudaSuccess ? 1 : 0;
    });
    if (e) return e;
    expert_kernel<SWIGLU><<<num_sms() & ~1, kExpertThreads, bytes, st>>>(a, map_w);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_many(const ExpertArgs &a, cudaStream_t st) {
    CUtensorMap map_w;
    if (cudaError_t e = matrix_map(a, &map_w)) return e;
    return a.q ? launch<true>(a, map_w, st) : launch<false>(a, map_w, st);
}

}  // namespace ep
