// Expert products for experts with few rows: the matrices are read once and
// that is what takes the time.
//
// Same operation as expert.cu, with the operands' parts exchanged: 128 matrix
// rows are the tensor core's M, the expert's rows its N (16, 32, 48 or 64, as
// many as there are), so a step costs next to nothing beside the copy of its
// matrix rows: SwiGLU 32 KB (128 gate and 128 up rows), else 16 KB, for which
// an SM's share of the memory rate takes some 1400 and 700 cycles.  160 KB of
// operands in flight cover the memory's latency several times.
//
// An accumulator in tensor memory has a matrix row in each lane and the
// expert's rows in its columns; four alternate.  A thread owns a matrix row:
// the matrix's scale is one number, the rows' scales are read from shared
// memory.  Warps as in expert.cu; SwiGLU's two warpgroups hold gate and up,
// swap halves of their columns through shared memory at the end, and each
// finishes its half.
//
// Measured: 32 tokens x top-8 over 256 experts of 7168 x 2048, SwiGLU: 680 to 720 us,
// 6.7 to 7.1 TB/s (reading alone is faster than the copy that the rate is judged by,
// 6.8); 1024 tokens 1.14 ms, 6.6 TB/s; one token's down product 25.0 us (117 MB; 22.9
// from a graph, 17 of them memory, the rest launch and first tiles).
#include <cstddef>

#include "expert_device.cuh"

// Most rows an expert, on average (tokens x top-k / experts, what the host
// knows), for this kernel: a tile of 64 rows has to hold nearly every expert.
// Measured, this kernel / the other, hidden 7168 x 2048, SwiGLU in us:
//                      32 rows        48 rows        64 rows
//   256 experts, uniform    1141 / 1493    1200 / 1516    1755 / 1534
//   256, popularity 1/rank  1373 / 1581    1564 / 1613    1835 / 1675
//   32, uniform                             186 / 207      267 / 208
// (down product of 256 experts at 48 rows: 634 / 819 uniform, 853 / 829 by 1/rank;
// at 64: 987 / 819).  The counts are on the device, so the average is what the rule
// has; where a few experts take every token it is the slower choice (all on 8 of
// 256 experts: 303 / 124 at an average of 16 rows, 893 / 317 at 48).
#ifndef EP_EXPERT_FEW_ROWS
#define EP_EXPERT_FEW_ROWS 48
#endif

namespace ep {

namespace {

constexpr int kThreads = 512;                   // warpgroup 0: boxes and products; 1: rows; 2, 3: accumulation
constexpr int kIssueRegs = 80, kCopyRegs = 80, kAccRegs = 176;   // 80 + 80 + 2 * 176 = 4 * 128, the launch's registers
constexpr int kRows = 64;                       // rows of a tile
constexpr int kCopyThreads = 128;
constexpr int kAcc = 4;                         // accumulators
template <bool SWIGLU>
constexpr int kStages = SWIGLU ? 4 : 7;         // operand buffers
// Steps whose scales are kept: a step's copies wait for the products kStages
// steps before, those for the loads of the accumulation kAcc steps before
// them, which may still be using that step's scales.
constexpr int kScaleRing = 16;

template <bool SWIGLU>
struct FewShared {
    unsigned char w[kStages<SWIGLU>][(SWIGLU ? 2 : 1) * kOperand];
    unsigned char rows[kStages<SWIGLU>][kRows * kBlock];
    uint64_t boxes[kStages<SWIGLU>];                              // matrix rows
    uint64_t rows_full[kStages<SWIGLU>], full[kStages<SWIGLU>];   // rows and scales; all operands
    uint64_t done[kStages<SWIGLU>];                               // a step's products: buffers free, sums, scales and
                                                                  // rows ready
    uint64_t tempty[kAcc];                                        // accumulators taken out
    uint64_t swapped, joined;                                     // the ends of a SwiGLU unit
    alignas(16) float row_scale[kScaleRing][kRows];               // (read 16 bytes at a time, as are the maxima)
    float w_scale[kScaleRing][2];
    float swap[SWIGLU ? 2 : 1][kRows / 2][kBlock];
    alignas(16) uint32_t amax[kRows][4];
    int row[kScaleRing][kRows];                                   // a unit's receive rows (kept like the scales)
    WorkList list;
    uint32_t tmem;
    int gave_up;
};

template <bool SWIGLU>
__global__ void __launch_bounds__(kThreads, 1)
    expert_few_kernel(const __grid_constant__ ExpertArgs a, const __grid_constant__ CUtensorMap map_w) {
    extern __shared__ __align__(1024) unsigned char raw[];    // (the only shared memory: it starts at its window's start)
    FewShared<SWIGLU> &s = *reinterpret_cast<FewShared<SWIGLU> *>(raw);
    constexpr int S = kStages<SWIGLU>, NB = SWIGLU ? 2 : 1;
    static_assert(offsetof(FewShared<SWIGLU>, rows) % 1024 == 0 && offsetof(FewShared<SWIGLU>, boxes) % 8 == 0, "");
    static_assert(offsetof(FewShared<SWIGLU>, row_scale) % 16 == 0 && offsetof(FewShared<SWIGLU>, amax) % 16 == 0, "");
    static_assert(kScaleRing > S + kAcc + 1, "scales are still in use when they are overwritten");
    const Dims &d = a.d;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = (int)d.E;
    const int kb_n = (int)(a.K / kBlock);
    const int n_cols = (int)(SWIGLU ? a.N / 2 : a.N);               // output columns
    const int col_tiles = (n_cols + kBlock - 1) / kBlock;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&s.rows_full[i], kCopyThreads + 2);   // the copies' own arrivals; two warps for what they stored
            mbar_init(&s.boxes[i], 1);
            mbar_init(&s.full[i], 1);
            mbar_init(&s.done[i], 2);          // the products' commit, word of the operands
        }
        for (int i = 0; i < kAcc; ++i) mbar_init(&s.tempty[i], 8);
        mbar_init(&s.swapped, 8);
        mbar_init(&s.joined, 8);
        s.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<1>(&s.tmem);
    make_list(s.list, a, kRows, kThreads);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = s.tmem;
    const int units = s.list.first[E] * col_tiles;   // below 2^31: checked on the host
    const Patience patience{&s.gave_up, a.wait_clocks};

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 0) {
            // ---- matrix rows ----
            if (lane == 0) {
                int st = 0, ph = 1, it = 0;
                bool ok = true;
                for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                    const Unit v = find_unit(s.list, E, kRows, col_tiles, u);
                    for (int kb = 0; kb < kb_n; ++kb, ++it) {
                        ok = mbar_wait(&s.done[st], ph, patience);
                        if (!ok) break;
                        mbar_expect_tx(&s.boxes[st], NB * kOperand);
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            tma_load_3d(s.w[st] + b * kOperand, &map_w, kb * kBlock, v.nb * kBlock + b * n_cols, v.e,
                                        &s.boxes[st]);
                        if (++st == S) { st = 0; ph ^= 1; }
                    }
                }
                drain(s.boxes, S, it);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ---- products (the loop is the whole warp's, so that its values are uniform; one lane issues) ----
            const bool issue = elect_one();
            const uint64_t dw = smem_desc(s.w[0]), dr = smem_desc(s.rows[0]);
            int st = 0, ph = 0, acc = 0, aph = 1, it = 0;
            bool ok = true;
            for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                const Unit v = find_unit(s.list, E, kRows, col_tiles, u);
                const uint32_t idesc = mma_idesc(kBlock, (v.rows + 15) & ~15);
                for (int kb = 0; kb < kb_n; ++kb, ++it) {
                    ok = warp_wait(&s.full[st], ph, patience) && warp_wait(&s.tempty[acc], aph, patience);
                    if (!ok) break;
                    tmem_fence_after();
                    if (issue) {
                        const uint64_t da = dw + (uint32_t)(st * (NB * kOperand >> 4));
                        const uint64_t db = dr + (uint32_t)(st * (kRows * kBlock >> 4));
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int k = 0; k < 4; ++k)   // 32 channels a step
                                mma_f8<1>(tmem + (acc * NB + b) * kRows, da + (b * (kOperand >> 4) + k * 2), db + k * 2, idesc,
                                          k > 0);
                        mma_commit<1>(&s.done[st]);
                    }
                    if (++st == S) { st = 0; ph ^= 1; }
                    acc = (acc + 1) % kAcc;
                    aph ^= acc == 0;
                }
            }
            drain(s.done, S, it);
            __syncwarp();
        } else if (warp == 2) {
            // ---- word of the operands: to the products, and to the accumulation, which reads the scales and the rows'
            // numbers with ordinary loads and has no other release of them to wait for (the commit's arrival tells of
            // the products) ----
            if (lane == 0) {
                int st = 0, ph = 0;
                bool ok = true;
                for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
                    for (int kb = 0; kb < kb_n; ++kb) {
                        ok = mbar_wait(&s.rows_full[st], ph, patience) && mbar_wait(&s.boxes[st], ph, patience);
                        if (!ok) break;
                        fence_async_shared();
                        mbar_arrive(&s.done[st]);
                        mbar_arrive(&s.full[st]);
                        if (++st == S) { st = 0; ph ^= 1; }
                    }
                }
            }
            __syncwarp();
        }
    } else if (warp < 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
        // ---- rows and scales: eight lanes copy a row's 128 bytes ----
        constexpr int kStep = kCopyThreads / 8, kMine = kRows / kStep;
        const int part = (threadIdx.x - 128) >> 3, piece = lane & 7;
        const int place = (threadIdx.x - 128) & (kRows - 1);      // the row whose scale this thread copies, if below 64
        const int n_blocks = (int)((a.N + kBlock - 1) / kBlock);
        int st = 0, ph = 1, ring = 0, unit = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x, ++unit) {
            const Unit v = find_unit(s.list, E, kRows, col_tiles, u);
            // offsets in blocks of 128 channels, of the rows and so of their scales (below 2^32)
            int m[kMine + 1], row[kMine + 1];
#pragma unroll
            for (int i = 0; i < kMine; ++i) m[i] = v.m0 + i * kStep + part;
            m[kMine] = v.m0 + place;
            receive_rows(a, v.e, m, row);
            if (warp < 6) s.row[unit % kScaleRing][place] = row[kMine];
#pragma unroll
            for (int i = 0; i <= kMine; ++i) row[i] = (int)((uint32_t)row[i] * kb_n);
            uint32_t ws = (uint32_t)(v.e * n_blocks + v.nb) * kb_n;
            if (lane == 1) ws += n_blocks / 2 * kb_n;             // (SwiGLU: the up block's)
            const bool has_scale = warp < 6 && place < v.rows;
            for (int kb = 0; kb < kb_n; ++kb) {
                ok = warp_wait(&s.done[st], ph, patience);
                if (!ok) break;
                const uint32_t dst = smem_addr(s.rows[st]) + part * kBlock + ((piece ^ (part & 7)) << 4);
                const uint8_t *src = a.a + kb * kBlock + piece * 16;
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    if (i * kStep + part < v.rows)
                        cp_async16(dst + i * kStep * kBlock, src + (uint64_t)(uint32_t)row[i] * kBlock);
                if (has_scale) cp_async4(smem_addr(&s.row_scale[ring][place]), a.a_scales + (uint32_t)(row[kMine] + kb));
                if (warp == 7 && lane < NB) cp_async4(smem_addr(&s.w_scale[ring][lane]), a.w_scales + (ws + kb));
                cp_async_arrive(&s.rows_full[st]);
                // the copies' arrival speaks for the copies only: an ordinary one releases the stores to s.row (every
                // step, since the barrier's count is)
                __syncwarp();
                if (warp < 6 && lane == 0) mbar_arrive(&s.rows_full[st]);
                if (++st == S) { st = 0; ph ^= 1; }
                ring = (ring + 1) % kScaleRing;
            }
        }
        cp_async_wait_all();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAccRegs));
        // ---- accumulation: thread = matrix row.  SwiGLU: a warpgroup has a block and all columns; else every other
        // 16 columns (rows of the tile), so that both have work from 17 rows on ----
        constexpr int kMine = SWIGLU ? kRows : kRows / 2;
        const int half = (warp - 8) >> 2, quarter = warp & 3;
        const int chan = quarter * 32 + lane;
        const auto column = [&](int q) { return SWIGLU ? q * 16 : (q * 2 + half) * 16; };   // first of my q-th sixteen
        const uint32_t tm = tmem + (uint32_t)(quarter * 32) * 65536 + (SWIGLU ? half * kRows : 0);
        int st = 0, ph = 0, p = 0, ring = 0, unit = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x, ++unit) {
            const Unit v = find_unit(s.list, E, kRows, col_tiles, u);
            uint64_t acc[kMine / 2];
#pragma unroll
            for (int c = 0; c < kMine / 2; ++c) acc[c] = 0;
            for (int kb = 0; kb < kb_n; ++kb) {
                ok = warp_wait(&s.done[st], ph, patience);
                if (!ok) break;
                tmem_fence_after();
                uint32_t t[kMine];
#pragma unroll
                for (int q = 0; q < kMine / 16; ++q)
                    if (column(q) < v.rows) tmem_ld16(tm + p * (NB * kRows) + column(q), t + q * 16);
                tmem_wait_ld<kMine>(t);
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.tempty[p]);
                const uint32_t w32 = __float_as_uint(s.w_scale[ring][SWIGLU ? half : 0]);
                const uint64_t sw = pair2(w32, w32);
#pragma unroll
                for (int q = 0; q < kMine / 16; ++q) {
                    if (column(q) >= v.rows) break;
                    const ulonglong2 *sr = reinterpret_cast<const ulonglong2 *>(&s.row_scale[ring][column(q)]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const ulonglong2 x = sr[c];
                        const int i = q * 16 + c * 4;
                        fma2(acc[i / 2], pair2(t[i], t[i + 1]), mul2(x.x, sw));
                        fma2(acc[i / 2 + 1], pair2(t[i + 2], t[i + 3]), mul2(x.y, sw));
                    }
                }
                if (++st == S) { st = 0; ph ^= 1; }
                p = (p + 1) % kAcc;
                ring = (ring + 1) % kScaleRing;
            }
            if (!ok) break;
            const int *rows = s.row[unit % kScaleRing];
            if (SWIGLU) {
                // The gate's warpgroup finishes columns 0-31 and hands over the gate of columns 32-63; the up's the
                // other way round.  Its own values of the columns that it finishes end up in acc[0 .. 15].
                constexpr int H = kRows / 2;
                float *mine = &s.swap[half][0][chan];
                const float *theirs = &s.swap[half ^ 1][0][chan];
#pragma unroll
                for (int c = 0; c < H / 2; ++c) {
                    const uint64_t give = half ? acc[c] : acc[H / 2 + c];
                    mine[(2 * c) * kBlock] = lo2(give);
                    mine[(2 * c + 1) * kBlock] = hi2(give);
                    if (half) acc[c] = acc[H / 2 + c];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.swapped);
                ok = warp_wait(&s.swapped, unit & 1, patience);
                if (!ok) break;
                const int n = min(v.rows - half * H, H);   // rows among this warpgroup's columns (may be negative)
                uint32_t top = 0;                          // lane c: of column c
#pragma unroll
                for (int c = 0; c < H; ++c) {
                    if (c >= n) break;
                    const float own = c & 1 ? hi2(acc[c / 2]) : lo2(acc[c / 2]), other = theirs[c * kBlock];
                    const uint32_t bits = __float_as_uint(half ? swiglu(other, own) : swiglu(own, other));
                    acc[c / 2] = c & 1 ? (acc[c / 2] & 0xffffffffull) | (uint64_t)bits << 32
                                       : (acc[c / 2] & ~0xffffffffull) | bits;
                    const uint32_t x = __reduce_max_sync(kFull, bits & 0x7fffffffu);   // (NaN above all numbers)
                    if (lane == c) top = x;
                }
                if (lane < n) s.amax[half * H + lane][quarter] = top;
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.joined);
                ok = warp_wait(&s.joined, unit & 1, patience);
                if (!ok) break;
                float inv = 0.f;                           // lane c: of column c
                if (lane < n) {
                    const uint4 t4 = *reinterpret_cast<const uint4 *>(s.amax[half * H + lane]);
                    const float amax = __uint_as_float(max(max(t4.x, t4.y), max(t4.z, t4.w)));
                    inv = amax > 0.f ? fminf(448.f / amax, 3.402823466e38f) : 0.f;
                    if (quarter == 0)
                        a.q_scales[(int64_t)rows[half * H + lane] * (n_cols / kBlock) + v.nb] = amax / 448.f;
                }
                uint8_t *q = a.q + v.nb * kBlock + chan;
#pragma unroll
                for (int c = 0; c < H; ++c) {
                    if (c >= n) break;
                    const float h = c & 1 ? hi2(acc[c / 2]) : lo2(acc[c / 2]);
                    q[(int64_t)rows[half * H + c] * n_cols] = (uint8_t)pack_e4m3x2(h * __shfl_sync(kFull, inv, c), 0.f);
                }
            } else {
                const int col = v.nb * kBlock + chan;
                uint16_t *y = a.y + col;
#pragma unroll
                for (int c = 0; c < kMine; ++c) {
                    const int at = column(c >> 4) + (c & 15);
                    if (at >= v.rows) break;
                    const float f = c & 1 ? hi2(acc[c / 2]) : lo2(acc[c / 2]);
                    if (col < n_cols) y[(int64_t)rows[at] * n_cols] = (uint16_t)pack_bf16x2(f, 0.f);
                }
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 1) {
        tmem_fence_after();
        tmem_free<1>(tmem);
    }
    if (threadIdx.x == 0 && s.gave_up) raise_status(a.dev_status, EP_STATUS_TIMEOUT);
}

template <bool SWIGLU>
cudaError_t launch(const ExpertArgs &a, const CUtensorMap &map_w, cudaStream_t st) {
    constexpr int bytes = sizeof(FewShared<SWIGLU>);
    static_assert(bytes <= 227 * 1024, "shared memory");
    static std::atomic<int> ready[kCacheDevices];
    cudaError_t e = cudaSuccess;
    cached_per_device(ready, [&](int) {
        e = cudaFuncSetAttribute(expert_few_kernel<SWIGLU>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        // the warpgroups' register shares are drawn from what the block was launched with
        cudaFuncAttributes f{};
        if (!e) e = cudaFuncGetAttributes(&f, expert_few_kernel<SWIGLU>);
        if (!e && f.numRegs * 4 < kIssueRegs + kCopyRegs + 2 * kAccRegs) e = cudaErrorInvalidDeviceFunction;
        return e == cudaSuccess ? 1 : 0;
    });
    if (e) return e;
    expert_few_kernel<SWIGLU><<<num_sms(), kThreads, bytes, st>>>(a, map_w);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_few(const ExpertArgs &a, cudaStream_t st) {
    CUtensorMap map_w;
    if (cudaError_t e = matrix_map(a, kBlock, &map_w)) return e;
    return a.q ? launch<true>(a, map_w, st) : launch<false>(a, map_w, st);
}

cudaError_t launch_expert(const ExpertArgs &a, cudaStream_t st) {
    return a.d.T * a.d.k <= a.d.E * EP_EXPERT_FEW_ROWS ? launch_expert_few(a, st) : launch_expert_many(a, st);
}

}  // namespace ep
