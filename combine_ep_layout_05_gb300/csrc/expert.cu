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
// taken out.  (Four of 128 columns would be free sooner, but products 128
// columns wide took 1.6 times as long for the same work.)  A pair, because
// shared memory bounds these products: a CTA alone (128 x 256) would write and
// read 96 KB of it for a step, 768 cycles at 128 bytes each for 512 cycles of
// products; a CTA of a pair holds half of the matrix rows, 64 KB.
//
// A persistent pair walks (expert, row tile, column tile) triples; each CTA
// holds 128 of the tile's rows and 128 of its matrix rows.
// An expert's rows lie in R segments.  Where few segments meet in a tile its
// rows come in boxes (TMA): two of the largest power of two for each segment,
// overlapping; a box costs some 80 cycles of the copy unit, whatever its size,
// so that from kBoxes boxes on threads copy the rows, 16 bytes each, in the
// swizzle that the products expect.  Warps of a CTA: 0 issues the boxes, 1 (of
// the first CTA) the products, 2 passes on that the boxes and the rows and scales
// copied by warps 4-7 are there, 3 plans the units ahead; eight warps (two warpgroups,
// one for each half of the columns) scale, accumulate and store: a thread owns
// a row.
//
// Measured: 8192 tokens x top-8 over 32 experts of 7168 x 2048 (2048 rows each):
// SwiGLU 1.74 to 1.79 ms, 2.2 PFLOP/s; down product 0.98 to 1.0 ms, 1.95 PFLOP/s;
// the tensor pipe is active 53% and 45% of the cycles.  A step takes some 950 cycles, bound by the
// way around an accumulator: 512 of products, 580 from the first load to its
// release, and 800 of signals between the two CTAs' warps, over two accumulators.
// Without the accumulation the same loop takes 730.
#include <cstddef>

#include "expert_device.cuh"
#include "vec8.cuh"

namespace ep {

namespace {

constexpr int kExpertThreads = 512;             // warpgroup 0: boxes, products, plans; 1: rows; 2, 3: accumulation
constexpr int kIssueRegs = 56, kCopyRegs = 40, kAccRegs = 208;   // 56 + 40 + 2 * 208 = 4 * 128, the launch's registers
constexpr int kStages = 6;                      // operand buffers: 192 KB
constexpr int kPairRows = 2 * kBlock;           // rows of a pair's tile
constexpr int kCopyWarps = 4;                   // warps that copy rows
constexpr int kBoxes = 8;                       // most boxes that bring a CTA's rows; else its threads copy them
constexpr int kPlans = 4;                       // units planned ahead
constexpr int kPlanUsers = 2 + 1 + kCopyWarps + 8;   // warps that read a plan: 0, 1, 2, copies, accumulation
// Steps whose scales are kept.  The copies of a step wait until the products
// kStages steps before are done, which waited for the loads of the accumulation
// two steps before those, whose scales may still be in use then.
constexpr int kScaleRing = 16;
static_assert(kScaleRing > kStages + 3, "scales are still in use when they are overwritten");

struct ExpertMaps {
    CUtensorMap a[8];     // the rows, in boxes of 2^i rows
    CUtensorMap w;        // the matrices, in boxes of 128 rows
};

// A unit of work as its CTA needs it
struct Plan {
    int e, nb;            // expert (-1: no more units) and column tile
    int rows;             // this CTA's rows, at most 128
    int boxes;            // boxes that bring them, or -1: the threads copy them
    uint32_t expect;      // bytes of this CTA's boxes in a step
};

struct ExpertShared {
    unsigned char buf[kStages][2 * kOperand];              // rows, then matrix rows
    uint64_t boxes[kStages], rows_full[kStages];           // this CTA's boxes; its copied rows and scales
    uint64_t full[kStages];                                // (the first CTA's) all operands of both CTAs
    uint64_t done[kStages];                                // a step's products: its buffers are free, its sums and
                                                           // this CTA's scales ready
    uint64_t tempty[2];                                    // accumulators taken out
    uint64_t plan_full[kPlans], plan_empty[kPlans];
    uint64_t joined;                                       // maxima of a unit are written
    float row_scale[kScaleRing][kBlock], w_scale[kScaleRing][2];
    float amax[2][2][kBlock];                              // [unit parity][warpgroup][row]
    Plan plan[kPlans];
    int row[kPlans][kBlock];                               // a unit's receive rows
    int3 box[kPlans][kBoxes];                              // first row, place, log2 of the height
    WorkList list;
    uint32_t tmem;
    int issued;                                            // steps whose products the first CTA has issued
    int gave_up;
};

__device__ __forceinline__ int clamp_rows(int n) { return min(max(n, 0), kBlock); }

// Lists the boxes that bring rows [m0, m0 + n) of expert e (n <= 128) to a
// CTA: the part of each segment in up to two boxes of the largest power of
// two that fits, which may overlap (the same rows to the same places).
// Returns their number, or more than kBoxes if they are too many.  Called by
// a whole warp; bytes gets the sum of their sizes (box null: counted only).
__device__ __forceinline__ int list_boxes(int3 *box, const ExpertArgs &a, int e, int m0, int n, uint32_t &bytes) {
    const Dims &d = a.d;
    const int lane = threadIdx.x & 31, R = (int)d.R, Tr = (int)d.Tr;
    int before = 0, boxes = 0;
    bytes = 0;
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
        const int lo = max(end - c, m0), hi = min(end, m0 + n), len = max(hi - lo, 0);
        const int lg = 31 - __clz(len | 1), size = 1 << lg;
        const int mine = len == 0 ? 0 : len == size ? 1 : 2;
        // boxes of the lanes before, from two ballots
        const unsigned one = __ballot_sync(kFull, mine >= 1), two = __ballot_sync(kFull, mine == 2);
        const int at = boxes + __popc(one & lanemask_lt()) + __popc(two & lanemask_lt());
        boxes += __popc(one) + __popc(two);
        const int row = (e * R + r) * Tr + lo - (end - c);
        if (box && mine >= 1 && at < kBoxes) box[at] = make_int3(row, lo - m0, lg);
        if (box && mine == 2 && at + 1 < kBoxes) box[at + 1] = make_int3(row + len - size, lo - m0 + len - size, lg);
        bytes += __reduce_add_sync(kFull, (unsigned)(mine * size * kBlock));
    }
    __syncwarp();
    return boxes;
}

template <bool SWIGLU>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kExpertThreads, 1)
    expert_kernel(const __grid_constant__ ExpertArgs a, const __grid_constant__ ExpertMaps maps) {
    extern __shared__ __align__(1024) unsigned char raw[];    // (the only shared memory: it starts at its window's start)
    ExpertShared &s = *reinterpret_cast<ExpertShared *>(raw);
    constexpr int S = kStages, NB = 2;
    static_assert(offsetof(ExpertShared, boxes) % 8 == 0 && offsetof(ExpertShared, w_scale) % 8 == 0, "");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();                           // place in the pair
    const int kb_n = (int)(a.K / kBlock);
    const int n_cols = (int)(SWIGLU ? a.N / 2 : a.N);               // output columns
    const int tile_cols = SWIGLU ? kBlock : NB * kBlock;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&s.boxes[i], 1);
            mbar_init(&s.rows_full[i], kCopyWarps * 32);
            mbar_init(&s.full[i], 2);      // word of both CTAs
            mbar_init(&s.done[i], 2);      // the products' commit, word of this CTA's operands
        }
        for (int i = 0; i < 2; ++i) mbar_init(&s.tempty[i], 16);   // (the first CTA's) the accumulating warps of both
        for (int i = 0; i < kPlans; ++i) {
            mbar_init(&s.plan_full[i], 1);
            mbar_init(&s.plan_empty[i], kPlanUsers);
        }
        mbar_init(&s.joined, 8);
        s.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<2>(&s.tmem);
    make_list(s.list, a, kPairRows, kExpertThreads);
    tmem_fence_before();
    __syncthreads();
    cluster_sync();    // the other CTA's barriers are there too
    tmem_fence_after();
    const uint32_t tmem = s.tmem;
    const Patience patience{&s.gave_up, a.wait_clocks};

    // the next unit's plan, for a whole warp; false after the last one (or where patience ran out)
    int slot = 0, pph = 0;
    bool ok = true;
    const auto next_plan = [&]() {
        ok = warp_wait(&s.plan_full[slot], pph, patience);
        return ok && s.plan[slot].e >= 0;
    };
    const auto plan_used = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.plan_empty[slot]);
        if (++slot == kPlans) { slot = 0; pph ^= 1; }
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 0) {
            // ---- boxes: the matrix rows, and the rows where few boxes bring them ----
            int st = 0, ph = 1, it = 0;
            for (; next_plan(); plan_used()) {
                const Plan &v = s.plan[slot];
                const int3 x = s.box[slot][lane & (kBoxes - 1)];
                const bool mine = lane < v.boxes;
                const uint32_t expect = v.expect;
                const int e = v.e, w_row = v.nb * tile_cols + rank * (SWIGLU ? n_cols : kBlock);
                for (int kb = 0; kb < kb_n; ++kb, ++it) {
                    ok = warp_wait(&s.done[st], ph, patience);
                    if (!ok) break;
                    if (lane == 0) mbar_expect_tx(&s.boxes[st], expect);
                    __syncwarp();
                    if (mine)
                        tma_load_2d(s.buf[st] + x.y * kBlock, &maps.a[x.z], kb * kBlock, x.x, &s.boxes[st]);
                    else if (lane == 31)
                        tma_load_3d(s.buf[st] + kOperand, &maps.w, kb * kBlock, w_row, e, &s.boxes[st]);
                    if (++st == S) { st = 0; ph ^= 1; }
                }
                if (!ok) break;
            }
            drain(s.boxes, S, it);
            __syncwarp();
        } else if (warp == 1) {
            // ---- products (the loop is the whole warp's, so that its values are uniform; one lane issues) ----
            constexpr uint32_t idesc = mma_idesc(kPairRows, NB * kBlock);
            const bool issue = elect_one();
            const uint64_t desc = smem_desc(s.buf[0]);
            int st = 0, ph = 0, acc = 0, aph = 1, it = 0;
            for (; next_plan(); plan_used()) {
                for (int kb = 0; kb < (rank == 0 ? kb_n : 0); ++kb, ++it) {
                    ok = warp_wait<true>(&s.full[st], ph, patience) && warp_wait<true>(&s.tempty[acc], aph, patience);
                    if (!ok) break;
                    acquire_shared_of_cluster();
                    tmem_fence_after();
                    if (issue) {
                        const uint64_t da = desc + (uint32_t)(st * (2 * kOperand >> 4)), db = da + (kOperand >> 4);
#pragma unroll
                        for (int k = 0; k < 4; ++k)   // 32 channels each
                            mma_f8<2>(tmem + acc * 256, da + k * 2, db + k * 2, idesc, k > 0);
                        mma_commit<2>(&s.done[st]);
                    }
                    if (++st == S) { st = 0; ph ^= 1; }
                    acc ^= 1;
                    aph ^= acc == 0;
                }
                if (!ok) break;
            }
            if (rank == 0 && lane < 2) store_cluster(cluster_addr(&s.issued, lane), it);
            __syncwarp();
        } else if (warp == 2) {
            // ---- word of this CTA's boxes, copied rows and scales: to this CTA's accumulation, which reads the scales
            // with ordinary loads (the commit's arrival tells of the products), and to the first CTA's products ----
            const uint32_t full = cluster_addr(&s.full[0], 0);
            int st = 0, ph = 0;
            for (; next_plan(); plan_used()) {
                for (int kb = 0; kb < kb_n; ++kb) {
                    ok = warp_wait(&s.rows_full[st], ph, patience) && warp_wait(&s.boxes[st], ph, patience);
                    if (!ok) break;
                    fence_async_shared();
                    if (lane == 0) {
                        mbar_arrive(&s.done[st]);
                        release_shared_to_cluster();
                        mbar_arrive_relaxed_cluster(full + st * 8);
                    }
                    if (++st == S) { st = 0; ph ^= 1; }
                }
                if (!ok) break;
            }
        } else {
            // ---- plans ----
            const int E = (int)a.d.E, col_tiles = (n_cols + tile_cols - 1) / tile_cols;
            const int units = s.list.first[E] * col_tiles;     // below 2^31: checked on the host
            int u = blockIdx.x >> 1;
            while (true) {
                // (after a round of the plans, the users of the one before have finished with it)
                ok = warp_wait(&s.plan_empty[slot], pph ^ 1, patience);
                if (!ok) break;
                const bool more = u < units;
                if (more) {
                    const Unit v = find_unit(s.list, E, kPairRows, col_tiles, u);
                    const int m0 = v.m0 + rank * kBlock, n = clamp_rows(v.rows - rank * kBlock);
                    uint32_t bytes, other;
                    const int boxes = list_boxes(s.box[slot], a, v.e, m0, n, bytes);
                    const int most = max(boxes, list_boxes(nullptr, a, v.e, v.m0 + (rank ^ 1) * kBlock,
                                                           clamp_rows(v.rows - (rank ^ 1) * kBlock), other));
                    const int m[4] = {m0 + lane, m0 + lane + 32, m0 + lane + 64, m0 + lane + 96};
                    int row[4];
                    receive_rows(a, v.e, m, row);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s.row[slot][lane + 32 * i] = row[i];
                    if (lane == 0)
                        s.plan[slot] = Plan{v.e, v.nb, n, most <= kBoxes ? boxes : -1,
                                            kOperand + (most <= kBoxes ? bytes : 0)};
                } else if (lane == 0) {
                    s.plan[slot].e = -1;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.plan_full[slot]);
                if (!more) break;
                if (++slot == kPlans) { slot = 0; pph ^= 1; }
                u += gridDim.x >> 1;
            }
        }
    } else if (warp < 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
        // ---- rows and scales: eight lanes copy a row's 128 bytes, warp w rows 4 w .. 4 w + 3 of every 16 ----
        constexpr int kStep = kCopyWarps * 4, kMine = kBlock / kStep;
        static_assert(kMine == 8, "32 rows a warp: one scale a lane");
        const int part = (warp - 4) * 4 + (lane >> 3), piece = lane & 7;
        const int place = (lane >> 2) * kStep + (warp - 4) * 4 + (lane & 3);      // the row whose scale this lane copies
        const uint32_t K = (uint32_t)a.K;
        int st = 0, ph = 1, ring = 0;
        for (; next_plan(); plan_used()) {
            const Plan &v = s.plan[slot];
            const int n = v.rows, copies = (v.boxes < 0 ? n : 0) - part;
            const int *rows = s.row[slot];
            // offsets of the scales, in blocks of 128 channels (below 2^32: 128 bytes of an operand have one)
            const uint32_t sc = (uint32_t)rows[place] * kb_n;
            const int n_blocks = (int)((a.N + kBlock - 1) / kBlock), blk = SWIGLU ? v.nb : v.nb * NB;
            uint32_t ws = (uint32_t)(v.e * n_blocks + blk) * kb_n;
            if (lane == 1) ws += SWIGLU ? n_blocks / 2 * kb_n : blk + 1 < n_blocks ? kb_n : 0;   // (zeros beyond N)
            for (int kb = 0; kb < kb_n; ++kb) {
                ok = warp_wait(&s.done[st], ph, patience);
                if (!ok) break;
                const uint32_t dst = smem_addr(s.buf[st]) + part * kBlock + ((piece ^ (part & 7)) << 4);
                const uint8_t *src = a.a + kb * kBlock + piece * 16;
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    if (i * kStep < copies)
                        cp_async16(dst + i * kStep * kBlock, src + (uint64_t)(uint32_t)rows[i * kStep + part] * K);
                if (place < n) cp_async4(smem_addr(&s.row_scale[ring][place]), a.a_scales + (sc + kb));
                if (warp == 4 && lane < 2) cp_async4(smem_addr(&s.w_scale[ring][lane]), a.w_scales + (ws + kb));
                cp_async_arrive(&s.rows_full[st]);
                if (++st == S) { st = 0; ph ^= 1; }
                ring = (ring + 1) % kScaleRing;
            }
            if (!ok) break;
        }
        cp_async_wait_all();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAccRegs));
        // ---- accumulation: thread = row, warpgroup = 64 of each block's 128 columns ----
        const int half = (warp - 8) >> 2, quarter = warp & 3;
        const int r = quarter * 32 + lane;
        const uint32_t tm = tmem + (uint32_t)(quarter * 32) * 65536 + half * 64;
        const uint32_t tempty = cluster_addr(&s.tempty[0], 0);
        // 32-byte stores where rows start at multiples of 32 bytes (a thread stores along its row, so that a warp's
        // store touches 32 lines: 16 bytes each took twice as many)
        const bool wide = SWIGLU ? ((uintptr_t)a.q & 31) == 0 : ((uintptr_t)a.y & 31) == 0 && n_cols % 16 == 0;
        // Arrivals on tempty order no memory and need not: they say that this warp's loads from tensor memory are
        // complete, and the fences of tcgen05 before them and after the products' wait order tensor memory.  (Releases
        // at cluster scope here, by 16 warps a step, took 4.6 ms in place of 1.75.)  The scales
        // of a step, which the copies of a later one overwrite, were read into registers eight steps before the release
        // that those copies wait for (kScaleRing - kStages - 2).
        int it = 0, unit = 0;       // (one counter of steps: registers are short here)
        for (; next_plan(); plan_used(), ++unit) {
            const bool some = quarter * 32 < s.plan[slot].rows;     // rows in this warp's lanes
            uint64_t acc[NB][32];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < 32; ++c) acc[b][c] = 0;
            for (int end = it + kb_n; it < end; ++it) {
                ok = warp_wait(&s.done[it % S], it / S & 1, patience);
                if (!ok) break;
                const int p = it & 1, ring = it % kScaleRing;
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
                            if (lane == 0) mbar_arrive_relaxed_cluster(tempty + p * 8);
                        }
#pragma unroll
                        for (int c = 0; c < 32; ++c) fma2(acc[b][c], pair2(t[2 * c], t[2 * c + 1]), sc[b]);
                    }
                } else if (lane == 0) {
                    mbar_arrive_relaxed_cluster(tempty + p * 8);
                }
            }
            if (!ok) break;
            const Plan &v = s.plan[slot];
            const bool live = r < v.rows;
            const int64_t row = s.row[slot][r];
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
                ok = warp_wait(&s.joined, unit & 1, patience);
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
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t *p = o + 8 * c;
                        if (wide) {
                            const uint32_t v8[8] = {p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7]};
                            st_v8(q + 32 * c, v8);
                        } else {
                            st_v4(q + 32 * c, make_uint4(p[0], p[1], p[2], p[3]));
                            st_v4(q + 32 * c + 16, make_uint4(p[4], p[5], p[6], p[7]));
                        }
                    }
                    if (half == 0) a.q_scales[row * (n_cols / kBlock) + v.nb] = amax / 448.f;
                }
            } else if (live) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int n0 = v.nb * tile_cols + b * kBlock + half * 64;
                    uint16_t *y = a.y + row * a.N + n0;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = pack_bf16x2(lo2(acc[b][8 * c + i]), hi2(acc[b][8 * c + i]));
                        if (wide) {
                            if (n0 + 16 * c < n_cols) st_v8(y + 16 * c, o);
                        } else {
                            if (n0 + 16 * c < n_cols) st_v4(y + 16 * c, make_uint4(o[0], o[1], o[2], o[3]));
                            if (n0 + 16 * c + 8 < n_cols) st_v4(y + 16 * c + 8, make_uint4(o[4], o[5], o[6], o[7]));
                        }
                    }
                }
            }
        }
    }
    tmem_fence_before();
    __syncthreads();
    cluster_sync();    // the other CTA's threads arrive here no more, and its boxes have landed
    if (warp == 1) {
        drain(s.done, S, s.issued);      // products read both CTAs' shared memory and arrive in both
        __syncwarp();
        tmem_fence_after();
        tmem_free<2>(tmem);
    }
    if (threadIdx.x == 0 && s.gave_up) raise_status(a.dev_status, EP_STATUS_TIMEOUT);
}

template <bool SWIGLU>
cudaError_t launch(const ExpertArgs &a, const ExpertMaps &maps, cudaStream_t st) {
    constexpr int bytes = sizeof(ExpertShared);
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
    expert_kernel<SWIGLU><<<num_sms() & ~1, kExpertThreads, bytes, st>>>(a, maps);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_many(const ExpertArgs &a, cudaStream_t st) {
    ExpertMaps maps;
    const cuuint64_t dims[2] = {(cuuint64_t)a.K, (cuuint64_t)(a.d.E * a.d.T)}, strides[1] = {(cuuint64_t)a.K};
    for (int i = 0; i < 8; ++i) {
        const cuuint32_t box[2] = {kBlock, 1u << i};
        if (cudaError_t e = encode_map(&maps.a[i], 2, a.a, dims, strides, box)) return e;
    }
    if (cudaError_t e = matrix_map(a, kBlock, &maps.w)) return e;
    return a.q ? launch<true>(a, maps, st) : launch<false>(a, maps, st);
}

}  // namespace ep
