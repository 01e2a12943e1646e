// A whole mixture-of-experts layer for a few tokens (ep_moe_few), in three
// launches: routing and the cast of the tokens; the gate and up products, SwiGLU
// and its cast; the down products and the weighted sum.
//
//   idx, w = route(logits);  a = e4m3(x);  h = e4m3(silu(a G_e^T) * (a U_e^T));
//   out[t] = residual[t] + sum_j w[t, j] (h D_e^T)[t, j],   e = idx[t, j]
//
// With a few tokens the time is that of reading the chosen experts' matrices
// once; what a layer made of separate calls adds is their latency and the
// receive buffers between them.  So the launches overlap: each begins while the one before
// it ends and does what needs nothing of it (tensor memory, barriers; the third, whose experts
// are known by then, fills its stages with matrix rows), and the second asks for the third's first rows towards
// L2.  Each CTA lists the chosen experts itself.  As in the products for few rows an
// expert, 128 matrix rows are the tensor core's M and the expert's tokens its N
// (16, 32, 48 or 64), every block of 128 channels is one accumulation in tensor
// memory, and a thread owns a matrix row and scales and adds the blocks in fp32.
//
// First launch: a CTA of each token routes it, the others cast the tokens (as ep_dispatch does, each rounding
// included) and zero the counters.
// Second launch: a unit of work is 128 columns of h, which are one block of its cast.  Both products of
// those columns land in the same thread.
// Third launch: a unit is 128 output columns of one expert.  Its products, in fp32, go
// to y [T, k, H] in the workspace; a CTA has a run of units, column tile after
// column tile; the one that brings a tile's last expert (a counter of units for each
// tile) adds the tile's k rows of each token in the order j = 0 .. k - 1.  So the sum does not depend on who comes
// last, and y is never rounded.  y is T k H 4 bytes against the experts' 3 I H each.
//
// Measured, from a graph, 256 experts of 7168 x 2048, 8 a token: one token 72 us (352 MB, 4.8 TB/s; the latency of three
// launches that fill and drain, 19 us at the smallest sizes), 32 tokens 0.97 to 0.99 ms (7.2 GB, 7.2 to 7.4 TB/s: at the memory's
// rate); 61 tokens, 64 experts of 4096 x 1408, 6 a token 196 us (1.1 GB, 5.6 TB/s).  One cooperative launch for the last two took
// 0 to 10% longer.
#include <algorithm>
#include <cstddef>

#include "launch_order.cuh"
#include "route_device.cuh"
#include "tcgen05.cuh"

namespace ep {

namespace {

constexpr int kBlock = 128;                     // channels, and matrix rows, of a scale
constexpr int kOperand = kBlock * kBlock;       // bytes of 128 matrix rows x 128 channels
constexpr int kThreads = 512;                   // warpgroup 0: boxes and products; 1: rows; 2, 3: accumulation
constexpr int kIssueRegs = 80, kCopyRegs = 80, kAccRegs = 176;   // 80 + 80 + 2 * 176 = 4 * 128, the launch's registers
constexpr int kRows = kMoeFewTokens;            // rows of a tile: an expert has at most one for each token
constexpr int kCopyThreads = 128;
constexpr int kMaxAcc = 16;                     // accumulators, as many as tensor memory holds
constexpr int kMaxStages = 12;                  // operand buffers, as many as shared memory holds
constexpr int kSharedBytes = 227 * 1024;
// Steps whose scales are kept: a step's copies wait for the products `stages`
// steps before, those for the loads of the accumulation kMaxAcc steps before
// them, which may still be using that step's scales.
constexpr int kScaleRing = 32;
static_assert(kMaxStages <= 16 && kMaxAcc == 16, "a lane for each barrier");
static_assert(kScaleRing > kMaxStages + kMaxAcc + 1, "scales are still in use when they are overwritten");

struct MoeBarriers {
    uint64_t boxes[kMaxStages];                             // matrix rows
    uint64_t rows_full[kMaxStages], full[kMaxStages];       // rows and scales; all operands
    uint64_t done[kMaxStages];                              // a step's products: buffers free, sums and scales ready
    uint64_t tempty[kMaxAcc];                                  // accumulators taken out
    uint64_t joined[2];                                     // UP: a warpgroup's maxima are written; else: y is, and who
                                                            // is last is known
    uint64_t split[2];                                      // a part is written, and who is last is known
    float w_scale[kScaleRing][2];
    int last[2], last_part[2];
    uint32_t tmem;
    int n, gave_up;                                         // chosen experts
};

// Shared memory: operands of the stages (matrix rows, then tokens' rows), the barriers, and what has the size of the
// problem.  Few tokens leave room for more stages.
template <bool UP>
struct MoeShared {
    static constexpr int kWBytes = (UP ? 2 : 1) * kOperand;
    unsigned char *w, *rows;             // [stages][kWBytes], [stages][pad][128]
    int rows_bytes;
    MoeBarriers *bar;
    float *row_scale;                    // [kScaleRing][pad]
    uint32_t (*amax)[4];                 // UP: [2 x pad]: [unit parity][row][warp of the warpgroup]
    // The chosen experts and their entries (t * k + j), in the order of the experts and, in an expert, of the tokens
    uint64_t *tokens;                    // [E]: bit t: token t goes to the expert
    float *weight;                       // [T k], not UP
    short *expert, *place, *start;       // [E], [E], [E + 1]
    short *entry, *idx;                  // [T k]
    // Sets the pointers; returns the bytes of the whole.
    __host__ __device__ int carve(unsigned char *base, int stages, int pad, int E, int entries) {
        int at = 0;
        const auto take = [&](int bytes) {
            unsigned char *p = base + at;
            at += (bytes + 15) & ~15;
            return p;
        };
        rows_bytes = pad * kBlock;
        w = take(stages * kWBytes);
        rows = take(stages * rows_bytes);
        bar = reinterpret_cast<MoeBarriers *>(take(sizeof(MoeBarriers)));
        row_scale = reinterpret_cast<float *>(take(kScaleRing * pad * 4));
        amax = reinterpret_cast<uint32_t(*)[4]>(take(UP ? 2 * pad * 16 : 0));
        tokens = reinterpret_cast<uint64_t *>(take(E * 8));
        weight = reinterpret_cast<float *>(take(UP ? 0 : entries * 4));
        expert = reinterpret_cast<short *>(take(E * 2));
        place = reinterpret_cast<short *>(take(E * 2));
        start = reinterpret_cast<short *>(take(E * 2 + 2));
        entry = reinterpret_cast<short *>(take(entries * 2));
        idx = reinterpret_cast<short *>(take(entries * 2));
        return at;
    }
};

// Fills the lists from s.idx, by all threads of the block, in turns of whole warps; complete when it returns.  s.tokens
// are zeros, and both are there for all threads.
template <bool UP>
__device__ __forceinline__ void list_chosen(const MoeShared<UP> &s, int E, int T, int k) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int t = warp; t < T; t += kThreads / 32) {
        const int e = lane < k ? s.idx[t * k + lane] : -1;
        if (e >= 0) atomicOr(reinterpret_cast<unsigned long long *>(&s.tokens[e]), 1ull << t);
    }
    __syncthreads();
    // a warp places 32 experts: how many are chosen, and their rows, in front of them
    const auto rows_of = [&](int e) { return e < E ? __popcll(s.tokens[e]) : 0; };
    int some = 0, rows = 0;
    for (int c = 0; c * 32 < E; ++c) {
        const int mine = rows_of(c * 32 + lane);
        if (c % (kThreads / 32) == warp) {
            const unsigned chosen = __ballot_sync(kFull, mine > 0);
            const int n = (int)__reduce_add_sync(kFull, some) + __popc(chosen & lanemask_lt());
            int inc = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, inc, o);
                if (lane >= o) inc += v;
            }
            inc += (int)__reduce_add_sync(kFull, rows);
            if (mine > 0) {
                s.expert[n] = (short)(c * 32 + lane);
                s.place[c * 32 + lane] = (short)n;
                s.start[n] = (short)(inc - mine);
            }
            if ((c + 1) * 32 >= E && lane == 31) {
                s.start[n + (mine > 0)] = (short)inc;
                s.bar->n = n + (mine > 0);
            }
        }
        some += mine > 0;
        rows += mine;
    }
    __syncthreads();
    for (int t = warp; t < T; t += kThreads / 32) {
        const int e = lane < k ? s.idx[t * k + lane] : -1;
        if (e >= 0) s.entry[s.start[s.place[e]] + __popcll(s.tokens[e] & ((1ull << t) - 1))] = (short)(t * k + lane);
    }
    __syncthreads();
}

// A part of a unit of work: blocks [kb0, kb1) of the contraction of a column tile of an expert
struct MoePart {
    int64_t unit;
    int e, tile, rows, kb0, kb1;
    const short *entry;
};
// A CTA's run of steps, all units' steps laid end to end: of whole units, or in equal runs that may begin and end within
// a unit.  With every CTA at work a step of 32 KB takes 0.69 us; a CTA whose neighbours are done takes 0.45 (measured: 8
// units alone), so that whole units end with a tail in which the memory idles; a split unit costs an exchange of some 4
// us.  (One token's 128 units of 56 steps: 77 us whole, 89 split; 8 such units 47 us whole, 34 split.)
template <bool UP>
struct MoeRun {
    int64_t total, at, end;
    int n;                               // CTAs that have steps (split)
    __device__ __forceinline__ MoeRun(int64_t units, int kb_n) {
        constexpr int kExchange = UP ? 6 : 12, kLeast = UP ? 4 : 8;     // steps: of 4 us, and of a run
        const int64_t ctas = gridDim.x, c = blockIdx.x, all = units * kb_n;
        const int64_t full = units > 0 ? (units - 1) / ctas : 0, rest = units - full * ctas;   // rounds of all, then of the rest
        total = all;
        n = (int)min(ctas, (all + kLeast - 1) / kLeast);
        if (full * kb_n * 100 + kb_n * max((int64_t)65, 100 * rest / ctas) <= 100 * all / ctas + 100 * kExchange) {
            at = units * c / ctas * kb_n;
            end = units * (c + 1) / ctas * kb_n;
        } else {
            at = c < n ? all * c / n : 0;
            end = c < n ? all * (c + 1) / n : 0;
        }
    }
    // the CTA that has a step of a split unit
    __device__ __forceinline__ int owner(int64_t step) const { return (int)(((step + 1) * n - 1) / total); }
};
// the run's next part; what follows it starts at run.at
template <bool UP, typename S>
__device__ __forceinline__ MoePart next_part(const S &s, int tiles, int chosen, int kb_n, MoeRun<UP> &run) {
    MoePart v;
    v.unit = run.at / kb_n;
    v.kb0 = (int)(run.at - v.unit * kb_n);
    v.kb1 = (int)min((int64_t)kb_n, v.kb0 + (run.end - run.at));
    run.at += v.kb1 - v.kb0;
    // second launch: an expert's column tiles follow one another; third: a column tile's experts
    const int at = (int)(UP ? v.unit / tiles : v.unit % chosen);
    v.tile = (int)(UP ? v.unit - (int64_t)at * tiles : v.unit / chosen);
    v.e = s.expert[at];
    v.rows = s.start[at + 1] - s.start[at];
    v.entry = s.entry + s.start[at];
    return v;
}

// out[t, columns of a tile] by the 256 accumulating threads: 4 columns a thread, two tokens a warp at a time; eight rows
// of y of each are under way together
template <bool UP>
__device__ __forceinline__ void combine_tile(const MoeFewArgs &a, const MoeShared<UP> &c, int tile) {
    const int thread = threadIdx.x - 256, col = tile * kBlock + (thread & 31) * 4, k = (int)a.route.k, T = (int)a.route.T;
    const float *y = a.y + col;
    for (int t0 = thread >> 5; t0 < T; t0 += 16) {
        float4 v[2];
        uint2 r[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = t0 + 8 * i;
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            r[i] = make_uint2(0, 0);
            if (a.residual && t < T) r[i] = *reinterpret_cast<const uint2 *>(a.residual + t * a.H + col);
        }
        for (int j0 = 0; j0 < k; j0 += 8) {
            float4 in[2][8];
            float w[2][8];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int t = t0 + 8 * i, at = t * k + j0 + j;
                    in[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
                    w[i][j] = 0.f;
                    if (t < T && j0 + j < k && c.idx[at] >= 0) {
                        in[i][j] = __ldcg(reinterpret_cast<const float4 *>(y + at * a.H));
                        w[i][j] = c.weight[at];
                    }
                }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    v[i].x += w[i][j] * in[i][j].x;
                    v[i].y += w[i][j] * in[i][j].y;
                    v[i].z += w[i][j] * in[i][j].z;
                    v[i].w += w[i][j] * in[i][j].w;
                }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = t0 + 8 * i;
            if (t < T)
                *reinterpret_cast<uint2 *>(a.out + t * a.H + col) =
                    make_uint2(pack_bf16x2(v[i].x + bf16_lo(r[i].x), v[i].y + bf16_hi(r[i].x)),
                               pack_bf16x2(v[i].z + bf16_lo(r[i].y), v[i].w + bf16_hi(r[i].y)));
        }
    }
}

// one box towards L2
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *map, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// a box that is read once
__device__ __forceinline__ void tma_load_once_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint64_t *bar,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
        "[%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar)), "l"(policy)
        : "memory");
}

// Steps of the third launch whose matrix rows the second one asks for ahead, so that the memory has work while it ends and
// the third begins: at most 640 KB a CTA, 97 MB of an L2 of 129.
constexpr int kAhead = 40;

template <bool UP>
__global__ void __launch_bounds__(kThreads, 1)
    moe_few_kernel(const __grid_constant__ MoeFewArgs a, const __grid_constant__ CUtensorMap map_w,
                   const __grid_constant__ CUtensorMap map_next, const int S) {
    extern __shared__ __align__(1024) unsigned char raw[];    // (the only shared memory: it starts at its window's start)
    constexpr int NB = UP ? 2 : 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int T = (int)a.route.T, k = (int)a.route.k, E = (int)a.route.E;
    const int K = (int)(UP ? a.H : a.I), n_cols = (int)(UP ? a.I : a.H), kb_n = K / kBlock, tiles = n_cols / kBlock;
    const int pad = (T + 15) & ~15;
    // Accumulators: 512 columns hold 16 of 16 tokens (UP), 4 of 64.  No more than stages: the accumulation tells a stage's
    // phases apart by their parity, so the products may not be further ahead of it than one round.
    const int accs = min(min(kMaxAcc, S), 512 / (NB * pad));
    MoeShared<UP> s;
    s.carve(raw, S, pad, E, T * k);
    MoeBarriers &bar = *s.bar;

    if (threadIdx.x == 0) asm volatile("prefetch.tensormap [%0];" ::"l"(&map_w) : "memory");
    for (int e = threadIdx.x; e < E; e += kThreads) s.tokens[e] = 0;
    if (warp == 15) {
        if (lane < S) {
            mbar_init(&bar.rows_full[lane], kCopyThreads);    // the copies' own arrivals
            mbar_init(&bar.boxes[lane], 1);
            mbar_init(&bar.full[lane], 1);
            mbar_init(&bar.done[lane], 2);                    // the products' commit, word of the operands
        } else if (lane >= 16) {
            mbar_init(&bar.tempty[lane - 16], 8);
        }
        if (lane == 0) {
            mbar_init(&bar.joined[0], UP ? 4 : 8);
            mbar_init(&bar.joined[1], UP ? 4 : 1);
            mbar_init(&bar.split[0], 8);
            mbar_init(&bar.split[1], 1);
            bar.gave_up = 0;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 14) tmem_alloc<1>(&bar.tmem);
    // The second launch waits for the routing before it lets the third begin, so that one finds the routing there (in L2:
    // it is read past L1) and fills its stages with matrix rows; it waits for the second where it takes h.
    if (UP) {
        wait_for_launch_before();
        let_next_launch_begin();
    }
    for (int i = threadIdx.x; i < T * k; i += kThreads) {
        s.idx[i] = (short)__ldcg(reinterpret_cast<const long long *>(a.route.topk_idx) + i);
        if (!UP) s.weight[i] = __ldcg(a.route.topk_weights + i);
    }
    __syncthreads();
    list_chosen(s, E, T, k);
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = bar.tmem;
    const int chosen = bar.n;
    const MoeRun<UP> whole_run((int64_t)chosen * tiles, kb_n);
    const Patience patience{&bar.gave_up, a.wait_clocks};

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 0) {
            // ---- matrix rows ----
            if (lane == 0) {
                const uint64_t once = l2_policy<1>();
                int st = 0, ph = 1, it = 0;
                bool ok = true;
                for (MoeRun<UP> run = whole_run; run.at < run.end && ok;) {
                    const MoePart v = next_part<UP>(s, tiles, chosen, kb_n, run);
                    for (int kb = v.kb0; kb < v.kb1; ++kb, ++it) {
                        ok = mbar_wait(&bar.done[st], ph, patience);
                        if (!ok) break;
                        mbar_expect_tx(&bar.boxes[st], NB * kOperand);
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            tma_load_once_3d(s.w + st * (NB * kOperand) + b * kOperand, &map_w, kb * kBlock,
                                             v.tile * kBlock + b * n_cols, v.e, &bar.boxes[st], once);
                        if (++st == S) { st = 0; ph ^= 1; }
                    }
                }
                if (UP) {
                    const int next_kb = (int)(a.I / kBlock), next_tiles = (int)(a.H / kBlock);
                    int left = kAhead;
                    for (MoeRun<false> run((int64_t)chosen * next_tiles, next_kb); run.at < run.end && left > 0;) {
                        const MoePart v = next_part<false>(s, next_tiles, chosen, next_kb, run);
                        for (int kb = v.kb0; kb < v.kb1 && left > 0; ++kb, --left)
                            tma_prefetch_3d(&map_next, kb * kBlock, v.tile * kBlock, v.e);
                    }
                }
                drain(bar.boxes, S, it);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ---- products (the loop is the whole warp's, so that its values are uniform; one lane issues) ----
            const bool issue = elect_one();
            const uint64_t dw = smem_desc(s.w), dr = smem_desc(s.rows);
            int st = 0, ph = 0, acc = 0, aph = 1, it = 0;
            bool ok = true;
            for (MoeRun<UP> run = whole_run; run.at < run.end && ok;) {
                const MoePart v = next_part<UP>(s, tiles, chosen, kb_n, run);
                const uint32_t idesc = mma_idesc(kBlock, (v.rows + 15) & ~15);
                for (int kb = v.kb0; kb < v.kb1; ++kb, ++it) {
                    ok = warp_wait(&bar.full[st], ph, patience) && warp_wait(&bar.tempty[acc], aph, patience);
                    if (!ok) break;
                    tmem_fence_after();
                    if (issue) {
                        const uint64_t da = dw + (uint32_t)(st * (NB * kOperand >> 4));
                        const uint64_t db = dr + (uint32_t)(st * (s.rows_bytes >> 4));
#pragma unroll
                        for (int b = 0; b < NB; ++b)
#pragma unroll
                            for (int i = 0; i < 4; ++i)   // 32 channels a step
                                mma_f8<1>(tmem + (acc * NB + b) * pad, da + (b * (kOperand >> 4) + i * 2), db + i * 2,
                                          idesc, i > 0);
                        mma_commit<1>(&bar.done[st]);
                    }
                    if (++st == S) { st = 0; ph ^= 1; }
                    if (++acc == accs) { acc = 0; aph ^= 1; }
                }
            }
            drain(bar.done, S, it);
            __syncwarp();
        } else if (warp == 2) {
            // ---- word of the operands: to the products, and to the accumulation, which reads the scales with
            // ordinary loads (the commit's arrival tells of the products) ----
            if (lane == 0) {
                int st = 0, ph = 0;
                for (int64_t at = whole_run.at; at < whole_run.end; ++at) {
                    if (!mbar_wait(&bar.rows_full[st], ph, patience) || !mbar_wait(&bar.boxes[st], ph, patience)) break;
                    fence_async_shared();
                    mbar_arrive(&bar.done[st]);
                    mbar_arrive(&bar.full[st]);
                    if (++st == S) { st = 0; ph ^= 1; }
                }
            }
            __syncwarp();
        }
    } else if (warp < 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
        if (!UP) wait_for_launch_before();
        // ---- rows and scales: eight lanes bring a row's 128 channels ----
        constexpr int kPass = kCopyThreads / 8, kMine = kRows / kPass;
        const int part = (threadIdx.x - 128) >> 3, piece = lane & 7;
        const int place = (threadIdx.x - 128) & (kRows - 1);      // the row whose scale this thread copies, if below 64
        const int n_blocks = NB * tiles;                          // of the matrix's rows
        int st = 0, ph = 1, ring = 0;
        bool ok = true;
        for (MoeRun<UP> run = whole_run; run.at < run.end && ok;) {
            const MoePart v = next_part<UP>(s, tiles, chosen, kb_n, run);
            uint32_t ws = (uint32_t)(v.e * n_blocks + v.tile) * kb_n;
            if (lane == 1) ws += (uint32_t)tiles * kb_n;          // (the up block's)
            const uint32_t swizzled = part * kBlock + ((piece ^ (part & 7)) << 4);
            int row[kMine];                                       // tokens, or entries
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                const int r = i * kPass + part;
                row[i] = r < v.rows ? (UP ? v.entry[r] / k : v.entry[r]) : 0;
            }
            const int scale_row = warp < 6 && place < v.rows ? (UP ? v.entry[place] / k : v.entry[place]) : -1;
            const float *row_scales = (UP ? a.x_scales : a.h_scales) + (int64_t)scale_row * kb_n;
            const float *w_scales = (UP ? a.gate_up_scales : a.down_scales) + ws;
            const uint8_t *src = (UP ? a.xq : a.h) + piece * 16;
            for (int kb = v.kb0; kb < v.kb1; ++kb) {
                ok = warp_wait(&bar.done[st], ph, patience);
                if (!ok) break;
                const uint32_t dst = smem_addr(s.rows + st * s.rows_bytes) + swizzled;
#pragma unroll
                for (int i = 0; i < kMine; ++i)
                    if (i * kPass + part < v.rows)
                        cp_async16(dst + i * kPass * kBlock, src + (int64_t)row[i] * K + kb * kBlock);
                if (scale_row >= 0) cp_async4(smem_addr(&s.row_scale[ring * pad + place]), row_scales + kb);
                if (warp == 7 && lane < NB) cp_async4(smem_addr(&bar.w_scale[ring][lane]), w_scales + kb);
                cp_async_arrive(&bar.rows_full[st]);
                if (++st == S) { st = 0; ph ^= 1; }
                ring = (ring + 1) % kScaleRing;
            }
        }
        cp_async_wait_all();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAccRegs));
        // ---- accumulation: thread = matrix row (UP: of the gate's and of the up block); a warpgroup has every other 16
        // columns (rows of the tile) ----
        constexpr int kMine = kRows / 2;
        const int half = (warp - 8) >> 2, quarter = warp & 3;
        const int chan = quarter * 32 + lane;
        const auto column = [&](int c) { return ((c >> 4) * 2 + half) * 16 + (c & 15); };   // my c-th column
        const uint32_t tm = tmem + (uint32_t)(quarter * 32) * 65536;
        if (!UP) wait_for_launch_before();                   // (before anything is written, and before this launch ends)
        const int thread = threadIdx.x - 256;
        int st = 0, ph = 0, p = 0, ring = 0;
        int parts = 0, unit = 0, word = 0, mine = 0;         // (mine: units of this column tile that ended here)
        bool ok = true;
        for (MoeRun<UP> run = whole_run; run.at < run.end && ok;) {
            const MoePart v = next_part<UP>(s, tiles, chosen, kb_n, run);
            uint64_t acc[NB][kMine / 2];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < kMine / 2; ++c) acc[b][c] = 0;
            for (int kb = v.kb0; kb < v.kb1; ++kb) {
                ok = warp_wait(&bar.done[st], ph, patience);
                if (!ok) break;
                tmem_fence_after();
                uint32_t t[NB * kMine];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int q = 0; q < kMine / 16; ++q)
                        if (column(q * 16) < v.rows)
                            tmem_ld16(tm + (p * NB + b) * pad + column(q * 16), t + b * kMine + q * 16);
                tmem_wait_ld<NB * kMine>(t);
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.tempty[p]);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint32_t w32 = __float_as_uint(bar.w_scale[ring][b]);
                    const uint64_t sw = pair2(w32, w32);
#pragma unroll
                    for (int q = 0; q < kMine / 16; ++q) {
                        if (column(q * 16) >= v.rows) break;
                        const ulonglong2 *sr = reinterpret_cast<const ulonglong2 *>(&s.row_scale[ring * pad + column(q * 16)]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const ulonglong2 x = sr[c];
                            const int i = q * 16 + c * 4;
                            const uint32_t *d = t + b * kMine + i;
                            fma2(acc[b][i / 2], pair2(d[0], d[1]), mul2(x.x, sw));
                            fma2(acc[b][i / 2 + 1], pair2(d[2], d[3]), mul2(x.y, sw));
                        }
                    }
                }
                if (++st == S) { st = 0; ph ^= 1; }
                if (++p == accs) p = 0;
                ring = (ring + 1) % kScaleRing;
            }
            if (!ok) break;
            bool complete = true;
            if (v.kb1 - v.kb0 < kb_n) {
                // A part of the unit's contraction: written down, and counted in steps with the CTA that has the first.  Who
                // brings the last adds the parts, in the order of the contraction.
                const int c0 = run.owner(v.unit * kb_n), c1 = run.owner(v.unit * kb_n + kb_n - 1), me = blockIdx.x;
                const auto part_of = [&](int c) {
                    return a.parts + (int64_t)(c * 2 + (c == c0)) * moe_part_floats(pad) + thread;
                };
                const int cols = moe_part_columns(pad);
                const auto each = [&](auto f) {
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int c = 0; c < kMine; c += 2)
                            if (column(c) < v.rows) f(acc[b][c / 2], (b * cols + c) * 256);
                };
                float *own = part_of(me);
                each([&](uint64_t &x, int at) {
                    own[at] = lo2(x);
                    own[at + 256] = hi2(x);
                });
                __threadfence();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.split[0]);
                if (warp == 8) {
                    ok = warp_wait(&bar.split[0], parts & 1, patience);
                    if (!ok) break;
                    if (lane == 0) {
                        const unsigned steps = v.kb1 - v.kb0;
                        bar.last_part[parts & 1] = atomicAdd(a.split + (UP ? 0 : kMoeCtas) + c0, steps) + steps == (unsigned)kb_n;
                        __threadfence();
                        mbar_arrive(&bar.split[1]);
                    }
                    __syncwarp();
                }
                ok = warp_wait(&bar.split[1], parts & 1, patience);
                if (!ok) break;
                complete = bar.last_part[parts & 1];
                ++parts;
                if (complete) {
                    const auto add = [&](int from, int to) {
                        // four parts at a time: their loads are under way together
                        for (int c = from; c < to; c += 4) {
                            const float *other[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) other[i] = part_of(min(c + i, to - 1));
                            each([&](uint64_t &x, int at) {
                                float lo[4], hi[4];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    lo[i] = __ldcg(other[i] + at);
                                    hi[i] = __ldcg(other[i] + at + 256);
                                }
                                float l = lo2(x), h = hi2(x);
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (c + i < to) {
                                        l += lo[i];
                                        h += hi[i];
                                    }
                                x = pair2(__float_as_uint(l), __float_as_uint(h));
                            });
                        }
                    };
                    if (me > c0) {                       // (mine is in its place in the order again)
                        each([&](uint64_t &x, int) { x = 0; });
                        add(c0, me + 1);
                    }
                    add(me + 1, c1 + 1);
                }
            }
            if (UP) {
                if (!complete) continue;
                // h of my columns; their maxima over the warp's 32 channels, then over the four warps
                uint32_t top = 0;                          // lane c: of column c
#pragma unroll
                for (int c = 0; c < kMine; ++c) {
                    if (column(c) >= v.rows) break;
                    const float g = c & 1 ? hi2(acc[0][c / 2]) : lo2(acc[0][c / 2]);
                    const float w = c & 1 ? hi2(acc[NB - 1][c / 2]) : lo2(acc[NB - 1][c / 2]);
                    const uint32_t bits = __float_as_uint(swiglu(g, w));
                    acc[0][c / 2] = c & 1 ? (acc[0][c / 2] & 0xffffffffull) | (uint64_t)bits << 32
                                          : (acc[0][c / 2] & ~0xffffffffull) | bits;
                    const uint32_t x = __reduce_max_sync(kFull, bits & 0x7fffffffu);   // (NaN above all numbers)
                    if (lane == c) top = x;
                }
                const int at = column(lane);
                uint32_t(*amax)[4] = s.amax + (unit & 1) * pad;     // (a warp a unit ahead writes to the other)
                if (at < v.rows) amax[at][quarter] = top;
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.joined[half]);
                ok = warp_wait(&bar.joined[half], unit & 1, patience);
                if (!ok) break;
                float inv = 0.f;                           // lane c: of column c
                if (at < v.rows) {
                    const uint4 t4 = *reinterpret_cast<const uint4 *>(amax[at]);
                    const float most = __uint_as_float(max(max(t4.x, t4.y), max(t4.z, t4.w)));
                    inv = most > 0.f ? fminf(448.f / most, kMaxFinite) : 0.f;
                    if (quarter == 0) a.h_scales[(int64_t)v.entry[at] * tiles + v.tile] = most / 448.f;
                }
                uint8_t *q = a.h + v.tile * kBlock + chan;
#pragma unroll
                for (int c = 0; c < kMine; ++c) {
                    if (column(c) >= v.rows) break;
                    const float h = c & 1 ? hi2(acc[0][c / 2]) : lo2(acc[0][c / 2]);
                    q[(int64_t)v.entry[column(c)] * n_cols] =
                        (uint8_t)pack_e4m3x2(h * __shfl_sync(kFull, inv, c), 0.f);
                }
                ++unit;
            } else {
                float *y = a.y + v.tile * kBlock + chan;
#pragma unroll
                for (int c = 0; c < kMine; ++c) {
                    if (!complete || column(c) >= v.rows) break;
                    y[(int64_t)v.entry[column(c)] * n_cols] = c & 1 ? hi2(acc[0][c / 2]) : lo2(acc[0][c / 2]);
                }
                // The last of my units of this tile: count them.  Everybody's y is out before, and in before it is read.
                mine += complete;
                if (mine == 0 || (run.at < run.end && run.at / kb_n / chosen == v.tile)) continue;
                __threadfence();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.joined[0]);
                if (warp == 8) {
                    ok = warp_wait(&bar.joined[0], word & 1, patience);
                    if (!ok) break;
                    if (lane == 0) {
                        bar.last[word & 1] = atomicAdd(a.arrived + v.tile, (unsigned)mine) + mine == (unsigned)chosen;
                        __threadfence();
                        mbar_arrive(&bar.joined[1]);
                    }
                    __syncwarp();
                }
                ok = warp_wait(&bar.joined[1], word & 1, patience);
                if (!ok) break;
                if (bar.last[word & 1]) combine_tile(a, s, v.tile);
                ++word;
                mine = 0;
            }
        }
        if (!UP && chosen == 0)                              // no token has an expert
            for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) combine_tile(a, s, tile);
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 14) {
        tmem_fence_after();
        tmem_free<1>(tmem);
    }
    if (threadIdx.x == 0 && bar.gave_up) raise_status(a.route.dev_status, EP_STATUS_TIMEOUT);
}

struct MoeMaps {
    CUtensorMap gate_up, down;
};
cudaError_t moe_map(const MoeFewArgs &a, const void *w, int64_t N, int64_t K, CUtensorMap *map) {
    const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)a.route.E};
    const cuuint64_t strides[2] = {(cuuint64_t)K, (cuuint64_t)(N * K)};
    const cuuint32_t box[3] = {kBlock, kBlock, 1};
    return encode_map(map, 3, w, dims, strides, box);
}

template <bool UP>
cudaError_t launch(const MoeFewArgs &a, const MoeMaps &maps, cudaStream_t st) {
    const int T = (int)a.route.T, pad = (T + 15) & ~15;
    MoeShared<UP> s;
    int stages = kMaxStages;
    while (s.carve(nullptr, stages, pad, (int)a.route.E, T * (int)a.route.k) > kSharedBytes) --stages;   // (4 at least)
    static std::atomic<int> ready[kCacheDevices];
    cudaError_t e = cudaSuccess;
    cached_per_device(ready, [&](int) {
        e = cudaFuncSetAttribute(moe_few_kernel<UP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kSharedBytes);
        // the warpgroups' register shares are drawn from what the block was launched with
        cudaFuncAttributes f{};
        if (!e) e = cudaFuncGetAttributes(&f, moe_few_kernel<UP>);
        if (!e && f.numRegs * 4 < kIssueRegs + kCopyRegs + 2 * kAccRegs) e = cudaErrorInvalidDeviceFunction;
        return e == cudaSuccess ? 1 : 0;
    });
    if (e) return e;
    // it begins while the launch before it ends, and waits before it reads what that one wrote
    return launch_in_order(kAfter, moe_few_kernel<UP>, dim3((unsigned)std::min(num_sms(), kMoeCtas)), kThreads,
                           s.carve(nullptr, stages, pad, (int)a.route.E, T * (int)a.route.k), 0, st, a,
                           UP ? maps.gate_up : maps.down, maps.down, stages);
}

}  // namespace

namespace {

constexpr int kCastThreads = 128;

// The first launch: a CTA of each token routes it (its first warp; its lanes hold up to V experts, entry j goes to lane
// j), the others cast 16 blocks of 128 channels each, as ep_dispatch does.
template <int V, int KEY>
__global__ void __launch_bounds__(kCastThreads) moe_few_start_kernel(const __grid_constant__ MoeFewArgs a, const LaneMap map) {
    let_next_launch_begin();
    const RouteArgs &r = a.route;
    const int t = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (blockIdx.x == 0) {
        if (warp == 0) {
            const int lo = map.first(lane), held = map.count(lane), k = (int)r.k;
            const uint16_t *half = reinterpret_cast<const uint16_t *>(r.logits) + t * r.stride;
            const float *full = reinterpret_cast<const float *>(r.logits) + t * r.stride;
            const auto logit = [&](int e) { return r.bf16 ? widen(__ldg(half + e)) : __ldg(full + e); };
            float x[V], b[V], weight;
            int id;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[i] = i < held ? logit(lo + i) : -INFINITY;
                b[i] = i < held && r.bias ? __ldg(r.bias + lo + i) : 0.f;
            }
            route_one<V, KEY>(r, map, x, b, logit, id, weight);
            if (lane < k) {
                r.topk_idx[t * k + lane] = id;
                r.topk_weights[t * k + lane] = weight;
            }
        } else if (t == 0) {
            for (int i = threadIdx.x - 32; i < (int)(a.H / kBlock); i += kCastThreads - 32) a.arrived[i] = 0;
            for (int i = threadIdx.x - 32; i < 2 * kMoeCtas; i += kCastThreads - 32) a.split[i] = 0;
        }
        return;
    }
    const int block = ((int)blockIdx.x - 1) * 16 + (threadIdx.x >> 3), piece = lane & 7, blocks = (int)(a.H / kBlock);
    float f[16], amax = 0.f;
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (block < blocks) {
        const uint4 *from = reinterpret_cast<const uint4 *>(a.x + t * a.H + block * kBlock + piece * 16);
        x = ld_stream(from);
        y = ld_stream(from + 1);
    }
    const uint32_t w8[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        f[2 * c] = bf16_lo(w8[c]);
        f[2 * c + 1] = bf16_hi(w8[c]);
        amax = fmaxf(amax, fmaxf(fabsf(f[2 * c]), fabsf(f[2 * c + 1])));
    }
#pragma unroll
    for (int o = 4; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    const float inv = amax > 0.f ? fminf(__fdiv_rn(448.f, amax), kMaxFinite) : 0.f;
    uint32_t q[4];
#pragma unroll
    for (int c = 0; c < 4; ++c)
        q[c] = (uint32_t)pack_e4m3x2(__fmul_rn(f[4 * c], inv), __fmul_rn(f[4 * c + 1], inv)) |
               (uint32_t)pack_e4m3x2(__fmul_rn(f[4 * c + 2], inv), __fmul_rn(f[4 * c + 3], inv)) << 16;
    if (block < blocks) {
        st_v4(a.xq + t * a.H + block * kBlock + piece * 16, make_uint4(q[0], q[1], q[2], q[3]));
        if (piece == 0) a.x_scales[t * blocks + block] = __fdiv_rn(amax, 448.f);
    }
}

template <int V>
cudaError_t launch_start(const MoeFewArgs &a, const LaneMap &map, cudaStream_t st) {
    const dim3 grid(1 + (unsigned)((a.H / kBlock + 15) / 16), (unsigned)a.route.T);
    if (a.route.r.scoring == EP_SCORE_SIGMOID) moe_few_start_kernel<V, kSigmoid><<<grid, kCastThreads, 0, st>>>(a, map);
    else if (a.route.r.softmax_key == EP_KEY_LOGIT)
        moe_few_start_kernel<V, kSoftmaxLogit><<<grid, kCastThreads, 0, st>>>(a, map);
    else moe_few_start_kernel<V, kSoftmaxScore><<<grid, kCastThreads, 0, st>>>(a, map);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_moe_few(const MoeFewArgs &a, cudaStream_t st) {
    MoeMaps maps;
    if (cudaError_t e = moe_map(a, a.gate_up, 2 * a.I, a.H, &maps.gate_up)) return e;
    if (cudaError_t e = moe_map(a, a.down, a.H, a.I, &maps.down)) return e;
    const LaneMap map = lane_map(a.route);
    if (cudaError_t e = map.each <= 8 ? launch_start<8>(a, map, st) : launch_start<32>(a, map, st)) return e;
    if (cudaError_t e = launch<true>(a, maps, st)) return e;
    return launch<false>(a, maps, st);
}

}  // namespace ep
