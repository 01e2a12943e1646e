// A whole mixture-of-experts layer for a few tokens (ep_moe_few), in two
// launches: routing, the cast of the tokens, the gate and up products, SwiGLU
// and its cast; then the down products and the weighted sum.
//
//   idx, w = route(logits);  a = e4m3(x);  h = e4m3(silu(a G_e^T) * (a U_e^T));
//   out[t] = residual[t] + sum_j w[t, j] (h D_e^T)[t, j],   e = idx[t, j]
//
// With a few tokens the time is that of reading the chosen experts' matrices
// once; what a layer made of separate launches adds is their latency and the
// receive buffers between them.  So every CTA routes all tokens itself (a warp a
// token; the logits are a few KB), lists the chosen experts, and starts on its
// share of their matrices; no CTA waits for another.  As in the products for few rows an
// expert, 128 matrix rows are the tensor core's M and the expert's tokens its N
// (16, 32, 48 or 64), every block of 128 channels is one accumulation in tensor
// memory, and a thread owns a matrix row and scales and adds the blocks in fp32.
//
// First launch: the warps that bring the tokens' rows read the bf16 tokens and
// cast them on the way to shared memory, so there is no cast tensor.  A unit of
// work is 128 columns of h, which are one block of its cast.  Both products of
// those columns land in the same thread.
// Second launch: a unit is 128 output columns of one expert.  Its products, in fp32, go
// to y [T, k, H] in the workspace; a CTA has a run of units, column tile after
// column tile; the one that brings a tile's last expert (a counter of units for each
// tile, which the first launch zeroes) adds the tile's k rows
// of each token in the order j = 0 .. k - 1.  So the sum does not depend on who comes
// last, and y is never rounded.  y is T k H 4 bytes against the experts' 3 I H each.
#include <algorithm>
#include <cstddef>
#include <type_traits>

#include "route_device.cuh"
#include "tcgen05.cuh"

namespace ep {

namespace {

constexpr int kBlock = 128;                     // channels, and matrix rows, of a scale
constexpr int kOperand = kBlock * kBlock;       // bytes of 128 matrix rows x 128 channels
constexpr int kThreads = 512;                   // warpgroup 0: boxes and products; 1: rows; 2, 3: accumulation
constexpr int kIssueRegs = 40, kCopyRegs = 120, kAccRegs = 176;   // 40 + 120 + 2 * 176 = 4 * 128, the launch's registers
constexpr int kRows = kMoeFewTokens;            // rows of a tile: an expert has at most one for each token
constexpr int kCopyThreads = 128;
constexpr int kAcc = 4;                         // accumulators
constexpr int kEntries = kRows * kMaxTopk;
template <bool UP>
constexpr int kStages = UP ? 4 : 7;             // operand buffers
// Steps whose scales are kept: a step's copies wait for the products kStages
// steps before, those for the loads of the accumulation kAcc steps before
// them, which may still be using that step's scales.
constexpr int kScaleRing = 16;

// The chosen experts and their entries (t * k + j), in the order of the experts and, in an expert, of the tokens
struct Chosen {
    uint64_t tokens[kMaxExperts];               // bit t: token t goes to the expert
    short expert[kMaxExperts], place[kMaxExperts], start[kMaxExperts + 1];
    short entry[kEntries], idx[kEntries];
    float weight[kEntries];
    int n;
};

template <bool UP>
struct MoeShared {
    unsigned char w[kStages<UP>][(UP ? 2 : 1) * kOperand];
    unsigned char rows[kStages<UP>][kRows * kBlock];
    uint64_t boxes[kStages<UP>];                            // matrix rows
    uint64_t rows_full[kStages<UP>], full[kStages<UP>];     // rows and scales; all operands
    uint64_t done[kStages<UP>];                             // a step's products: buffers free, sums and scales ready
    uint64_t tempty[kAcc];                                  // accumulators taken out
    uint64_t joined[2];                                     // UP: a warpgroup's maxima are written; else: y is, and who
                                                            // is last is known
    alignas(16) float row_scale[kScaleRing][kRows];
    float w_scale[kScaleRing][2];
    alignas(16) uint32_t amax[2][UP ? kRows : 1][4];        // [unit parity][row][warp of the warpgroup]
    int last[2];
    Chosen chosen;
    uint32_t tmem;
    int gave_up;
};
static_assert(kThreads / 32 * 2 * kMaxExperts * 4 <= sizeof(MoeShared<true>::w), "the routing's words fit the operands");
static_assert(kThreads / 32 * 2 * kMaxExperts * 4 <= sizeof(MoeShared<false>::w) + sizeof(MoeShared<false>::rows), "");

__device__ __forceinline__ float logit(const RouteArgs &a, int t, int e) {
    return a.bf16 ? widen(__ldg(reinterpret_cast<const uint16_t *>(a.logits) + t * a.stride + e))
                  : __ldg(reinterpret_cast<const float *>(a.logits) + t * a.stride + e);
}

// ep_route of one token by a warp, with the same keys, sums and ties, for one
// token at a time: the keys lie in shared memory (key and score: kMaxExperts
// words each), and each round only the lane that lost its best looks again.
// Lane j gets entry j.
__device__ __forceinline__ void route_token(const RouteArgs &a, const LaneMap &map, int t, uint32_t *key,
                                            uint32_t *score, int &id, float &weight) {
    const int lane = threadIdx.x & 31, E = (int)a.E, k = (int)a.k;
    const bool sig = a.r.scoring == EP_SCORE_SIGMOID, by_score = !sig && a.r.softmax_key == EP_KEY_SCORE;
    const int lo = map.first(lane), held = map.count(lane);
    float m = 0.f, z = 1.f;
    if (!sig && (by_score || !a.r.renormalize)) {
        m = -INFINITY;
        for (int i = 0; i < held; ++i) {
            const float x = logit(a, t, lo + i);
            if (x > -INFINITY) m = fmaxf(m, fminf(x, kMaxFinite));
        }
        m = warp_max(m);
        z = 0.f;
        for (int i = 0; i < held; ++i) {
            const float x = logit(a, t, lo + i);
            if (x > -INFINITY) z += expf(fminf(x, kMaxFinite) - m);
        }
        z = lanes_sum<32>(z);
    }
    bool nan = false;
    for (int i = 0; i < held; ++i) {
        const float x = logit(a, t, lo + i), b = a.bias ? __ldg(a.bias + lo + i) : 0.f;
        float c = sig ? sigmoid(x) : x;
        if (by_score && x > -INFINITY) c = expf(fminf(x, kMaxFinite) - m) / z;
        const float f = c + b + 0.f;           // (-0 + 0 = +0: equal keys, equal words)
        nan |= x != x || b != b;
        key[lo + i] = x > -INFINITY && f > -INFINITY ? order_word(f) : 0;
    }
    if (nan) raise_status(a.dev_status, EP_STATUS_BAD_LOGIT);
    __syncwarp();
    const int G = a.r.num_groups, per = E / G;
    if (a.r.topk_groups < G) {
        for (int g = lane; g < G; g += 32) {
            uint32_t b1 = 0, b2 = 0;
            for (int i = 0; i < per; ++i) {
                const uint32_t v = key[g * per + i];
                b2 = max(b2, min(b1, v));
                b1 = max(b1, v);
            }
            score[g] = a.r.group_best == 2 && b1 && b2 ? order_word(order_float(b1) + order_float(b2)) : b1;
        }
        __syncwarp();
        // the groups that stay are marked by a score of 0 once they are taken, the others keep theirs
        uint32_t best = 0;
        int at = 0x7fffffff;
        const auto look = [&]() {
            best = 0;
            for (int g = lane; g < G; g += 32)
                if (score[g] > best) { best = score[g]; at = g; }
        };
        look();
        for (int n = 0; n < a.r.topk_groups; ++n) {
            const uint32_t top = __reduce_max_sync(kFull, best);
            if (!top) break;
            const int g = (int)__reduce_min_sync(kFull, best == top ? (unsigned)at : 0x7fffffffu);
            if (best == top && at == g) {
                score[g] = 0;
                look();
            }
        }
        __syncwarp();
        for (int e = lane; e < E; e += 32)
            if (score[e / per]) key[e] = 0;    // (a group without eligible experts has no keys to clear)
        __syncwarp();
    }
    uint32_t best = 0;
    int at = 0x7fffffff;
    const auto look = [&]() {
        best = 0;
        for (int e = lane; e < E; e += 32)
            if (key[e] > best) { best = key[e]; at = e; }
    };
    look();
    id = -1;
    for (int j = 0; j < k; ++j) {
        const uint32_t top = __reduce_max_sync(kFull, best);
        if (!top) break;
        const int e = (int)__reduce_min_sync(kFull, best == top ? (unsigned)at : 0x7fffffffu);
        if (lane == j) id = e;
        if (best == top && at == e) {
            key[e] = 0;
            look();
        }
    }
    float s = 0.f, xj = id >= 0 ? logit(a, t, id) : -INFINITY;
    if (sig) {
        s = id >= 0 ? sigmoid(xj) : 0.f;
    } else {
        xj = fminf(xj, kMaxFinite);
        if (a.r.renormalize) m = warp_max(xj);
        s = id >= 0 ? expf(xj - m) : 0.f;
    }
    if (a.r.renormalize) z = lanes_sum<32>(s);
    weight = id >= 0 && z > 0.f ? s / z * a.r.scale : 0.f;
}

// Fills the lists from c.idx, by all threads of the block; complete when it returns.
__device__ __forceinline__ void list_chosen(Chosen &c, int E, int T, int k) {
    const int lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < E; e += kThreads) c.tokens[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < T * k; i += kThreads)
        if (c.idx[i] >= 0) atomicOr(reinterpret_cast<unsigned long long *>(&c.tokens[c.idx[i]]), 1ull << (i / k));
    __syncthreads();
    if (threadIdx.x < 32) {
        int n = 0, sum = 0;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane, rows = e < E ? __popcll(c.tokens[e]) : 0;
            const unsigned some = __ballot_sync(kFull, rows > 0);
            int inc = rows;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kFull, inc, o);
                if (lane >= o) inc += v;
            }
            if (rows > 0) {
                const int at = n + __popc(some & lanemask_lt());
                c.expert[at] = (short)e;
                c.place[e] = (short)at;
                c.start[at] = (short)(sum + inc - rows);
            }
            n += __popc(some);
            sum += __shfl_sync(kFull, inc, 31);
        }
        if (lane == 0) {
            c.start[n] = (short)sum;
            c.n = n;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < T * k; i += kThreads) {
        const int e = c.idx[i];
        if (e >= 0) c.entry[c.start[c.place[e]] + __popcll(c.tokens[e] & ((1ull << (i / k)) - 1))] = (short)i;
    }
    __syncthreads();
}

// A unit of work
struct MoeUnit {
    int e, tile, rows;
    const short *entry;
};
template <bool UP>
__device__ __forceinline__ MoeUnit moe_unit(const Chosen &c, int tiles, int u) {
    // first launch: an expert's column tiles follow one another; second: a column tile's experts
    const int at = UP ? u / tiles : u % c.n;
    return MoeUnit{c.expert[at], UP ? u - at * tiles : u / c.n, c.start[at + 1] - c.start[at], c.entry + c.start[at]};
}

// out[t, columns of a tile] by the 256 accumulating threads
__device__ __forceinline__ void combine_tile(const MoeFewArgs &a, const Chosen &c, int tile) {
    const int thread = threadIdx.x - 256, col = tile * kBlock + (thread & 31) * 4, k = (int)a.route.k;
    for (int t = thread >> 5; t < (int)a.route.T; t += 8) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int j = 0; j < k; ++j) {
            if (c.idx[t * k + j] < 0) continue;
            const float w = c.weight[t * k + j];
            const float4 y = __ldcg(reinterpret_cast<const float4 *>(a.y + (int64_t)(t * k + j) * a.H + col));
            v.x += w * y.x;
            v.y += w * y.y;
            v.z += w * y.z;
            v.w += w * y.w;
        }
        if (a.residual) {
            const uint2 r = *reinterpret_cast<const uint2 *>(a.residual + t * a.H + col);
            v.x += bf16_lo(r.x);
            v.y += bf16_hi(r.x);
            v.z += bf16_lo(r.y);
            v.w += bf16_hi(r.y);
        }
        *reinterpret_cast<uint2 *>(a.out + t * a.H + col) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
}

template <bool UP>
__global__ void __launch_bounds__(kThreads, 1)
    moe_few_kernel(const __grid_constant__ MoeFewArgs a, const __grid_constant__ CUtensorMap map_w, const LaneMap map) {
    extern __shared__ __align__(1024) unsigned char raw[];    // (the only shared memory: it starts at its window's start)
    MoeShared<UP> &s = *reinterpret_cast<MoeShared<UP> *>(raw);
    constexpr int S = kStages<UP>, NB = UP ? 2 : 1;
    static_assert(offsetof(MoeShared<UP>, rows) % 1024 == 0 && offsetof(MoeShared<UP>, boxes) % 8 == 0, "");
    static_assert(offsetof(MoeShared<UP>, row_scale) % 16 == 0 && offsetof(MoeShared<UP>, amax) % 16 == 0, "");
    static_assert(kScaleRing > S + kAcc + 1, "scales are still in use when they are overwritten");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int T = (int)a.route.T, k = (int)a.route.k, E = (int)a.route.E;
    const int K = (int)(UP ? a.H : a.I), n_cols = (int)(UP ? a.I : a.H), kb_n = K / kBlock, tiles = n_cols / kBlock;
    Chosen &ch = s.chosen;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&s.rows_full[i], UP ? kCopyThreads / 32 : kCopyThreads);   // (else the copies' own arrivals)
            mbar_init(&s.boxes[i], 1);
            mbar_init(&s.full[i], 1);
            mbar_init(&s.done[i], 2);          // the products' commit, word of the operands
        }
        for (int i = 0; i < kAcc; ++i) mbar_init(&s.tempty[i], 8);
        mbar_init(&s.joined[0], UP ? 4 : 8);
        mbar_init(&s.joined[1], UP ? 4 : 1);
        s.gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc<1>(&s.tmem);
    if (UP) {
        // ---- routing: a warp a token; the first CTA writes it out and zeroes the second launch's counters ----
        uint32_t *key = reinterpret_cast<uint32_t *>(raw) + warp * 2 * kMaxExperts;
        RouteArgs r = a.route;
        if (blockIdx.x > 0) r.dev_status = nullptr;
        for (int t = warp; t < T; t += kThreads / 32) {
            int id;
            float weight;
            route_token(r, map, t, key, key + kMaxExperts, id, weight);
            if (lane < k) {
                ch.idx[t * k + lane] = (short)id;
                if (blockIdx.x == 0) {
                    a.route.topk_idx[t * k + lane] = id;
                    a.route.topk_weights[t * k + lane] = weight;
                }
            }
        }
        if (blockIdx.x == 0)
            for (int i = threadIdx.x; i < (int)(a.H / kBlock); i += kThreads) a.arrived[i] = 0;
    } else {
        for (int i = threadIdx.x; i < T * k; i += kThreads) {
            ch.idx[i] = (short)a.route.topk_idx[i];
            ch.weight[i] = a.route.topk_weights[i];
        }
    }
    __syncthreads();
    list_chosen(ch, E, T, k);
    fence_async_shared();          // the routing's words are behind the boxes that come to the same place
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = s.tmem;
    // this CTA's units: a run of them, so that in the second launch it has few column tiles to give word of
    const int64_t units = (int64_t)ch.n * tiles;
    const int u0 = (int)(units * blockIdx.x / gridDim.x), u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
    const Patience patience{&s.gave_up, a.wait_clocks};

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
        if (warp == 0) {
            // ---- matrix rows ----
            if (lane == 0) {
                int st = 0, ph = 1, it = 0;
                bool ok = true;
                for (int u = u0; u < u1 && ok; ++u) {
                    const MoeUnit v = moe_unit<UP>(ch, tiles, u);
                    for (int kb = 0; kb < kb_n; ++kb, ++it) {
                        ok = mbar_wait(&s.done[st], ph, patience);
                        if (!ok) break;
                        mbar_expect_tx(&s.boxes[st], NB * kOperand);
#pragma unroll
                        for (int b = 0; b < NB; ++b)
                            tma_load_3d(s.w[st] + b * kOperand, &map_w, kb * kBlock, v.tile * kBlock + b * n_cols, v.e,
                                        &s.boxes[st]);
                        if (++st == S) { st = 0; ph ^= 1; }
                    }
                }
                drain<S>(s.boxes, it);
            }
            __syncwarp();
        } else if (warp == 1) {
            // ---- products (the loop is the whole warp's, so that its values are uniform; one lane issues) ----
            const bool issue = elect_one();
            const uint64_t dw = smem_desc(s.w[0]), dr = smem_desc(s.rows[0]);
            int st = 0, ph = 0, acc = 0, aph = 1, it = 0;
            bool ok = true;
            for (int u = u0; u < u1 && ok; ++u) {
                const MoeUnit v = moe_unit<UP>(ch, tiles, u);
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
                            for (int i = 0; i < 4; ++i)   // 32 channels a step
                                mma_f8<1>(tmem + (acc * NB + b) * kRows, da + (b * (kOperand >> 4) + i * 2), db + i * 2,
                                          idesc, i > 0);
                        mma_commit<1>(&s.done[st]);
                    }
                    if (++st == S) { st = 0; ph ^= 1; }
                    acc = (acc + 1) % kAcc;
                    aph ^= acc == 0;
                }
            }
            drain<S>(s.done, it);
            __syncwarp();
        } else if (warp == 2) {
            // ---- word of the operands: to the products, and to the accumulation, which reads the scales with
            // ordinary loads (the commit's arrival tells of the products) ----
            if (lane == 0) {
                int st = 0, ph = 0;
                bool ok = true;
                for (int u = u0; u < u1 && ok; ++u) {
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
        // ---- rows and scales: eight lanes bring a row's 128 channels ----
        constexpr int kPass = kCopyThreads / 8, kMine = kRows / kPass;
        const int part = (threadIdx.x - 128) >> 3, piece = lane & 7;
        const int place = (threadIdx.x - 128) & (kRows - 1);      // the row whose scale this thread copies, if below 64
        const int n_blocks = NB * tiles;                          // of the matrix's rows
        int st = 0, ph = 1, ring = 0;
        bool ok = true;
        for (int u = u0; u < u1 && ok; ++u) {
            const MoeUnit v = moe_unit<UP>(ch, tiles, u);
            uint32_t ws = (uint32_t)(v.e * n_blocks + v.tile) * kb_n;
            if (lane == 1) ws += (uint32_t)tiles * kb_n;          // (the up block's)
            const uint32_t swizzled = part * kBlock + ((piece ^ (part & 7)) << 4);
            if (UP) {
                // few rows: their loads run further ahead (the tokens come from L2, and a step has to take less than
                // the copy of its matrix rows, some 1400 cycles)
                const auto rows = [&](auto passes) {
                    constexpr int P = decltype(passes)::value, D = P > 1 ? 1 : 4;   // passes of 16 rows; steps ahead
                    uint32_t src[P];                              // in 16 bytes
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const int r = i * kPass + part;
                        src[i] = (uint32_t)(r < v.rows ? v.entry[r] / k : 0) * (uint32_t)(a.H / 8) + piece * 2;
                    }
                    const float *scale = a.gate_up_scales + ws;
                    const bool has_scale = warp == 7 && lane < NB;
                    uint4 in[D][P][2];
                    float sw[D];
                    const auto load = [&](int d, int kb) {
#pragma unroll
                        for (int i = 0; i < P; ++i) {
                            const uint4 *from = reinterpret_cast<const uint4 *>(a.x) + (src[i] + kb * (kBlock / 8));
                            in[d][i][0] = __ldg(from);
                            in[d][i][1] = __ldg(from + 1);
                        }
                        sw[d] = has_scale ? __ldg(scale + kb) : 0.f;
                    };
#pragma unroll
                    for (int d = 0; d < D; ++d)
                        if (d < kb_n) load(d, d);
                    for (int kb0 = 0; kb0 < kb_n; kb0 += D)
#pragma unroll
                        for (int d = 0; d < D; ++d) {
                            const int kb = kb0 + d;
                            if (kb >= kb_n) break;
                            if (!warp_wait(&s.done[st], ph, patience)) return false;
#pragma unroll
                            for (int i = 0; i < P; ++i) {
                                // the cast of ep_dispatch
                                const uint4 x = in[d][i][0], y = in[d][i][1];
                                const uint32_t w8[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
                                float f[16], amax = 0.f;
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
                                           (uint32_t)pack_e4m3x2(__fmul_rn(f[4 * c + 2], inv), __fmul_rn(f[4 * c + 3], inv))
                                               << 16;
                                if (i * kPass + part < v.rows) {
                                    *reinterpret_cast<uint4 *>(s.rows[st] + i * kPass * kBlock + swizzled) =
                                        make_uint4(q[0], q[1], q[2], q[3]);
                                    if (piece == 0) s.row_scale[ring][i * kPass + part] = __fdiv_rn(amax, 448.f);
                                }
                                asm volatile("" ::: "memory");    // (one row after the other: registers)
                            }
                            if (has_scale) s.w_scale[ring][lane] = sw[d];
                            fence_async_shared();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(&s.rows_full[st]);
                            if (kb + D < kb_n) load(d, kb + D);
                            if (++st == S) { st = 0; ph ^= 1; }
                            ring = (ring + 1) % kScaleRing;
                        }
                    return true;
                };
                if (v.rows <= 16) ok = rows(std::integral_constant<int, 1>());
                else ok = rows(std::integral_constant<int, 4>());
            } else {
                int row[kMine];                                   // entries
#pragma unroll
                for (int i = 0; i < kMine; ++i) {
                    const int r = i * kPass + part;
                    row[i] = r < v.rows ? v.entry[r] : 0;
                }
                const int scale_row = warp < 6 && place < v.rows ? v.entry[place] : -1;
                for (int kb = 0; kb < kb_n; ++kb) {
                    ok = warp_wait(&s.done[st], ph, patience);
                    if (!ok) break;
                    const uint32_t dst = smem_addr(s.rows[st]) + swizzled;
#pragma unroll
                    for (int i = 0; i < kMine; ++i)
                        if (i * kPass + part < v.rows)
                            cp_async16(dst + i * kPass * kBlock, a.h + (int64_t)row[i] * K + kb * kBlock + piece * 16);
                    if (scale_row >= 0)
                        cp_async4(smem_addr(&s.row_scale[ring][place]), a.h_scales + (int64_t)scale_row * kb_n + kb);
                    if (warp == 7 && lane == 0) cp_async4(smem_addr(&s.w_scale[ring][0]), a.down_scales + (ws + kb));
                    cp_async_arrive(&s.rows_full[st]);
                    if (++st == S) { st = 0; ph ^= 1; }
                    ring = (ring + 1) % kScaleRing;
                }
            }
        }
        if (!UP) cp_async_wait_all();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kAccRegs));
        // ---- accumulation: thread = matrix row (UP: of the gate's and of the up block); a warpgroup has every other 16
        // columns (rows of the tile) ----
        constexpr int kMine = kRows / 2;
        const int half = (warp - 8) >> 2, quarter = warp & 3;
        const int chan = quarter * 32 + lane;
        const auto column = [&](int c) { return ((c >> 4) * 2 + half) * 16 + (c & 15); };   // my c-th column
        const uint32_t tm = tmem + (uint32_t)(quarter * 32) * 65536;
        int st = 0, ph = 0, p = 0, ring = 0, unit = 0, word = 0, mine = 0;   // (mine: units of this column tile)
        bool ok = true;
        for (int u = u0; u < u1 && ok; ++u, ++unit) {
            const MoeUnit v = moe_unit<UP>(ch, tiles, u);
            uint64_t acc[NB][kMine / 2];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int c = 0; c < kMine / 2; ++c) acc[b][c] = 0;
            for (int kb = 0; kb < kb_n; ++kb) {
                ok = warp_wait(&s.done[st], ph, patience);
                if (!ok) break;
                tmem_fence_after();
                uint32_t t[NB * kMine];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int q = 0; q < kMine / 16; ++q)
                        if (column(q * 16) < v.rows)
                            tmem_ld16(tm + (p * NB + b) * kRows + column(q * 16), t + b * kMine + q * 16);
                tmem_wait_ld<NB * kMine>(t);
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.tempty[p]);
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const uint32_t w32 = __float_as_uint(s.w_scale[ring][b]);
                    const uint64_t sw = pair2(w32, w32);
#pragma unroll
                    for (int q = 0; q < kMine / 16; ++q) {
                        if (column(q * 16) >= v.rows) break;
                        const ulonglong2 *sr = reinterpret_cast<const ulonglong2 *>(&s.row_scale[ring][column(q * 16)]);
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
                p = (p + 1) % kAcc;
                ring = (ring + 1) % kScaleRing;
            }
            if (!ok) break;
            if (UP) {
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
                uint32_t(*amax)[4] = s.amax[unit & 1];     // (a warp a unit ahead writes to the other)
                if (at < v.rows) amax[UP ? at : 0][quarter] = top;
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.joined[half]);
                ok = warp_wait(&s.joined[half], unit & 1, patience);
                if (!ok) break;
                float inv = 0.f;                           // lane c: of column c
                if (at < v.rows) {
                    const uint4 t4 = *reinterpret_cast<const uint4 *>(amax[UP ? at : 0]);
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
            } else {
                float *y = a.y + v.tile * kBlock + chan;
#pragma unroll
                for (int c = 0; c < kMine; ++c) {
                    if (column(c) >= v.rows) break;
                    y[(int64_t)v.entry[column(c)] * n_cols] = c & 1 ? hi2(acc[0][c / 2]) : lo2(acc[0][c / 2]);
                }
                // The last of my units of this tile: count them.  Everybody's y is out before, and in before it is read.
                ++mine;
                if (u + 1 < u1 && (u + 1) / ch.n == v.tile) continue;
                __threadfence();
                __syncwarp();
                if (lane == 0) mbar_arrive(&s.joined[0]);
                if (warp == 8) {
                    ok = warp_wait(&s.joined[0], word & 1, patience);
                    if (!ok) break;
                    if (lane == 0) {
                        s.last[word & 1] = atomicAdd(a.arrived + v.tile, (unsigned)mine) + mine == (unsigned)ch.n;
                        __threadfence();
                        mbar_arrive(&s.joined[1]);
                    }
                    __syncwarp();
                }
                ok = warp_wait(&s.joined[1], word & 1, patience);
                if (!ok) break;
                if (s.last[word & 1]) combine_tile(a, ch, v.tile);
                ++word;
                mine = 0;
            }
        }
        if (!UP && ch.n == 0)                              // no token has an expert
            for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) combine_tile(a, ch, tile);
    }
    tmem_fence_before();
    __syncthreads();
    if (warp == 1) {
        tmem_fence_after();
        tmem_free<1>(tmem);
    }
    if (threadIdx.x == 0 && s.gave_up) raise_status(a.route.dev_status, EP_STATUS_TIMEOUT);
}

template <bool UP>
cudaError_t launch(const MoeFewArgs &a, const LaneMap &map, cudaStream_t st) {
    const int64_t K = UP ? a.H : a.I, N = UP ? 2 * a.I : a.H;
    const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)N, (cuuint64_t)a.route.E};
    const cuuint64_t strides[2] = {(cuuint64_t)K, (cuuint64_t)(N * K)};
    const cuuint32_t box[3] = {kBlock, kBlock, 1};
    CUtensorMap w;
    if (cudaError_t e = encode_map(&w, 3, UP ? a.gate_up : a.down, dims, strides, box)) return e;
    constexpr int bytes = sizeof(MoeShared<UP>);
    static_assert(bytes <= 227 * 1024, "shared memory");
    static std::atomic<int> ready[kCacheDevices];
    cudaError_t e = cudaSuccess;
    cached_per_device(ready, [&](int) {
        e = cudaFuncSetAttribute(moe_few_kernel<UP>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        // the warpgroups' register shares are drawn from what the block was launched with
        cudaFuncAttributes f{};
        if (!e) e = cudaFuncGetAttributes(&f, moe_few_kernel<UP>);
        if (!e && f.numRegs * 4 < kIssueRegs + kCopyRegs + 2 * kAccRegs) e = cudaErrorInvalidDeviceFunction;
        return e == cudaSuccess ? 1 : 0;
    });
    if (e) return e;
    moe_few_kernel<UP><<<num_sms(), kThreads, bytes, st>>>(a, w, map);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_moe_few(const MoeFewArgs &a, cudaStream_t st) {
    const LaneMap map = lane_map(a.route);
    if (cudaError_t e = launch<true>(a, map, st)) return e;
    return launch<false>(a, map, st);
}

}  // namespace ep
