// Routing: a token's logits -> its k experts and their weights, and the
// gradient of the weights with respect to the logits.
//
// A warp owns one token.  Lanes hold consecutive experts in registers, up to V
// each (V a power of two), so a row is read once and "lowest index first" is
// lane order; where experts form groups, a group has lanes of its own.  Keys
// are compared as unsigned words in the order of the floats; 0 stands for
// "not eligible".
//
// The memory traffic is small (a row read, k pairs written); what takes the
// time is instructions: the scores (an exponential and a reciprocal for each
// expert) and the choice.  The choice sorts each lane's keys once (blocks of
// eight, a network of minima and maxima without the indices), after which
// each of the k rounds is one warp maximum over the lanes' heads, a ballot for
// the lowest lane that has it, and a shift of that lane's list; lane j notes
// the key and the lane of round j and looks its index up at the end.
//
// Measured (256 experts, top-8, grouped sigmoid with a bias): 65536 tokens 59.5 us,
// 980 instructions a token at 90% of the issue slots, of which some 200 are the
// exponentials and reciprocals of the scores, correctly rounded because a key
// decides; the memory alone would take 11 us.  32 tokens: 3.3 us from a graph.
#include "moe_internal.cuh"

namespace ep {

namespace {

constexpr int kRouteWarps = 4;
constexpr float kMaxFinite = 3.402823466e38f;

// order-preserving word of a float that is neither NaN nor -inf (always > 0)
__device__ __forceinline__ uint32_t order_word(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_float(uint32_t w) {
    return __uint_as_float(w & 0x80000000u ? w ^ 0x80000000u : ~w);
}

__device__ __forceinline__ float sigmoid(float x) { return __frcp_rn(1.f + expf(-x)); }

// sum, and maximum, over the W lanes of a token
template <int W>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
template <int W>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int o = W / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}
// maximum of numbers (not NaN) as the maximum of their words
__device__ __forceinline__ float warp_max(float v) {
    const uint32_t w = v > -INFINITY ? order_word(v) : 0;
    const uint32_t m = __reduce_max_sync(kFull, w);
    return m ? order_float(m) : -INFINITY;
}

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ void narrow(float v, float &out) { out = v; }
__device__ __forceinline__ void narrow(float v, uint16_t &out) { out = (uint16_t)pack_bf16x2(v, 0.f); }

// widest vector that V elements of a lane make up
template <int BYTES> struct Vec { typedef uint4 T; };
template <> struct Vec<8> { typedef uint2 T; };
template <> struct Vec<4> { typedef uint32_t T; };
template <> struct Vec<2> { typedef uint16_t T; };

// Which experts a lane holds: 1 << log lanes share each of the groups of `per`
// experts, `each` a lane.
struct LaneMap {
    int groups, per, log, each;
    __device__ __forceinline__ int in(int lane) const { return (lane & ((1 << log) - 1)) * each; }
    __device__ __forceinline__ int first(int lane) const { return (lane >> log) * per + in(lane); }
    __device__ __forceinline__ int count(int lane) const {
        return lane >> log < groups ? max(0, min(each, per - in(lane))) : 0;
    }
};

// A lane's n <= V elements of a row, from element lo on; the rest read as -inf.
// vec: every lane has V, and rows are aligned to the vector.
template <typename L, int V>
__device__ __forceinline__ void load_lane(const L *row, int lo, int n, bool vec, float (&x)[V]) {
    if (vec) {
        typedef typename Vec<(sizeof(L) * V > 16 ? 16 : sizeof(L) * V)>::T W;
        constexpr int N = sizeof(L) * V / sizeof(W);
        union { W w[N]; L l[V]; } u;
#pragma unroll
        for (int i = 0; i < N; ++i) u.w[i] = __ldg(reinterpret_cast<const W *>(row + lo) + i);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = widen(u.l[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i < n ? widen(row[lo + i]) : -INFINITY;
    }
}

// The same for work that needs no order (the gradient): W lanes share a row of
// E elements in turns, of 16 bytes where E is a multiple of them, else of one
// element.  Only E decides which, so that the order of the sums does not depend
// on where a row lies; vec: the rows are aligned to 16 bytes.
template <typename L, int W, int V>
__device__ __forceinline__ void load_turns(const L *row, int E, int lane, bool vec, float (&x)[V]) {
    constexpr int C = 16 / sizeof(L);
    if (V >= C && E % C == 0) {
#pragma unroll
        for (int i = 0; i < V / C; ++i) {
            union { uint4 w; L l[C]; } u;
            const int e = (i * W + lane) * C;
            if (e < E && vec) u.w = __ldg(reinterpret_cast<const uint4 *>(row + e));
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (e < E && !vec) u.l[c] = row[e + c];
                x[(i * C + c) % V] = e < E ? widen(u.l[c]) : -INFINITY;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = i * W + lane < E ? widen(row[i * W + lane]) : -INFINITY;
    }
}
template <typename L, int W, int V>
__device__ __forceinline__ void store_turns(L *row, int E, int lane, bool vec, const float (&x)[V]) {
    constexpr int C = 16 / sizeof(L);
    if (V >= C && E % C == 0) {
#pragma unroll
        for (int i = 0; i < V / C; ++i) {
            union { uint4 w; L l[C]; } u;
            const int e = (i * W + lane) * C;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                narrow(x[(i * C + c) % V], u.l[c]);
                if (e < E && !vec) row[e + c] = u.l[c];
            }
            if (e < E && vec) *reinterpret_cast<uint4 *>(row + e) = u.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i * W + lane < E) narrow(x[i], row[i * W + lane]);
    }
}

__device__ __forceinline__ void order2(uint32_t &a, uint32_t &b) {
    const uint32_t hi = max(a, b);
    b = min(a, b);
    a = hi;
}
// Descending order of 2, 4 or 8 words (Batcher's odd-even merge sort).
template <int N>
__device__ __forceinline__ void sort_words(uint32_t *w) {
#pragma unroll
    for (int p = 1; p < N; p <<= 1)
#pragma unroll
        for (int k = p; k >= 1; k >>= 1)
#pragma unroll
            for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; ++i)
                    if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) order2(w[i + j], w[i + j + k]);
}

// Clears the keys of the groups that are not among the best.  Any split of the
// experts (more than 32 groups, or groups too large for lanes of their own):
// groups one after the other, scores kept by lane g % 32.
template <int V>
__device__ __forceinline__ void keep_groups(const RouteArgs &a, int first, uint32_t (&key)[V]) {
    const int lane = threadIdx.x & 31;
    const int G = a.r.num_groups, per = (int)a.E / G, slots = (G + 31) / 32;
    uint32_t score[kMaxExperts / 32], kept[kMaxExperts / 32];
    for (int s = 0; s < slots; ++s) score[s] = kept[s] = 0;
    for (int g = 0; g < G; ++g) {
        const int lo = g * per, hi = lo + per;
        uint32_t b1 = 0, b2 = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = first + i;
            const uint32_t v = e >= lo && e < hi ? key[i] : 0;
            b2 = max(b2, min(b1, v));
            b1 = max(b1, v);
        }
        const uint32_t top = __reduce_max_sync(kFull, b1);
        uint32_t w = top;
        if (a.r.group_best == 2) {
            const unsigned who = __ballot_sync(kFull, b1 == top);
            const uint32_t second = __reduce_max_sync(kFull, lane == __ffs(who) - 1 ? b2 : b1);
            if (top && second) w = order_word(order_float(top) + order_float(second));
        }
        if ((g & 31) == lane) score[g >> 5] = w;
    }
    for (int n = 0; n < a.r.topk_groups; ++n) {
        uint32_t b = 0, at = 0x7fffffffu;
        for (int s = 0; s < slots; ++s)
            if (score[s] > b) { b = score[s]; at = s * 32 + lane; }
        const uint32_t top = __reduce_max_sync(kFull, b);
        if (!top) break;
        const int g = (int)__reduce_min_sync(kFull, b == top ? at : 0x7fffffffu);
        for (int s = 0; s < slots; ++s) {
            if (g == s * 32 + lane) score[s] = 0;
            if ((g >> 5) == s) kept[s] |= 1u << (g & 31);
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int g = (first + i) / per;
        if (g >= G || !((kept[g >> 5] >> (g & 31)) & 1)) key[i] = 0;
    }
}

// The same where every group has `lanes` lanes of its own: the best two of a
// group meet in a butterfly, then topk_groups rounds take the best score left.
template <int V>
__device__ __forceinline__ void keep_lane_groups(const RouteArgs &a, int lanes, uint32_t (&key)[V]) {
    const int lane = threadIdx.x & 31;
    uint32_t b1 = 0, b2 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        b2 = max(b2, min(b1, key[i]));
        b1 = max(b1, key[i]);
    }
    for (int o = 1; o < lanes; o <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(kFull, b1, o), o2 = __shfl_xor_sync(kFull, b2, o);
        b2 = max(min(b1, o1), max(b2, o2));
        b1 = max(b1, o1);
    }
    const uint32_t score =
        a.r.group_best == 2 && b1 && b2 ? order_word(order_float(b1) + order_float(b2)) : b1;   // (never -0: no key is)
    uint32_t left = score;
    bool keep = false;
    for (int n = 0; n < a.r.topk_groups; ++n) {
        const uint32_t top = __reduce_max_sync(kFull, left);
        if (!top) break;
        const int first = __ffs(__ballot_sync(kFull, left == top)) - 1;     // a group's lowest lane
        if ((unsigned)(lane - first) < (unsigned)lanes) {
            keep = true;
            left = 0;
        }
    }
    if (!keep) {
#pragma unroll
        for (int i = 0; i < V; ++i) key[i] = 0;
    }
}

// What the keys are, as a template argument: as a run-time branch the softmax scores cost the other softmax key 2 us
// of 37 (65536 tokens x 256 experts, fp32, renormalised; by score 55 us: an exponential and a quotient for each expert)
enum { kSoftmaxLogit, kSoftmaxScore, kSigmoid };

template <typename L, int V, int KEY>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a, LaneMap map, bool vec) {
    constexpr bool SIG = KEY == kSigmoid, by_score = KEY == kSoftmaxScore;
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const int k = (int)a.k, lo = map.first(lane), held = map.count(lane);
    const L *row = reinterpret_cast<const L *>(a.logits) + t * a.stride;
    float x[V], b[V];
    uint32_t key[V];
    load_lane<L, V>(row, lo, held, vec, x);
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = 0.f;
    if (a.bias) load_lane<float, V>(a.bias, lo, held, vec && ((uintptr_t)a.bias & 15) == 0, b);
    // softmax over the logits that are numbers, where a weight or a key needs it
    float m = 0.f, z = 1.f;
    if (!SIG && (by_score || !a.r.renormalize)) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (x[i] > -INFINITY) m = fmaxf(m, fminf(x[i], kMaxFinite));
        m = warp_max(m);
        z = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (x[i] > -INFINITY) z += expf(fminf(x[i], kMaxFinite) - m);
        z = lanes_sum<32>(z);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        float c = SIG ? sigmoid(x[i]) : x[i];
        if (by_score && x[i] > -INFINITY) c = expf(fminf(x[i], kMaxFinite) - m) / z;
        const float f = c + b[i] + 0.f;        // (-0 + 0 = +0: equal keys, equal words)
        nan |= f != f;
        key[i] = x[i] > -INFINITY && f > -INFINITY ? order_word(f) : 0;   // comparisons are false for NaN
    }
    if (nan) {                // (infinities of opposite signs also add to NaN; they only make an expert ineligible)
        nan = false;
#pragma unroll
        for (int i = 0; i < V; ++i) nan |= x[i] != x[i] || b[i] != b[i];
        if (nan) raise_status(a.dev_status, EP_STATUS_BAD_LOGIT);
    }
    if (a.r.topk_groups < a.r.num_groups) {
        if (map.groups == a.r.num_groups) keep_lane_groups<V>(a, 1 << map.log, key);
        else keep_groups<V>(a, lo, key);
    }

    constexpr int N = V < 8 ? V : 8, B = V / N;   // sorted blocks of a lane
    uint32_t list[B][N];
#pragma unroll
    for (int c = 0; c < B; ++c) {
#pragma unroll
        for (int i = 0; i < N; ++i) list[c][i] = key[c * N + i];
        sort_words<N>(list[c]);
    }
    uint32_t mine = 0;        // of round j = lane: the key, and the lane that had it
    int from = 0;
    for (int j = 0; j < k; ++j) {
        uint32_t head = list[0][0];
#pragma unroll
        for (int c = 1; c < B; ++c) head = max(head, list[c][0]);
        const uint32_t top = __reduce_max_sync(kFull, head);
        if (!top) break;
        const int win = __ffs(__ballot_sync(kFull, head == top)) - 1;
        if (lane == j) { mine = top; from = win; }
        bool pop = lane == win;
#pragma unroll
        for (int c = 0; c < B; ++c) {
            if (pop && (B == 1 || list[c][0] == top)) {
#pragma unroll
                for (int i = 0; i + 1 < N; ++i) list[c][i] = list[c][i + 1];
                list[c][N - 1] = 0;
                pop = false;
            }
        }
    }
    // The index: the lane's n-th key of that value, n the earlier rounds with the same key and lane (which come one
    // after the other).
    const uint32_t before = __shfl_up_sync(kFull, mine, 1);
    const int of = __shfl_up_sync(kFull, from, 1);
    const unsigned fresh = __ballot_sync(kFull, lane == 0 || before != mine || of != from);
    int n = lane - (31 - __clz(fresh & (lanemask_lt() | 1u << lane)));
    int id = -1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t w = __shfl_sync(kFull, key[i], from);
        if (mine && w == mine && n-- == 0) id = map.first(from) + i;
    }

    float s = 0.f;
    float xj = id >= 0 ? widen(__ldg(row + id)) : -INFINITY;
    if (SIG) {
        s = id >= 0 ? sigmoid(xj) : 0.f;
    } else {
        xj = fminf(xj, kMaxFinite);
        if (a.r.renormalize) m = warp_max(xj);
        s = id >= 0 ? expf(xj - m) : 0.f;
    }
    if (a.r.renormalize) z = lanes_sum<32>(s);
    if (lane < k) {
        a.topk_idx[t * k + lane] = id;
        a.topk_weights[t * k + lane] = id >= 0 && z > 0.f ? s / z * a.r.scale : 0.f;
    }
}

// W lanes own a token: 16 where they can (k <= 16, E <= 512), for two tokens a
// warp, because the part that entries need (lane j: entry j) takes as many
// instructions for two tokens as for one.  Measured with 16 and 32 lanes, from a
// graph: 32768 tokens x 256 experts, softmax, bf16: 10.9 and 13.9 us (the memory alone
// 5.4; 65% of the issue slots are used: a token's loads and reductions wait for one
// another); 4120 x 160, sigmoid, fp32: 2.7 and 3.3 us.
// DENSE: softmax without renormalisation, where every logit has a gradient and
// the row is read; otherwise only the chosen logits are.  The row of the
// gradient is written whole (zeros, or the dense part), then lane j writes the
// value of entry j over it.
template <typename L, int W, int V, bool DENSE>
__global__ void __launch_bounds__(kRouteWarps * 32) route_backward_kernel(RouteArgs a, const int64_t *topk_idx, bool vec) {
    const int lane = threadIdx.x & (W - 1);
    const int64_t own = ((int64_t)blockIdx.x * kRouteWarps * 32 + threadIdx.x) / W;
    const bool live = own < a.T;                 // (lanes beyond the last token repeat it and write nothing)
    const int64_t t = live ? own : a.T - 1;
    const int E = (int)a.E, k = (int)a.k;
    const bool sig = a.r.scoring == EP_SCORE_SIGMOID, norm = a.r.renormalize;
    const L *row = reinterpret_cast<const L *>(a.logits) + t * a.stride;
    L *out = reinterpret_cast<L *>(a.grad_logits) + t * a.grad_stride;
    float x[V];
    if (DENSE) load_turns<L, W, V>(row, E, lane, vec, x);
    const int64_t id = lane < k ? topk_idx[t * k + lane] : -1;
    float g = lane < k ? a.grad_weights[t * k + lane] * a.r.scale : 0.f;
    const bool in_range = id >= 0 && id < E;
    int st = id != -1 && !in_range ? EP_STATUS_BAD_EXPERT : 0;
    const int wl = threadIdx.x & 31;
    const unsigned same = __match_any_sync(kFull, in_range ? (int)id + (wl / W) * kMaxExperts : -2 - wl);
    const bool dup = in_range && (same & lanemask_lt());
    if (dup) st |= EP_STATUS_DUP_EXPERT;
    if (st) raise_status(a.dev_status, st);
    float xj = in_range && !dup ? widen(__ldg(row + id)) : -INFINITY;
    const bool kept = xj > -INFINITY;
    if (!kept) g = 0.f;
    float m = 0.f, inv_z = 1.f;
    if (!sig) xj = fminf(xj, kMaxFinite);
    if (!sig && norm) m = lanes_max<W>(kept ? xj : -INFINITY);
    if (DENSE) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = x[i] > -INFINITY ? fminf(x[i], kMaxFinite) : -INFINITY;    // (NaN: takes no part)
            m = fmaxf(m, x[i]);
        }
        m = lanes_max<W>(m);
        const float base = m > -INFINITY ? m : 0.f;
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = expf(x[i] - base);
            z += x[i];
        }
        z = lanes_sum<W>(z);
        inv_z = z > 0.f ? 1.f / z : 0.f;
    }
    const float s = !kept ? 0.f : sig ? sigmoid(xj) : expf(xj - m) * inv_z;
    // sigmoid: s' = sigmoid(x) sigmoid(-x); 1 - s has no digits left where s rounds to 1.  Renormalised weights: the
    // quotients s_j / S, not 1 / S, which is infinite for scores that are not yet 0.
    float p = s, d = g, mean = 0.f;
    if (norm) {
        const float total = lanes_sum<W>(s);
        p = total > 0.f ? s / total : 0.f;
        d = g - lanes_sum<W>(g * p);
    } else if (DENSE) {
        mean = lanes_sum<W>(g * s);
        d = g - mean;
    }
    const float v = sig ? d * p * sigmoid(-xj) : d * p;   // (softmax, renormalised: the mean is already taken out)
    const float f = -inv_z * mean;
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = DENSE ? x[i] * f : 0.f;
    if (live) store_turns<L, W, V>(out, E, lane, vec, x);
    __syncwarp();
    if (kept && live) narrow(v, out[id]);
}

}  // namespace

// The kernel for V = 1, 2, 4, .. 32 (at least `per`) experts a lane, W lanes a token
#define EP_ROUTE_CASES(W, KERNEL, ...)                                          \
    do {                                                                        \
        if (per <= 1) EP_ROUTE_LAUNCH(W, 1, KERNEL, __VA_ARGS__);               \
        else if (per <= 2) EP_ROUTE_LAUNCH(W, 2, KERNEL, __VA_ARGS__);          \
        else if (per <= 4) EP_ROUTE_LAUNCH(W, 4, KERNEL, __VA_ARGS__);          \
        else if (per <= 8) EP_ROUTE_LAUNCH(W, 8, KERNEL, __VA_ARGS__);          \
        else if (per <= 16) EP_ROUTE_LAUNCH(W, 16, KERNEL, __VA_ARGS__);        \
        else EP_ROUTE_LAUNCH(W, 32, KERNEL, __VA_ARGS__);                       \
    } while (0)
#define EP_ROUTE_LAUNCH(W, V, KERNEL, ...) KERNEL(W, V)<<<grid, kRouteWarps * 32, 0, st>>>(__VA_ARGS__)

cudaError_t launch_route(const RouteArgs &a, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.T + kRouteWarps - 1) / kRouteWarps);
    const int E = (int)a.E, G = a.r.num_groups, size = a.bf16 ? 2 : 4;
    // A group to lanes of its own, if 32 lanes of up to 32 experts can hold them so.  65536 tokens, 160 experts in 8
    // groups: 61 us, against 140 us with the groups taken one after the other; 384 in 12: 127 against 302.
    LaneMap map{1, E, 5, (E + 31) / 32};
    if (a.r.topk_groups < G && G <= 32) {
        int log = 5;
        while (G << log > 32) --log;
        const int each = (E / G + (1 << log) - 1) >> log;
        if (each <= 32) map = LaneMap{G, E / G, log, each};
    }
    const int per = map.each;
    const bool full = (per & (per - 1)) == 0 && per * 32 == E;       // every lane has V experts, one after the other
    const int64_t bytes = (int64_t)per * size, width = bytes > 16 ? 16 : bytes;
    const bool vec = full && (uintptr_t)a.logits % width == 0 && a.stride * size % width == 0;
#define EP_ROUTE_BG(W, V) route_kernel<uint16_t, V, kSigmoid>
#define EP_ROUTE_BL(W, V) route_kernel<uint16_t, V, kSoftmaxLogit>
#define EP_ROUTE_BS(W, V) route_kernel<uint16_t, V, kSoftmaxScore>
#define EP_ROUTE_FG(W, V) route_kernel<float, V, kSigmoid>
#define EP_ROUTE_FL(W, V) route_kernel<float, V, kSoftmaxLogit>
#define EP_ROUTE_FS(W, V) route_kernel<float, V, kSoftmaxScore>
    if (a.r.scoring == EP_SCORE_SIGMOID) {
        if (a.bf16) EP_ROUTE_CASES(32, EP_ROUTE_BG, a, map, vec);
        else EP_ROUTE_CASES(32, EP_ROUTE_FG, a, map, vec);
    } else if (a.r.softmax_key == EP_KEY_LOGIT) {
        if (a.bf16) EP_ROUTE_CASES(32, EP_ROUTE_BL, a, map, vec);
        else EP_ROUTE_CASES(32, EP_ROUTE_FL, a, map, vec);
    } else {
        if (a.bf16) EP_ROUTE_CASES(32, EP_ROUTE_BS, a, map, vec);
        else EP_ROUTE_CASES(32, EP_ROUTE_FS, a, map, vec);
    }
    return cudaGetLastError();
}

cudaError_t launch_route_backward(const RouteArgs &a, const int64_t *topk_idx, cudaStream_t st) {
    const bool half = a.k <= 16 && a.E <= 512;
    const int W = half ? 16 : 32, per = ((int)a.E + W - 1) / W, size = a.bf16 ? 2 : 4, tokens = kRouteWarps * 32 / W;
    const unsigned grid = (unsigned)((a.T + tokens - 1) / tokens);
    const auto in16 = [&](const void *p, int64_t stride) { return (uintptr_t)p % 16 == 0 && stride * size % 16 == 0; };
    const bool vec = in16(a.logits, a.stride) && in16(a.grad_logits, a.grad_stride);
#define EP_ROUTE_BD(W, V) route_backward_kernel<uint16_t, W, V, true>
#define EP_ROUTE_BC(W, V) route_backward_kernel<uint16_t, W, V, false>
#define EP_ROUTE_FD(W, V) route_backward_kernel<float, W, V, true>
#define EP_ROUTE_FC(W, V) route_backward_kernel<float, W, V, false>
#define EP_ROUTE_BACK(W)                                                             \
    do {                                                                             \
        if (dense) {                                                                 \
            if (a.bf16) EP_ROUTE_CASES(W, EP_ROUTE_BD, a, topk_idx, vec);   \
            else EP_ROUTE_CASES(W, EP_ROUTE_FD, a, topk_idx, vec);          \
        } else {                                                                     \
            if (a.bf16) EP_ROUTE_CASES(W, EP_ROUTE_BC, a, topk_idx, vec);   \
            else EP_ROUTE_CASES(W, EP_ROUTE_FC, a, topk_idx, vec);          \
        }                                                                            \
    } while (0)
    const bool dense = a.r.scoring == EP_SCORE_SOFTMAX && !a.r.renormalize;
    if (half) EP_ROUTE_BACK(16);
    else EP_ROUTE_BACK(32);
    return cudaGetLastError();
}

}  // namespace ep
