// What both routing kernels share: keys as ordered words, scores, sums over
// lanes, and which experts a lane holds.
#pragma once

#include "moe_internal.cuh"

namespace ep {

namespace {

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

// A group to lanes of its own, if 32 lanes of up to 32 experts can hold them so.  65536 tokens, 160 experts in 8
// groups: 61 us, against 140 us with the groups taken one after the other; 384 in 12: 127 against 302.
inline LaneMap lane_map(const RouteArgs &a) {
    const int E = (int)a.E, G = a.r.num_groups;
    if (a.r.topk_groups < G && G <= 32) {
        int log = 5;
        while (G << log > 32) --log;
        const int each = (E / G + (1 << log) - 1) >> log;
        if (each <= 32) return LaneMap{G, E / G, log, each};
    }
    return LaneMap{1, E, 5, (E + 31) / 32};
}

// widest vector that V elements of a lane make up
template <int BYTES> struct Vec { typedef uint4 T; };
template <> struct Vec<8> { typedef uint2 T; };
template <> struct Vec<4> { typedef uint32_t T; };
template <> struct Vec<2> { typedef uint16_t T; };

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

// A token's routing by a warp, from the lanes' logits x and bias b (those that a lane does not hold: -inf); logit(e) is
// logit e.  Lane j gets entry j.
template <int V, int KEY, typename F>
__device__ __forceinline__ void route_one(const RouteArgs &a, const LaneMap &map, const float (&x)[V], const float (&b)[V],
                                          const F &logit, int &id, float &weight) {
    constexpr bool SIG = KEY == kSigmoid, by_score = KEY == kSoftmaxScore;
    const int lane = threadIdx.x & 31, k = (int)a.k, lo = map.first(lane);
    uint32_t key[V];
    bool nan = false;
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
    id = -1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const uint32_t w = __shfl_sync(kFull, key[i], from);
        if (mine && w == mine && n-- == 0) id = map.first(from) + i;
    }

    float s = 0.f;
    float xj = id >= 0 ? logit(id) : -INFINITY;
    if (SIG) {
        s = id >= 0 ? sigmoid(xj) : 0.f;
    } else {
        xj = fminf(xj, kMaxFinite);
        if (a.r.renormalize) m = warp_max(xj);
        s = id >= 0 ? expf(xj - m) : 0.f;
    }
    if (a.r.renormalize) z = lanes_sum<32>(s);
    weight = id >= 0 && z > 0.f ? s / z * a.r.scale : 0.f;
}

}  // namespace

}  // namespace ep
