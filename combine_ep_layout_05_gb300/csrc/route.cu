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
#include "route_device.cuh"

namespace ep {

namespace {

constexpr int kRouteWarps = 4;

// load_lane for work that needs no order (the gradient): W lanes share a row of
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

template <typename L, int V, int KEY>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a, LaneMap map, bool vec) {
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const int k = (int)a.k, lo = map.first(lane), held = map.count(lane);
    const L *row = reinterpret_cast<const L *>(a.logits) + t * a.stride;
    float x[V], b[V];
    load_lane<L, V>(row, lo, held, vec, x);
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = 0.f;
    if (a.bias) load_lane<float, V>(a.bias, lo, held, vec && ((uintptr_t)a.bias & 15) == 0, b);
    int id;
    float weight;
    route_one<V, KEY>(a, map, x, b, [&](int e) { return widen(__ldg(row + e)); }, id, weight);
    if (lane < k) {
        a.topk_idx[t * k + lane] = id;
        a.topk_weights[t * k + lane] = weight;
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
    const int E = (int)a.E, size = a.bf16 ? 2 : 4;
    const LaneMap map = lane_map(a);
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
