// Routing: a token's logits -> its k experts and their weights, and the
// gradient of the weights with respect to the logits.
//
// A warp owns one token.  Lane l holds the V consecutive experts l * V ..
// l * V + V - 1 in registers (V a power of two, 32 V >= E), so a row is read
// once and "lowest index first" is lane order.  Keys are compared as
// unsigned words in the order of the floats; 0 stands for "not eligible".
#include "ep_internal.cuh"

namespace ep {

namespace {

constexpr int kRouteWarps = 4;

// order-preserving word of a float that is neither NaN nor -inf (always > 0)
__device__ __forceinline__ uint32_t order_word(float f) {
    const uint32_t u = __float_as_uint(f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_float(uint32_t w) {
    return __uint_as_float(w & 0x80000000u ? w ^ 0x80000000u : ~w);
}

__device__ __forceinline__ float sigmoid(float x) { return __frcp_rn(1.f + expf(-x)); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

template <typename L>
__device__ __forceinline__ float load_logit(const L *p);
template <>
__device__ __forceinline__ float load_logit<float>(const float *p) { return *p; }
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }

template <typename L, int V>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(RouteArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const int E = (int)a.E, k = (int)a.k;
    const bool sig = a.r.scoring == EP_SCORE_SIGMOID;
    const L *row = reinterpret_cast<const L *>(a.logits) + t * a.stride;
    float x[V];
    uint32_t key[V];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        x[i] = e < E ? load_logit(row + e) : -INFINITY;
        const float b = a.bias && e < E ? a.bias[e] : 0.f;
        const float f = (sig ? sigmoid(x[i]) : x[i]) + b;
        nan |= x[i] != x[i] || b != b;
        const bool fit = x[i] > -INFINITY && f > -INFINITY;   // false for NaN
        key[i] = fit ? order_word(f) : 0;
    }
    if (nan) raise_status(a.dev_status, EP_STATUS_BAD_LOGIT);

    float m = 0.f, z = 1.f;   // softmax over the logits that are numbers
    if (!sig && !a.r.renormalize) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (x[i] > -INFINITY) m = fmaxf(m, fminf(x[i], 3.402823466e38f));
        m = warp_max(m);
        z = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (x[i] > -INFINITY) z += expf(fminf(x[i], 3.402823466e38f) - m);
        z = warp_sum(z);
    }

    const int G = a.r.num_groups;
    if (G > 1 && a.r.topk_groups < G) {
        // scores of the groups: lane g % 32 keeps group g's word
        const int per = E / G;
        uint32_t score[kMaxExperts / 32];
        for (int s = 0; s < (G + 31) / 32; ++s) score[s] = 0;
        for (int g = 0; g < G; ++g) {
            const int lo = g * per, hi = lo + per;
            uint32_t b1 = 0, b2 = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane * V + i;
                const uint32_t v = e >= lo && e < hi ? key[i] : 0;
                if (v > b1) { b2 = b1; b1 = v; }
                else if (v > b2) b2 = v;
            }
            const uint32_t top = __reduce_max_sync(kFull, b1);
            uint32_t w = top;
            if (a.r.group_best == 2) {
                const unsigned who = __ballot_sync(kFull, b1 == top);
                const bool mine = lane == __ffs(who) - 1;
                const uint32_t second = __reduce_max_sync(kFull, mine ? b2 : b1);
                if (top && second) w = order_word(order_float(top) + order_float(second));
            }
            if ((g & 31) == lane) score[g >> 5] = w;
        }
        // the topk_groups best, lowest group first among equals
        uint32_t kept[kMaxExperts / 32];
        for (int s = 0; s < (G + 31) / 32; ++s) kept[s] = 0;
        for (int n = 0; n < a.r.topk_groups; ++n) {
            uint32_t b = 0;
            int at = 0x7fffffff;
            for (int s = 0; s < (G + 31) / 32; ++s)
                if (score[s] > b) { b = score[s]; at = s * 32 + lane; }
            const uint32_t top = __reduce_max_sync(kFull, b);
            if (!top) break;
            const int g = (int)__reduce_min_sync(kFull, b == top ? (unsigned)at : 0x7fffffffu);
            for (int s = 0; s < (G + 31) / 32; ++s) {
                if (g == s * 32 + lane) score[s] = 0;
                if ((g >> 5) == s) kept[s] |= 1u << (g & 31);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int g = (lane * V + i) / per;
            if (g >= G || !((kept[g >> 5] >> (g & 31)) & 1)) key[i] = 0;
        }
    }

    // k times the largest key; lane j keeps entry j
    int id = -1;
    float xj = -INFINITY;
    for (int j = 0; j < k; ++j) {
        uint32_t b = 0;
        int at = 0;
        float bx = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (key[i] > b) { b = key[i]; at = i; bx = x[i]; }
        const uint32_t top = __reduce_max_sync(kFull, b);
        if (!top) break;
        const int win = __ffs(__ballot_sync(kFull, b == top)) - 1;
        const int e = win * V + __shfl_sync(kFull, at, win);
        const float ex = __shfl_sync(kFull, bx, win);
        if (lane == j) { id = e; xj = ex; }
        if (lane == win) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i == at) key[i] = 0;
        }
    }
    float s = 0.f;
    if (sig) {
        s = id >= 0 ? sigmoid(xj) : 0.f;
    } else {
        xj = fminf(xj, 3.402823466e38f);
        if (a.r.renormalize) m = warp_max(id >= 0 ? xj : -INFINITY);
        s = id >= 0 ? expf(xj - m) : 0.f;
    }
    if (a.r.renormalize) z = warp_sum(s);
    if (lane < k) {
        a.topk_idx[t * k + lane] = id;
        a.topk_weights[t * k + lane] = id >= 0 && z > 0.f ? s / z * a.r.scale : 0.f;
    }
}

template <typename L>
__device__ __forceinline__ void store_grad(L *p, float v);
template <>
__device__ __forceinline__ void store_grad<float>(float *p, float v) { *p = v; }
template <>
__device__ __forceinline__ void store_grad<uint16_t>(uint16_t *p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.f); }

template <typename L, int V>
__global__ void __launch_bounds__(kRouteWarps * 32) route_backward_kernel(RouteArgs a, const int64_t *topk_idx) {
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const int E = (int)a.E, k = (int)a.k;
    const bool sig = a.r.scoring == EP_SCORE_SIGMOID, norm = a.r.renormalize;
    const L *row = reinterpret_cast<const L *>(a.logits) + t * a.stride;
    L *out = reinterpret_cast<L *>(a.grad_logits) + t * a.grad_stride;
    const int64_t id = lane < k ? topk_idx[t * k + lane] : -1;
    float g = lane < k ? a.grad_weights[t * k + lane] * a.r.scale : 0.f;
    const bool in_range = id >= 0 && id < E;
    int st = id != -1 && !in_range ? EP_STATUS_BAD_EXPERT : 0;
    const unsigned same = __match_any_sync(kFull, in_range ? (long long)id : -2 - lane);
    const bool dup = in_range && (same & lanemask_lt());
    if (dup) st |= EP_STATUS_DUP_EXPERT;
    if (st) raise_status(a.dev_status, st);
    float xj = in_range && !dup ? load_logit(row + id) : -INFINITY;
    const bool kept = xj > -INFINITY;
    if (!kept) g = 0.f;
    float x[V];
    float m = 0.f, inv_z = 1.f;
    if (!sig) xj = fminf(xj, 3.402823466e38f);
    if (!sig && norm) m = warp_max(kept ? xj : -INFINITY);
    if (!sig && !norm) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
            x[i] = e < E ? load_logit(row + e) : -INFINITY;
            x[i] = x[i] > -INFINITY ? fminf(x[i], 3.402823466e38f) : -INFINITY;
            m = fmaxf(m, x[i]);
        }
        m = warp_max(m);
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = x[i] > -INFINITY ? expf(x[i] - m) : 0.f;
            z += x[i];
        }
        z = warp_sum(z);
        inv_z = z > 0.f ? 1.f / z : 0.f;
    }
    const float s = !kept ? 0.f : sig ? sigmoid(xj) : expf(xj - m) * inv_z;
    float ds = g;
    if (norm) {
        const float total = warp_sum(s), inv = total > 0.f ? 1.f / total : 0.f;
        ds = (g - warp_sum(g * s) * inv) * inv;
        if (!kept) ds = 0.f;
    }
    float mean = 0.f, v;
    if (sig) {
        v = ds * s * (1.f - s);
    } else if (norm) {
        v = s * ds;       // sum_j ds_j s_j = 0: the mean is already taken out
    } else {
        mean = warp_sum(ds * s);
        v = s * (ds - mean);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = !sig && !norm ? -(x[i] * inv_z) * mean : 0.f;
    for (int j = 0; j < k; ++j) {
        const int e = __shfl_sync(kFull, kept ? (int)id : -1, j);
        const float vj = __shfl_sync(kFull, v, j);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (e == lane * V + i) x[i] = vj;
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane * V + i < E) store_grad(out + lane * V + i, x[i]);
}

}  // namespace

#define EP_ROUTE_CASES(KERNEL, L, ...)                                            \
    if (a.E <= 32) KERNEL<L, 1><<<grid, kRouteWarps * 32, 0, st>>>(__VA_ARGS__);  \
    else if (a.E <= 64) KERNEL<L, 2><<<grid, kRouteWarps * 32, 0, st>>>(__VA_ARGS__);   \
    else if (a.E <= 128) KERNEL<L, 4><<<grid, kRouteWarps * 32, 0, st>>>(__VA_ARGS__);  \
    else if (a.E <= 256) KERNEL<L, 8><<<grid, kRouteWarps * 32, 0, st>>>(__VA_ARGS__);  \
    else if (a.E <= 512) KERNEL<L, 16><<<grid, kRouteWarps * 32, 0, st>>>(__VA_ARGS__); \
    else KERNEL<L, 32><<<grid, kRouteWarps * 32, 0, st>>>(__VA_ARGS__);

cudaError_t launch_route(const RouteArgs &a, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.T + kRouteWarps - 1) / kRouteWarps);
    if (a.bf16) { EP_ROUTE_CASES(route_kernel, uint16_t, a) }
    else { EP_ROUTE_CASES(route_kernel, float, a) }
    return cudaGetLastError();
}

cudaError_t launch_route_backward(const RouteArgs &a, const int64_t *topk_idx, cudaStream_t st) {
    const unsigned grid = (unsigned)((a.T + kRouteWarps - 1) / kRouteWarps);
    if (a.bf16) { EP_ROUTE_CASES(route_backward_kernel, uint16_t, a, topk_idx) }
    else { EP_ROUTE_CASES(route_backward_kernel, float, a, topk_idx) }
    return cudaGetLastError();
}

}  // namespace ep
