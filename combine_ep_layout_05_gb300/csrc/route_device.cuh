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

}  // namespace

}  // namespace ep
