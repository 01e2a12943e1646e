// Arguments and launchers of routing, combine backward and the expert
// products.
#pragma once

#include "ep_internal.cuh"

namespace ep {

struct RouteArgs {
    int64_t T, E, k;
    ep_router r;
    bool bf16;               // logits and their gradient: bf16, else fp32
    const void *logits;
    int64_t stride;          // elements between rows of logits
    const float *bias;
    int64_t *topk_idx;
    float *topk_weights;
    const float *grad_weights;
    void *grad_logits;
    int64_t grad_stride;
    int32_t *dev_status;
};

constexpr int64_t kWaitClocks = (int64_t)1 << 32;   // after which the expert products' waits give up: some two seconds

struct ExpertArgs {
    Dims d;
    int64_t N, K;            // matrix rows (2 * I with SwiGLU) and channels
    const uint8_t *a;
    const float *a_scales;
    const uint8_t *w;
    const float *w_scales;
    const int32_t *tokens_per_expert;
    uint16_t *y;             // bf16 output, or
    uint8_t *q;              // e4m3 codes and scales of the SwiGLU
    float *q_scales;
    int32_t *dev_status;
    int64_t wait_clocks;
};

cudaError_t launch_route(const RouteArgs &a, cudaStream_t st);
cudaError_t launch_route_backward(const RouteArgs &a, const int64_t *topk_idx, cudaStream_t st);
cudaError_t launch_combine_backward(int layout, const CombineArgs &a, const uint16_t *grad_out, uint16_t *grad_y,
                                    float *grad_weights, cudaStream_t st);
cudaError_t launch_expert(const ExpertArgs &a, cudaStream_t st);        // chooses between
cudaError_t launch_expert_many(const ExpertArgs &a, cudaStream_t st);
cudaError_t launch_expert_few(const ExpertArgs &a, cudaStream_t st);

}  // namespace ep
