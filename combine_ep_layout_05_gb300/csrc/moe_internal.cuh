// Arguments and launchers of routing, combine backward and the expert
// products.
#pragma once

#include "ep_internal.cuh"

namespace ep {

// How a launch follows the one before it on its stream.  kAfter and kBeside begin while that one runs (programmatic
// dependent launch) once each of its CTAs has said that they may; each says so behind its own wait, if it has one.
//   kFirst   an ordinary launch, the first of a call
//   kAfter   waits at its start for the launch before it: it reads what that one writes
//   kBeside  runs beside it and waits at its end: it reads only what launches before that one wrote (which are over:
//            that one has waited for them, or began behind one that had) and writes nothing that one reads or writes
enum { kFirst, kAfter, kBeside };

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

constexpr int kMoeFewTokens = 64;      // most tokens of ep_moe_few: a tile of every expert holds them

constexpr int kMoeCtas = 152;          // and most CTAs that work on it

// A part of a unit: sums of two blocks of 128 matrix rows by 256 threads, which have every other 16 columns
__host__ __device__ constexpr int moe_part_columns(int pad) { return (pad + 31) / 32 * 16; }
__host__ __device__ constexpr int moe_part_floats(int pad) { return 2 * moe_part_columns(pad) * 256; }

struct MoeFewArgs {
    RouteArgs route;         // T, E, k, logits and where the routing goes
    int64_t H, I;
    const uint16_t *x, *residual;
    const uint8_t *gate_up, *down;
    const float *gate_up_scales, *down_scales;
    uint8_t *xq;             // workspace: [T, H] codes, [T, H / 128] scales of x
    float *x_scales;
    uint8_t *h;              // [T k, I] codes, [T k, I / 128] scales, [T k, H] products, [H / 128] counters
    float *h_scales, *y;
    unsigned *arrived;
    float *parts;            // [kMoeCtas][2][moe_part_floats]: parts of units
    unsigned *split;         // [2][kMoeCtas]: their steps
    uint16_t *out;
    int64_t wait_clocks;
};

// A dense product out[r, c] = sum over l of A(r, l) B(c, l), R x C x L, with its
// epilogue: ep_linear, and the two products of its gradient.
struct LinearArgs {
    int64_t R, C, L;         // (SwiGLU: C output columns, 2 C rows of B)
    int act;
    const float *bias;
    const uint16_t *residual;
    int64_t residual_stride; // elements between rows, as below
    bool out32;              // fp32 output, else bf16
    void *out;
    int64_t out_stride;
    uint16_t *pre;           // or null: bf16 pre-activations [R, C or 2 C]
    int64_t pre_stride;
    int out_align, pre_align, residual_align;   // see row_align
    int splits;              // parts of the contraction (at least 1; every part has steps)
    int row_tiles, col_tiles, split_steps, steps;           // by the launcher, as is
    int half_rows, half_cols;    // rows and columns of a tile of a pair that a CTA brings
    int a_bytes, stage_bytes, stages;   // a step's A, its operands, and how many of these
    bool boxes;              // whether results leave by tensor map
    int order;               // kFirst, kAfter or kBeside
    int64_t split_stride;    // elements between the partial sums of two splits
    int32_t *dev_status;
    int64_t wait_clocks;
};

// alignment, in bytes, of every 16th column of rows that start `stride` bytes apart
inline int row_align(const void *p, int64_t stride) {
    const uintptr_t a = (uintptr_t)p | (uintptr_t)stride;
    return a % 32 == 0 ? 32 : a % 16 == 0 ? 16 : 1;
}

enum { kFormForward, kFormGradX, kFormGradW };   // what the operands are: see launch_linear
struct LinearOperand {
    const uint16_t *p;
    int64_t rows, cols, stride;   // as they lie in memory: elements of a row side by side
};

struct ActGradArgs {         // G = grad_out * act'(pre), bf16, and its column sums
    int64_t M, N;            // (SwiGLU: N columns of grad_out, 2 N of pre and G)
    int act;
    bool grad32;
    const void *grad;
    int64_t grad_stride;
    const uint16_t *pre;
    uint16_t *G;             // or null: only the sums
    int64_t G_stride;
    float *sums;             // or null: [blocks, columns of G] partial sums
    int blocks;
    float *bias;             // the sums' sum
};

struct SumPartsArgs {        // out = sum of parts [rows, cols], cols a multiple of 8, one after the other
    const float *p;
    int parts;
    int64_t rows, cols;
    bool out32;
    void *out;
    int64_t stride;          // elements between rows of out
    bool vec;                // by the launcher (always kAfter)
};

// Parts into which the contraction L of an R x C product is split
int linear_splits(int64_t R, int64_t C, int64_t L);
// What the two kernels take, in us: linear.cu's in `splits` parts, and linear_few.cu's
double linear_time(int64_t R, int64_t C, int64_t L, bool swiglu, int splits);
double linear_few_time(int form, const LinearArgs &a);
cudaError_t launch_linear_few(int form, const LinearArgs &a, const LinearOperand &A, const LinearOperand &B, cudaStream_t st);
cudaError_t launch_linear(int form, LinearArgs a, const LinearOperand &A, const LinearOperand &B, cudaStream_t st);
cudaError_t launch_moe_few(const MoeFewArgs &a, cudaStream_t st);
cudaError_t launch_act_grad(const ActGradArgs &a, cudaStream_t st);
int act_grad_blocks(int64_t M, int64_t N);
cudaError_t launch_sum_parts(SumPartsArgs a, cudaStream_t st);

cudaError_t launch_route(const RouteArgs &a, cudaStream_t st);
cudaError_t launch_route_backward(const RouteArgs &a, const int64_t *topk_idx, cudaStream_t st);
cudaError_t launch_combine_backward(int layout, const CombineArgs &a, const uint16_t *grad_out, uint16_t *grad_y,
                                    float *grad_weights, cudaStream_t st);
cudaError_t launch_expert(const ExpertArgs &a, cudaStream_t st);        // chooses between
cudaError_t launch_expert_many(const ExpertArgs &a, cudaStream_t st);
cudaError_t launch_expert_few(const ExpertArgs &a, cudaStream_t st);

}  // namespace ep
