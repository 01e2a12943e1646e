// C-ABI entry points: argument checks, problem sizes, launches.
// The semantics of every entry point are documented in include/ep.h.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "moe_internal.cuh"

// bf16 dispatch goes through the bulk-copy engine from this many tokens on;
// below it (decode and low-latency sizes) 16-byte register copies spread
// over more warps finish sooner.
#ifndef EP_DISPATCH_BULK_MIN_TOKENS
#define EP_DISPATCH_BULK_MIN_TOKENS 2048
#endif

namespace {

thread_local char g_err[512] = "";

int fail(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return code;
}

int cuda_fail(cudaError_t e, const char *where) {
    return fail(EP_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

// Fills d from p; returns false (with the message set) if p describes no problem.
bool make_dims(const ep_problem *p, ep::Dims &d) {
    if (!p) return fail(EP_ERR_INVALID_ARG, "problem is NULL"), false;
    d.T = p->num_tokens;
    d.H = p->hidden;
    d.k = p->num_topk;
    d.E = p->num_experts;
    d.R = p->num_ranks;
    d.G = p->gpus_per_node;
    if (d.T < 0 || d.H < 8 || d.H % 8 || d.k < 1 || d.k > ep::kMaxTopk || d.E < 1 ||
        d.E > ep::kMaxExperts || d.R < 1 || d.R > ep::kMaxRanks || d.G < 1)
        return fail(EP_ERR_INVALID_ARG,
                    "sizes out of range (T=%lld H=%lld k=%lld E=%lld R=%lld G=%lld): need T>=0, H>=8, H%%8==0, "
                    "1<=k<=32, 1<=E<=1024, 1<=R<=64, G>=1",
                    (long long)d.T, (long long)d.H, (long long)d.k, (long long)d.E, (long long)d.R,
                    (long long)d.G),
               false;
    if (d.E % d.R) return fail(EP_ERR_INVALID_ARG, "num_experts %% num_ranks != 0"), false;
    if (d.R % d.G) return fail(EP_ERR_INVALID_ARG, "num_ranks %% gpus_per_node != 0"), false;
    if (d.T % d.R) return fail(EP_ERR_INVALID_ARG, "num_tokens %% num_ranks != 0"), false;
    d.N = d.R / d.G;
    d.Er = d.E / d.R;
    d.En = d.E / d.N;
    d.Tr = d.T / d.R;
    if (d.Tr > INT32_MAX) return fail(EP_ERR_INVALID_ARG, "tokens per rank exceed int32"), false;
    d.cps = (d.Tr + ep::kChunk - 1) / ep::kChunk;
    d.cols = d.R + d.E + d.N;
    ep::div_magic(d.Er, d.er_mul, d.er_shift);
    ep::div_magic(d.En, d.en_mul, d.en_shift);
    return true;
}

// Splits a token row into pieces when there are too few tokens to give every
// warp slot of the GPU a unit of work.  granule: elements one warp step covers.
void pick_pieces(const ep::Dims &d, int64_t granule, int64_t &pieces, int64_t &piece_elems) {
    const int64_t target = (int64_t)ep::num_sms() * 32;   // warps to keep busy
    const int64_t max_pieces = (d.H + granule - 1) / granule;
    int64_t want = d.T > 0 ? (target + d.T - 1) / d.T : 1;
    if (want > max_pieces) want = max_pieces;
    if (want < 1) want = 1;
    int64_t per = (d.H + want - 1) / want;
    per = (per + granule - 1) / granule * granule;
    piece_elems = per;
    pieces = (d.H + per - 1) / per;
}

int64_t unit_grid(int64_t units, int cap) {
    int64_t g = (units + 7) / 8;
    if (g > cap) g = cap;
    return g < 1 ? 1 : g;
}

}  // namespace

namespace ep {
int set_last_error(int code, const char *fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_err, sizeof g_err, fmt, ap);
    va_end(ap);
    return code;
}
}  // namespace ep

extern "C" {

const char *ep_last_error_string(void) { return g_err; }

int ep_get_status(const int32_t *dev_status, int32_t *status_out, ep_stream_t stream) {
    g_err[0] = 0;
    if (!dev_status || !aligned(dev_status, 4)) return fail(EP_ERR_INVALID_ARG, "dev_status NULL or misaligned");
    cudaStream_t st = (cudaStream_t)stream;
    int32_t word = 0;
    cudaError_t e = cudaMemcpyAsync(&word, dev_status, sizeof word, cudaMemcpyDeviceToHost, st);
    if (!e) e = cudaStreamSynchronize(st);
    if (e) return cuda_fail(e, "ep_get_status");
    if (status_out) *status_out = word;
    if (word) return fail(EP_ERR_DEVICE, "the kernels reported status bits 0x%x", (unsigned)word);
    return EP_OK;
}

int64_t ep_recv_rows(const ep_problem *p, int layout) {
    ep::Dims d;
    if (!make_dims(p, d)) return -1;
    if (layout == EP_RANK_MAJOR) return d.R * d.R * d.Tr;
    if (layout == EP_EXPERT_MAJOR) return d.E * d.R * d.Tr;
    fail(EP_ERR_INVALID_ARG, "unknown layout %d", layout);
    return -1;
}

size_t ep_layout_workspace_bytes(const ep_problem *p) {
    ep::Dims d;
    if (!make_dims(p, d)) return 0;
    const size_t b = (size_t)(d.R * d.cps * d.cols) * sizeof(int32_t);
    return (b + 255) / 256 * 256;
}

double ep_rdma_physical_formula(int64_t algo_tokens, int64_t num_nodes) {
    if (num_nodes < 1) return 0.0;
    return (double)(algo_tokens * (num_nodes - 1)) / (double)num_nodes;
}

int ep_layout(const ep_problem *p, const int64_t *topk_idx, uint8_t *is_token_in_rank,
              int32_t *tokens_per_rank, int32_t *tokens_per_expert, int32_t *tokens_per_node,
              int32_t *recv_tokens_per_rank, int32_t *rank_slot, int32_t *token_major_offset,
              int32_t *expert_slot, int32_t *node_slot, int64_t *algo_per_rank,
              int64_t *physical_exact_per_rank, void *workspace, size_t workspace_bytes, int32_t *dev_status,
              ep_stream_t stream) {
    g_err[0] = 0;
    ep::Dims d;
    if (!make_dims(p, d)) return EP_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    if (d.T == 0) {
        // nothing routed: counts are zero
        cudaError_t e = cudaSuccess;
        if (tokens_per_rank && !e) e = cudaMemsetAsync(tokens_per_rank, 0, d.R * d.R * 4, st);
        if (tokens_per_expert && !e) e = cudaMemsetAsync(tokens_per_expert, 0, d.R * d.E * 4, st);
        if (tokens_per_node && !e) e = cudaMemsetAsync(tokens_per_node, 0, d.R * d.N * 4, st);
        if (recv_tokens_per_rank && !e) e = cudaMemsetAsync(recv_tokens_per_rank, 0, d.R * 4, st);
        if (algo_per_rank && !e) e = cudaMemsetAsync(algo_per_rank, 0, d.R * 8, st);
        if (physical_exact_per_rank && !e) e = cudaMemsetAsync(physical_exact_per_rank, 0, d.R * 8, st);
        return e ? cuda_fail(e, "ep_layout memset") : EP_OK;
    }
    if (!topk_idx || !aligned(topk_idx, 8)) return fail(EP_ERR_INVALID_ARG, "topk_idx NULL or misaligned");
    if (!workspace || !aligned(workspace, 16))
        return fail(EP_ERR_INVALID_ARG, "workspace NULL or not 16-byte aligned");
    if (workspace_bytes < ep_layout_workspace_bytes(p))
        return fail(EP_ERR_INVALID_ARG, "workspace too small: %zu < %zu", workspace_bytes,
                    ep_layout_workspace_bytes(p));
    const void *i32s[] = {tokens_per_rank, tokens_per_expert, tokens_per_node, recv_tokens_per_rank,
                          rank_slot, token_major_offset, expert_slot, node_slot, dev_status};
    for (const void *q : i32s)
        if (!aligned(q, 4)) return fail(EP_ERR_INVALID_ARG, "int32 output not 4-byte aligned");
    if (!aligned(algo_per_rank, 8) || !aligned(physical_exact_per_rank, 8))
        return fail(EP_ERR_INVALID_ARG, "int64 output not 8-byte aligned");
    ep::LayoutArgs a{};
    a.d = d;
    a.topk_idx = topk_idx;
    a.is_token_in_rank = is_token_in_rank;
    a.tokens_per_rank = tokens_per_rank;
    a.tokens_per_expert = tokens_per_expert;
    a.tokens_per_node = tokens_per_node;
    a.recv_tokens_per_rank = recv_tokens_per_rank;
    a.rank_slot = rank_slot;
    a.token_major_offset = token_major_offset;
    a.expert_slot = expert_slot;
    a.node_slot = node_slot;
    a.algo_per_rank = algo_per_rank;
    a.phys_per_rank = physical_exact_per_rank;
    a.chunk_counts = (int32_t *)workspace;
    a.dev_status = dev_status;
    cudaError_t e = ep::launch_layout(a, a.chunk_counts, st);
    return e ? cuda_fail(e, "ep_layout launch") : EP_OK;
}

int ep_rdma_token_count(const ep_problem *p, const int64_t *topk_idx, int64_t *algo_per_rank,
                        int64_t *physical_exact_per_rank, int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    ep::Dims d;
    if (!make_dims(p, d)) return EP_ERR_INVALID_ARG;
    if (!algo_per_rank || !aligned(algo_per_rank, 8) || !aligned(physical_exact_per_rank, 8))
        return fail(EP_ERR_INVALID_ARG, "algo_per_rank NULL or outputs misaligned");
    if (d.T > 0 && (!topk_idx || !aligned(topk_idx, 8)))
        return fail(EP_ERR_INVALID_ARG, "topk_idx NULL or misaligned");
    if (!aligned(dev_status, 4)) return fail(EP_ERR_INVALID_ARG, "dev_status misaligned");
    cudaStream_t st = (cudaStream_t)stream;
    cudaError_t e = cudaMemsetAsync(algo_per_rank, 0, d.R * 8, st);
    if (!e && physical_exact_per_rank) e = cudaMemsetAsync(physical_exact_per_rank, 0, d.R * 8, st);
    if (e) return cuda_fail(e, "ep_rdma_token_count memset");
    if (d.T == 0) return EP_OK;
    ep::RdmaArgs a{};
    a.d = d;
    a.topk_idx = topk_idx;
    a.algo = (unsigned long long *)algo_per_rank;
    a.phys = (unsigned long long *)physical_exact_per_rank;
    a.dev_status = dev_status;
    e = ep::launch_rdma_count(a, st);
    return e ? cuda_fail(e, "ep_rdma_token_count launch") : EP_OK;
}

}  // extern "C"

namespace {

// Checks ep_dispatch's arguments and fills a (everything but the launch);
// mode: the kernel that will run.  Returns EP_OK or the error code.
int prepare_dispatch(const ep::Dims &d, int layout, int dtype, const uint16_t *x, const int64_t *topk_idx,
                     const int32_t *rank_slot, const int32_t *expert_slot, void *recv, float *recv_scales,
                     int32_t *dev_status, ep::DispatchArgs &a, int &mode) {
    if (layout != EP_RANK_MAJOR && layout != EP_EXPERT_MAJOR)
        return fail(EP_ERR_INVALID_ARG, "unknown layout %d", layout);
    if (dtype != EP_BF16 && dtype != EP_FP8_E4M3) return fail(EP_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (dtype == EP_FP8_E4M3 && d.H % 128) return fail(EP_ERR_INVALID_ARG, "FP8 needs hidden %% 128 == 0");
    if (d.T == 0) return EP_OK;
    if (!x || !aligned(x, 16)) return fail(EP_ERR_INVALID_ARG, "x NULL or not 16-byte aligned");
    if (!recv || !aligned(recv, 16)) return fail(EP_ERR_INVALID_ARG, "recv NULL or not 16-byte aligned");
    if (layout == EP_RANK_MAJOR && (!rank_slot || !aligned(rank_slot, 4)))
        return fail(EP_ERR_INVALID_ARG, "rank_slot NULL or misaligned");
    if (layout == EP_EXPERT_MAJOR && (!topk_idx || !aligned(topk_idx, 8) || !expert_slot || !aligned(expert_slot, 4)))
        return fail(EP_ERR_INVALID_ARG, "topk_idx / expert_slot NULL or misaligned");
    if (dtype == EP_FP8_E4M3 && (!recv_scales || !aligned(recv_scales, 4)))
        return fail(EP_ERR_INVALID_ARG, "recv_scales NULL or misaligned");
    if (!aligned(dev_status, 4)) return fail(EP_ERR_INVALID_ARG, "dev_status misaligned");
    a.d = d;
    a.x = x;
    a.topk_idx = topk_idx;
    a.rank_slot = rank_slot;
    a.expert_slot = expert_slot;
    a.recv = recv;
    a.recv_scales = recv_scales;
    a.dev_status = dev_status;
    if (dtype == EP_BF16 && d.T >= EP_DISPATCH_BULK_MIN_TOKENS) {
        // bulk-copy path: whole rows, or the fewest pieces that fit one
        // shared-memory buffer each
        const int64_t maxe = ep::dispatch_bulk_piece_bytes() / 2;
        a.pieces = (d.H + maxe - 1) / maxe;
        a.piece_elems = ((d.H + a.pieces - 1) / a.pieces + 7) / 8 * 8;
        a.pieces = (d.H + a.piece_elems - 1) / a.piece_elems;
        mode = ep::kFusedBulk;
    } else {
        pick_pieces(d, dtype == EP_BF16 ? 256 : 512, a.pieces, a.piece_elems);
        mode = dtype == EP_BF16 ? ep::kFusedLsu : ep::kFusedFp8;
    }
    return EP_OK;
}

int launch_prepared_dispatch(int layout, int dtype, int mode, const ep::DispatchArgs &a, cudaStream_t st) {
    cudaError_t e;
    if (mode == ep::kFusedBulk) {
        e = ep::launch_dispatch_bulk(layout, a, st);
    } else {
        const int64_t grid = unit_grid(a.d.T * a.pieces, ep::dispatch_grid_cap(layout, dtype));
        e = ep::launch_dispatch(layout, dtype, a, (int)grid, st);
    }
    return e ? cuda_fail(e, "ep_dispatch launch") : EP_OK;
}

}  // namespace

extern "C" {

int ep_dispatch(const ep_problem *p, int layout, int dtype, const uint16_t *x, const int64_t *topk_idx,
                const int32_t *rank_slot, const int32_t *expert_slot, void *recv, float *recv_scales,
                int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    ep::Dims d;
    if (!make_dims(p, d)) return EP_ERR_INVALID_ARG;
    ep::DispatchArgs a{};
    int mode = 0;
    const int rc = prepare_dispatch(d, layout, dtype, x, topk_idx, rank_slot, expert_slot, recv, recv_scales,
                                    dev_status, a, mode);
    if (rc != EP_OK || d.T == 0) return rc;
    return launch_prepared_dispatch(layout, dtype, mode, a, (cudaStream_t)stream);
}

size_t ep_layout_dispatch_workspace_bytes(const ep_problem *p) {
    const size_t w = ep_layout_workspace_bytes(p);
    return w ? w + 256 : 0;
}

int ep_layout_dispatch(const ep_problem *p, int layout, int dtype, const uint16_t *x, const int64_t *topk_idx,
                       uint8_t *is_token_in_rank, int32_t *tokens_per_rank, int32_t *tokens_per_expert,
                       int32_t *tokens_per_node, int32_t *recv_tokens_per_rank, int32_t *rank_slot,
                       int32_t *token_major_offset, int32_t *expert_slot, int32_t *node_slot,
                       int64_t *algo_per_rank, int64_t *physical_exact_per_rank, void *recv, float *recv_scales,
                       void *workspace, size_t workspace_bytes, int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    ep::Dims d;
    if (!make_dims(p, d)) return EP_ERR_INVALID_ARG;
    cudaStream_t st = (cudaStream_t)stream;
    const size_t lw = ep_layout_workspace_bytes(p);
    if (d.T == 0)
        return ep_layout(p, topk_idx, is_token_in_rank, tokens_per_rank, tokens_per_expert, tokens_per_node,
                         recv_tokens_per_rank, rank_slot, token_major_offset, expert_slot, node_slot,
                         algo_per_rank, physical_exact_per_rank, workspace, workspace_bytes, dev_status, stream);
    if (!topk_idx || !aligned(topk_idx, 8)) return fail(EP_ERR_INVALID_ARG, "topk_idx NULL or misaligned");
    if (!workspace || !aligned(workspace, 16))
        return fail(EP_ERR_INVALID_ARG, "workspace NULL or not 16-byte aligned");
    if (workspace_bytes < ep_layout_dispatch_workspace_bytes(p))
        return fail(EP_ERR_INVALID_ARG, "workspace too small: %zu < %zu", workspace_bytes,
                    ep_layout_dispatch_workspace_bytes(p));
    const void *i32s[] = {tokens_per_rank, tokens_per_expert, tokens_per_node, recv_tokens_per_rank,
                          rank_slot, token_major_offset, expert_slot, node_slot, dev_status};
    for (const void *q : i32s)
        if (!aligned(q, 4)) return fail(EP_ERR_INVALID_ARG, "int32 output not 4-byte aligned");
    if (!aligned(algo_per_rank, 8) || !aligned(physical_exact_per_rank, 8))
        return fail(EP_ERR_INVALID_ARG, "int64 output not 8-byte aligned");
    ep::DispatchArgs da{};
    int mode = 0;
    int rc = prepare_dispatch(d, layout, dtype, x, topk_idx, rank_slot, expert_slot, recv, recv_scales, dev_status,
                              da, mode);
    if (rc != EP_OK) return rc;
    ep::LayoutArgs la{};
    la.d = d;
    la.topk_idx = topk_idx;
    la.is_token_in_rank = is_token_in_rank;
    la.tokens_per_rank = tokens_per_rank;
    la.tokens_per_expert = tokens_per_expert;
    la.tokens_per_node = tokens_per_node;
    la.recv_tokens_per_rank = recv_tokens_per_rank;
    la.rank_slot = rank_slot;
    la.token_major_offset = token_major_offset;
    la.expert_slot = expert_slot;
    la.node_slot = node_slot;
    la.algo_per_rank = algo_per_rank;
    la.phys_per_rank = physical_exact_per_rank;
    la.chunk_counts = (int32_t *)workspace;
    la.dev_status = dev_status;
    unsigned *bar = (unsigned *)((char *)workspace + lw);
    cudaError_t e = ep::launch_layout_dispatch(layout, mode, la, da, bar, st);
    if (e == cudaErrorCooperativeLaunchTooLarge || e == cudaErrorNotSupported) {
        // no room for a resident grid: the same work as two calls
        (void)cudaGetLastError();
        rc = ep_layout(p, topk_idx, is_token_in_rank, tokens_per_rank, tokens_per_expert, tokens_per_node,
                       recv_tokens_per_rank, rank_slot, token_major_offset, expert_slot, node_slot, algo_per_rank,
                       physical_exact_per_rank, workspace, workspace_bytes, dev_status, stream);
        if (rc != EP_OK) return rc;
        return launch_prepared_dispatch(layout, dtype, mode, da, st);
    }
    return e ? cuda_fail(e, "ep_layout_dispatch launch") : EP_OK;
}

int ep_combine(const ep_problem *p, int layout, const uint16_t *y, const int64_t *topk_idx,
               const float *topk_weights, const int32_t *rank_slot, const int32_t *expert_slot,
               uint16_t *out, int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    ep::Dims d;
    if (!make_dims(p, d)) return EP_ERR_INVALID_ARG;
    if (layout != EP_RANK_MAJOR && layout != EP_EXPERT_MAJOR)
        return fail(EP_ERR_INVALID_ARG, "unknown layout %d", layout);
    if (d.T == 0) return EP_OK;
    if (!y || !aligned(y, 16)) return fail(EP_ERR_INVALID_ARG, "y NULL or not 16-byte aligned");
    if (!out || !aligned(out, 16)) return fail(EP_ERR_INVALID_ARG, "out NULL or not 16-byte aligned");
    if (!topk_idx || !aligned(topk_idx, 8) || !topk_weights || !aligned(topk_weights, 4))
        return fail(EP_ERR_INVALID_ARG, "topk_idx / topk_weights NULL or misaligned");
    if (layout == EP_RANK_MAJOR && (!rank_slot || !aligned(rank_slot, 4)))
        return fail(EP_ERR_INVALID_ARG, "rank_slot NULL or misaligned");
    if (layout == EP_EXPERT_MAJOR && (!expert_slot || !aligned(expert_slot, 4)))
        return fail(EP_ERR_INVALID_ARG, "expert_slot NULL or misaligned");
    if (!aligned(dev_status, 4)) return fail(EP_ERR_INVALID_ARG, "dev_status misaligned");
    ep::CombineArgs a{};
    a.d = d;
    a.y = y;
    a.topk_idx = topk_idx;
    a.topk_weights = topk_weights;
    a.rank_slot = rank_slot;
    a.expert_slot = expert_slot;
    a.out = out;
    a.dev_status = dev_status;
    cudaError_t e = ep::launch_combine(layout, a, (cudaStream_t)stream);
    return e ? cuda_fail(e, "ep_combine launch") : EP_OK;
}

int ep_dequant_fp8(const ep_problem *p, int layout, const int64_t *topk_idx, const int32_t *rank_slot,
                   const int32_t *expert_slot, const uint8_t *recv, const float *recv_scales, uint16_t *y,
                   ep_stream_t stream) {
    g_err[0] = 0;
    ep::Dims d;
    if (!make_dims(p, d)) return EP_ERR_INVALID_ARG;
    if (layout != EP_RANK_MAJOR && layout != EP_EXPERT_MAJOR)
        return fail(EP_ERR_INVALID_ARG, "unknown layout %d", layout);
    if (d.H % 128) return fail(EP_ERR_INVALID_ARG, "FP8 needs hidden %% 128 == 0");
    if (d.T == 0) return EP_OK;
    if (!recv || !aligned(recv, 16) || !recv_scales || !aligned(recv_scales, 4) || !y || !aligned(y, 16))
        return fail(EP_ERR_INVALID_ARG, "recv / recv_scales / y NULL or misaligned");
    if (layout == EP_RANK_MAJOR && (!rank_slot || !aligned(rank_slot, 4)))
        return fail(EP_ERR_INVALID_ARG, "rank_slot NULL or misaligned");
    if (layout == EP_EXPERT_MAJOR && (!topk_idx || !aligned(topk_idx, 8) || !expert_slot || !aligned(expert_slot, 4)))
        return fail(EP_ERR_INVALID_ARG, "topk_idx / expert_slot NULL or misaligned");
    ep::DispatchArgs a{};
    a.d = d;
    a.x = nullptr;
    a.topk_idx = topk_idx;
    a.rank_slot = rank_slot;
    a.expert_slot = expert_slot;
    a.recv = const_cast<uint8_t *>(recv);
    a.recv_scales = const_cast<float *>(recv_scales);
    a.dev_status = nullptr;
    cudaError_t e = ep::launch_dequant(layout, a, y, (cudaStream_t)stream);
    return e ? cuda_fail(e, "ep_dequant_fp8 launch") : EP_OK;
}

int ep_selftest_wait_timeout(uint32_t *words, uint32_t polls, int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    if (!words || !aligned(words, 4) || !aligned(dev_status, 4))
        return fail(EP_ERR_INVALID_ARG, "words NULL or misaligned");
    if (polls > (1u << 20)) return fail(EP_ERR_INVALID_ARG, "polls must be at most 2^20 for a self-test");
    cudaError_t e = cudaMemsetAsync(words, 0, 2 * sizeof(uint32_t), (cudaStream_t)stream);
    if (!e) e = ep::launch_wait_selftest((unsigned *)words, polls, dev_status, (cudaStream_t)stream);
    return e ? cuda_fail(e, "ep_selftest_wait_timeout launch") : EP_OK;
}

int ep_combine_quantize(const ep_problem *p, int layout, int fmt, const uint16_t *y, const int64_t *topk_idx,
                        const int32_t *rank_slot, const int32_t *expert_slot, uint8_t *wq, void *wscales,
                        ep_stream_t stream) {
    g_err[0] = 0;
    ep::Dims d;
    if (!make_dims(p, d)) return EP_ERR_INVALID_ARG;
    if (layout != EP_RANK_MAJOR && layout != EP_EXPERT_MAJOR)
        return fail(EP_ERR_INVALID_ARG, "unknown layout %d", layout);
    if (fmt != EP_WIRE_MXFP8 && fmt != EP_WIRE_NVFP4) return fail(EP_ERR_INVALID_ARG, "unknown wire format %d", fmt);
    if (d.H % (fmt == EP_WIRE_MXFP8 ? 32 : 16))
        return fail(EP_ERR_INVALID_ARG, "hidden must be a multiple of the wire block");
    if (d.T == 0) return EP_OK;
    if (!y || !aligned(y, 16) || !wq || !aligned(wq, 16) || !wscales || !aligned(wscales, 2))
        return fail(EP_ERR_INVALID_ARG, "y / wq / wscales NULL or misaligned");
    if (layout == EP_RANK_MAJOR && (!rank_slot || !aligned(rank_slot, 4)))
        return fail(EP_ERR_INVALID_ARG, "rank_slot NULL or misaligned");
    if (layout == EP_EXPERT_MAJOR && (!topk_idx || !aligned(topk_idx, 8) || !expert_slot || !aligned(expert_slot, 4)))
        return fail(EP_ERR_INVALID_ARG, "topk_idx / expert_slot NULL or misaligned");
    ep::DispatchArgs a{};
    a.d = d;
    a.x = nullptr;
    a.topk_idx = topk_idx;
    a.rank_slot = rank_slot;
    a.expert_slot = expert_slot;
    a.recv = nullptr;
    a.recv_scales = nullptr;
    a.dev_status = nullptr;
    pick_pieces(d, 512, a.pieces, a.piece_elems);
    cudaError_t e = ep::launch_wire_quant(layout, fmt, a, y, wq, wscales, (cudaStream_t)stream);
    return e ? cuda_fail(e, "ep_combine_quantize launch") : EP_OK;
}

int ep_combine_wire(const ep_problem *p, int layout, int fmt, const uint8_t *wq, const void *wscales,
                    const int64_t *topk_idx, const float *topk_weights, const int32_t *rank_slot,
                    const int32_t *expert_slot, uint16_t *out, int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    ep::Dims d;
    if (!make_dims(p, d)) return EP_ERR_INVALID_ARG;
    if (layout != EP_RANK_MAJOR && layout != EP_EXPERT_MAJOR)
        return fail(EP_ERR_INVALID_ARG, "unknown layout %d", layout);
    if (fmt != EP_WIRE_MXFP8 && fmt != EP_WIRE_NVFP4) return fail(EP_ERR_INVALID_ARG, "unknown wire format %d", fmt);
    if (d.H % (fmt == EP_WIRE_MXFP8 ? 32 : 16))
        return fail(EP_ERR_INVALID_ARG, "hidden must be a multiple of the wire block");
    if (d.T == 0) return EP_OK;
    if (!wq || !aligned(wq, 16) || !wscales || !aligned(wscales, 2) || !out || !aligned(out, 16))
        return fail(EP_ERR_INVALID_ARG, "wq / wscales / out NULL or misaligned");
    if (!topk_idx || !aligned(topk_idx, 8) || !topk_weights || !aligned(topk_weights, 4))
        return fail(EP_ERR_INVALID_ARG, "topk_idx / topk_weights NULL or misaligned");
    if (layout == EP_RANK_MAJOR && (!rank_slot || !aligned(rank_slot, 4)))
        return fail(EP_ERR_INVALID_ARG, "rank_slot NULL or misaligned");
    if (layout == EP_EXPERT_MAJOR && (!expert_slot || !aligned(expert_slot, 4)))
        return fail(EP_ERR_INVALID_ARG, "expert_slot NULL or misaligned");
    if (!aligned(dev_status, 4)) return fail(EP_ERR_INVALID_ARG, "dev_status misaligned");
    ep::CombineArgs a{};
    a.d = d;
    a.y = nullptr;
    a.topk_idx = topk_idx;
    a.topk_weights = topk_weights;
    a.rank_slot = rank_slot;
    a.expert_slot = expert_slot;
    a.out = out;
    a.dev_status = dev_status;
    pick_pieces(d, 512, a.pieces, a.piece_elems);
    cudaError_t e = ep::launch_combine_wire(layout, fmt, a, wq, wscales, (cudaStream_t)stream);
    return e ? cuda_fail(e, "ep_combine_wire launch") : EP_OK;
}

int64_t ep_stage_rows(const ep_problem *p) {
    ep::Dims d;
    if (!make_dims(p, d)) return -1;
    return d.N * d.R * d.Tr;
}

int ep_dispatch_two_level(const ep_problem *p, const uint16_t *x, const int32_t *rank_slot,
                          const int32_t *node_slot, uint16_t *stage, uint16_t *recv, int32_t *dev_status,
                          ep_stream_t stream) {
    g_err[0] = 0;
    ep::Dims d;
    if (!make_dims(p, d)) return EP_ERR_INVALID_ARG;
    if (d.T == 0) return EP_OK;
    if (!x || !aligned(x, 16) || !stage || !aligned(stage, 16) || !recv || !aligned(recv, 16))
        return fail(EP_ERR_INVALID_ARG, "x / stage / recv NULL or not 16-byte aligned");
    if (!rank_slot || !aligned(rank_slot, 4) || !node_slot || !aligned(node_slot, 4))
        return fail(EP_ERR_INVALID_ARG, "rank_slot / node_slot NULL or misaligned");
    if (!aligned(dev_status, 4)) return fail(EP_ERR_INVALID_ARG, "dev_status misaligned");
    cudaStream_t st = (cudaStream_t)stream;
    // hop 1: one copy per (token, node) into the node-major staging buffer
    ep::DispatchArgs a{};
    a.d = d;
    a.x = x;
    a.rank_slot = rank_slot;
    a.node_slot = node_slot;
    a.recv = stage;
    a.dev_status = dev_status;
    cudaError_t e;
    if (d.T >= EP_DISPATCH_BULK_MIN_TOKENS) {
        const int64_t maxe = ep::dispatch_bulk_piece_bytes() / 2;
        a.pieces = (d.H + maxe - 1) / maxe;
        a.piece_elems = ((d.H + a.pieces - 1) / a.pieces + 7) / 8 * 8;
        a.pieces = (d.H + a.piece_elems - 1) / a.piece_elems;
        e = ep::launch_dispatch_bulk(ep::kNodeMajor, a, st);
    } else {
        pick_pieces(d, 256, a.pieces, a.piece_elems);
        e = ep::launch_dispatch(ep::kNodeMajor, EP_BF16, a, (int)unit_grid(d.T * a.pieces,
                                ep::dispatch_grid_cap(ep::kNodeMajor, EP_BF16)), st);
    }
    if (e) return cuda_fail(e, "ep_dispatch_two_level hop 1");
    // hop 2: each staged row to the token's ranks inside the node
    pick_pieces(d, 256, a.pieces, a.piece_elems);
    e = ep::launch_forward(a, stage, recv, st);
    return e ? cuda_fail(e, "ep_dispatch_two_level hop 2") : EP_OK;
}

int ep_combine_two_level(const ep_problem *p, const uint16_t *y, const int64_t *topk_idx,
                         const float *topk_weights, const int32_t *rank_slot, const int32_t *node_slot,
                         uint16_t *stage, uint16_t *out, int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    ep::Dims d;
    if (!make_dims(p, d)) return EP_ERR_INVALID_ARG;
    if (d.T == 0) return EP_OK;
    if (!y || !aligned(y, 16) || !stage || !aligned(stage, 16) || !out || !aligned(out, 16))
        return fail(EP_ERR_INVALID_ARG, "y / stage / out NULL or not 16-byte aligned");
    if (!topk_idx || !aligned(topk_idx, 8) || !topk_weights || !aligned(topk_weights, 4))
        return fail(EP_ERR_INVALID_ARG, "topk_idx / topk_weights NULL or misaligned");
    if (!rank_slot || !aligned(rank_slot, 4) || !node_slot || !aligned(node_slot, 4))
        return fail(EP_ERR_INVALID_ARG, "rank_slot / node_slot NULL or misaligned");
    if (!aligned(dev_status, 4)) return fail(EP_ERR_INVALID_ARG, "dev_status misaligned");
    ep::CombineArgs a{};
    a.d = d;
    a.y = y;
    a.topk_idx = topk_idx;
    a.topk_weights = topk_weights;
    a.rank_slot = rank_slot;
    a.node_slot = node_slot;
    a.out = out;
    a.dev_status = dev_status;
    pick_pieces(d, 256, a.pieces, a.piece_elems);
    cudaError_t e = ep::launch_combine_two_level(a, stage, (cudaStream_t)stream);
    return e ? cuda_fail(e, "ep_combine_two_level launch") : EP_OK;
}

}  // extern "C"

namespace {

// Checks what ep_route and ep_route_backward share and fills a.
int prepare_route(const ep_problem *p, const ep_router *r, int dtype, const void *logits, int64_t stride,
                  int32_t *dev_status, ep::RouteArgs &a) {
    ep::Dims d;
    if (!make_dims(p, d)) return EP_ERR_INVALID_ARG;
    if (!r) return fail(EP_ERR_INVALID_ARG, "router is NULL");
    if (r->scoring != EP_SCORE_SOFTMAX && r->scoring != EP_SCORE_SIGMOID)
        return fail(EP_ERR_INVALID_ARG, "unknown scoring %d", r->scoring);
    if (r->num_groups < 1 || d.E % r->num_groups)
        return fail(EP_ERR_INVALID_ARG, "num_experts must be a multiple of num_groups >= 1");
    if (r->topk_groups < 1 || r->topk_groups > r->num_groups)
        return fail(EP_ERR_INVALID_ARG, "topk_groups must be in 1..num_groups");
    if (r->group_best != 1 && r->group_best != 2) return fail(EP_ERR_INVALID_ARG, "group_best must be 1 or 2");
    if (!std::isfinite(r->scale)) return fail(EP_ERR_INVALID_ARG, "scale must be finite");
    if (r->softmax_key != EP_KEY_LOGIT && r->softmax_key != EP_KEY_SCORE)
        return fail(EP_ERR_INVALID_ARG, "unknown softmax_key %d", r->softmax_key);
    if (dtype != EP_BF16 && dtype != EP_FP32) return fail(EP_ERR_INVALID_ARG, "logits must be EP_BF16 or EP_FP32");
    if (stride < d.E) return fail(EP_ERR_INVALID_ARG, "logits_row_stride smaller than num_experts");
    if (!aligned(dev_status, 4)) return fail(EP_ERR_INVALID_ARG, "dev_status misaligned");
    if (d.T > 0 && (!logits || !aligned(logits, dtype == EP_BF16 ? 2 : 4)))
        return fail(EP_ERR_INVALID_ARG, "logits NULL or misaligned");
    a.T = d.T;
    a.E = d.E;
    a.k = d.k;
    a.r = *r;
    a.bf16 = dtype == EP_BF16;
    a.logits = logits;
    a.stride = stride;
    a.dev_status = dev_status;
    return EP_OK;
}

// Checks what ep_expert_gemm and ep_expert_swiglu share and fills a.
int prepare_expert(const ep_problem *p, int64_t N, int64_t K, const uint8_t *act, const float *act_scales,
                   const uint8_t *w, const float *w_scales, const int32_t *tokens_per_expert, int32_t *dev_status,
                   ep::ExpertArgs &a) {
    ep::Dims &d = a.d;
    if (!make_dims(p, d)) return EP_ERR_INVALID_ARG;
    if (K < 128 || K % 128 || K > (1 << 24))
        return fail(EP_ERR_INVALID_ARG, "the product's channels must be a multiple of 128, at most 2^24");
    if (N < 8 || N % 8 || N > (1 << 24))
        return fail(EP_ERR_INVALID_ARG, "out_features must be a multiple of 8, at most 2^24");
    if (N * K >= (int64_t)1 << 40) return fail(EP_ERR_INVALID_ARG, "out_features * channels must be below 2^40");
    if (d.T > 0 && d.E > INT32_MAX / d.T) return fail(EP_ERR_INVALID_ARG, "num_experts * num_tokens exceeds int32");
    // tiles of 64 rows x 128 columns are counted in 32 bits, with room for a step of the grid beyond the last
    if (d.E * d.T / 64 + d.E > (INT32_MAX - 65536) / ((N + 127) / 128))
        return fail(EP_ERR_INVALID_ARG, "num_experts * num_tokens * out_features too large (about 2^44)");
    if (d.T > 0) {
        if (!act || !aligned(act, 16) || !w || !aligned(w, 16))
            return fail(EP_ERR_INVALID_ARG, "a / w NULL or not 16-byte aligned");
        if (!act_scales || !aligned(act_scales, 4) || !w_scales || !aligned(w_scales, 4))
            return fail(EP_ERR_INVALID_ARG, "a_scales / w_scales NULL or misaligned");
        if (!tokens_per_expert || !aligned(tokens_per_expert, 4))
            return fail(EP_ERR_INVALID_ARG, "tokens_per_expert NULL or misaligned");
    }
    if (!aligned(dev_status, 4)) return fail(EP_ERR_INVALID_ARG, "dev_status misaligned");
    a.N = N;
    a.K = K;
    a.a = act;
    a.a_scales = act_scales;
    a.w = w;
    a.w_scales = w_scales;
    a.tokens_per_expert = tokens_per_expert;
    a.dev_status = dev_status;
    a.wait_clocks = ep::kWaitClocks;
    return EP_OK;
}

}  // namespace

extern "C" {

int ep_route(const ep_problem *p, const ep_router *r, int dtype, const void *logits, int64_t logits_row_stride,
             const float *bias, int64_t *topk_idx, float *topk_weights, int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    ep::RouteArgs a{};
    const int rc = prepare_route(p, r, dtype, logits, logits_row_stride, dev_status, a);
    if (rc != EP_OK || a.T == 0) return rc;
    if (!aligned(bias, 4)) return fail(EP_ERR_INVALID_ARG, "bias misaligned");
    if (!topk_idx || !aligned(topk_idx, 8) || !topk_weights || !aligned(topk_weights, 4))
        return fail(EP_ERR_INVALID_ARG, "topk_idx / topk_weights NULL or misaligned");
    a.bias = bias;
    a.topk_idx = topk_idx;
    a.topk_weights = topk_weights;
    cudaError_t e = ep::launch_route(a, (cudaStream_t)stream);
    return e ? cuda_fail(e, "ep_route launch") : EP_OK;
}

int ep_route_backward(const ep_problem *p, const ep_router *r, int dtype, const void *logits,
                      int64_t logits_row_stride, const int64_t *topk_idx, const float *grad_weights,
                      void *grad_logits, int64_t grad_row_stride, int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    ep::RouteArgs a{};
    const int rc = prepare_route(p, r, dtype, logits, logits_row_stride, dev_status, a);
    if (rc != EP_OK) return rc;
    if (grad_row_stride < a.E) return fail(EP_ERR_INVALID_ARG, "grad_row_stride smaller than num_experts");
    if (a.T == 0) return EP_OK;
    if (!topk_idx || !aligned(topk_idx, 8) || !grad_weights || !aligned(grad_weights, 4))
        return fail(EP_ERR_INVALID_ARG, "topk_idx / grad_weights NULL or misaligned");
    if (!grad_logits || !aligned(grad_logits, a.bf16 ? 2 : 4))
        return fail(EP_ERR_INVALID_ARG, "grad_logits NULL or misaligned");
    a.grad_weights = grad_weights;
    a.grad_logits = grad_logits;
    a.grad_stride = grad_row_stride;
    cudaError_t e = ep::launch_route_backward(a, topk_idx, (cudaStream_t)stream);
    return e ? cuda_fail(e, "ep_route_backward launch") : EP_OK;
}

int ep_combine_backward(const ep_problem *p, int layout, const uint16_t *grad_out, const uint16_t *y,
                        const int64_t *topk_idx, const float *topk_weights, const int32_t *rank_slot,
                        const int32_t *expert_slot, uint16_t *grad_y, float *grad_weights, int32_t *dev_status,
                        ep_stream_t stream) {
    g_err[0] = 0;
    ep::Dims d;
    if (!make_dims(p, d)) return EP_ERR_INVALID_ARG;
    if (layout != EP_RANK_MAJOR && layout != EP_EXPERT_MAJOR)
        return fail(EP_ERR_INVALID_ARG, "unknown layout %d", layout);
    if (!aligned(dev_status, 4)) return fail(EP_ERR_INVALID_ARG, "dev_status misaligned");
    if (d.T == 0 || (!grad_y && !grad_weights)) return EP_OK;
    if (!grad_out || !aligned(grad_out, 16)) return fail(EP_ERR_INVALID_ARG, "grad_out NULL or not 16-byte aligned");
    if (!aligned(grad_y, 16)) return fail(EP_ERR_INVALID_ARG, "grad_y not 16-byte aligned");
    if (!aligned(grad_weights, 4)) return fail(EP_ERR_INVALID_ARG, "grad_weights misaligned");
    if (grad_weights && (!y || !aligned(y, 16))) return fail(EP_ERR_INVALID_ARG, "y NULL or not 16-byte aligned");
    if (!topk_idx || !aligned(topk_idx, 8) || !topk_weights || !aligned(topk_weights, 4))
        return fail(EP_ERR_INVALID_ARG, "topk_idx / topk_weights NULL or misaligned");
    if (layout == EP_RANK_MAJOR && (!rank_slot || !aligned(rank_slot, 4)))
        return fail(EP_ERR_INVALID_ARG, "rank_slot NULL or misaligned");
    if (layout == EP_EXPERT_MAJOR && (!expert_slot || !aligned(expert_slot, 4)))
        return fail(EP_ERR_INVALID_ARG, "expert_slot NULL or misaligned");
    ep::CombineArgs a{};
    a.d = d;
    a.y = y;
    a.topk_idx = topk_idx;
    a.topk_weights = topk_weights;
    a.rank_slot = rank_slot;
    a.expert_slot = expert_slot;
    a.dev_status = dev_status;
    cudaError_t e = ep::launch_combine_backward(layout, a, grad_out, grad_y, grad_weights, (cudaStream_t)stream);
    return e ? cuda_fail(e, "ep_combine_backward launch") : EP_OK;
}

int ep_expert_gemm(const ep_problem *p, int64_t out_features, int64_t in_features, const uint8_t *act,
                   const float *a_scales, const uint8_t *w, const float *w_scales,
                   const int32_t *tokens_per_expert, uint16_t *y, int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    ep::ExpertArgs a{};
    const int rc = prepare_expert(p, out_features, in_features, act, a_scales, w, w_scales, tokens_per_expert,
                                  dev_status, a);
    if (rc != EP_OK || a.d.T == 0) return rc;
    if (!y || !aligned(y, 16)) return fail(EP_ERR_INVALID_ARG, "y NULL or not 16-byte aligned");
    a.y = y;
    cudaError_t e = ep::launch_expert(a, (cudaStream_t)stream);
    return e ? cuda_fail(e, "ep_expert_gemm launch") : EP_OK;
}

int ep_expert_swiglu(const ep_problem *p, int64_t intermediate, const uint8_t *act, const float *a_scales,
                     const uint8_t *w, const float *w_scales, const int32_t *tokens_per_expert, uint8_t *q,
                     float *q_scales, int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    ep::ExpertArgs a{};
    if (intermediate < 128 || intermediate % 128 || intermediate > (1 << 23))
        return fail(EP_ERR_INVALID_ARG, "intermediate must be a multiple of 128, at most 2^23");
    const int rc = prepare_expert(p, 2 * intermediate, p ? p->hidden : 0, act, a_scales, w, w_scales,
                                  tokens_per_expert, dev_status, a);
    if (rc != EP_OK || a.d.T == 0) return rc;
    if (!q || !aligned(q, 16) || !q_scales || !aligned(q_scales, 4))
        return fail(EP_ERR_INVALID_ARG, "q / q_scales NULL or misaligned");
    a.q = q;
    a.q_scales = q_scales;
    cudaError_t e = ep::launch_expert(a, (cudaStream_t)stream);
    return e ? cuda_fail(e, "ep_expert_swiglu launch") : EP_OK;
}

int ep_selftest_expert_timeout(const ep_problem *p, int kernel, int64_t out_features, int64_t in_features,
                               const uint8_t *act, const float *a_scales, const uint8_t *w, const float *w_scales,
                               const int32_t *tokens_per_expert, uint16_t *y, uint8_t *q, float *q_scales,
                               int64_t clocks, int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    if (kernel != EP_EXPERT_FEW_ROWS && kernel != EP_EXPERT_MANY_ROWS)
        return fail(EP_ERR_INVALID_ARG, "unknown kernel %d", kernel);
    if (clocks < 1 || clocks > ep::kWaitClocks) return fail(EP_ERR_INVALID_ARG, "clocks must be in 1..2^32");
    if (!dev_status) return fail(EP_ERR_INVALID_ARG, "dev_status is NULL");
    ep::ExpertArgs a{};
    const int rc = prepare_expert(p, out_features, in_features, act, a_scales, w, w_scales, tokens_per_expert,
                                  dev_status, a);
    if (rc != EP_OK || a.d.T == 0) return rc;
    if (y ? !aligned(y, 16) : !q || !aligned(q, 16) || !q_scales || !aligned(q_scales, 4) || out_features % 256)
        return fail(EP_ERR_INVALID_ARG, "y, or q and q_scales (out_features a multiple of 256), NULL or misaligned");
    a.y = y;
    a.q = y ? nullptr : q;
    a.q_scales = q_scales;
    a.wait_clocks = clocks;
    cudaError_t e = kernel == EP_EXPERT_FEW_ROWS ? ep::launch_expert_few(a, (cudaStream_t)stream)
                                                 : ep::launch_expert_many(a, (cudaStream_t)stream);
    return e ? cuda_fail(e, "ep_selftest_expert_timeout launch") : EP_OK;
}

}  // extern "C"

namespace {

// How a call does its work: by the kernel for few or for many rows (EP_LINEAR_*; -1: the faster one), with waits that
// give up after `clocks` cycles.  Self-tests choose.
struct Manner {
    int kernel = -1;
    int64_t clocks = ep::kWaitClocks;
};
bool self_test_manner(int kernel, int64_t clocks, const int32_t *dev_status) {
    if (kernel != EP_LINEAR_FEW_ROWS && kernel != EP_LINEAR_MANY_ROWS)
        return fail(EP_ERR_INVALID_ARG, "unknown kernel %d", kernel), false;
    if (clocks < 1 || clocks > ep::kWaitClocks) return fail(EP_ERR_INVALID_ARG, "clocks must be in 1..2^32"), false;
    if (!dev_status) return fail(EP_ERR_INVALID_ARG, "dev_status is NULL"), false;
    return true;
}

// whether the kernel for few rows does a product that the other one does in `many` us
bool by_few_rows(const Manner &how, int form, const ep::LinearArgs &a, double many) {
    return how.kernel < 0 ? ep::linear_few_time(form, a) < many : how.kernel == EP_LINEAR_FEW_ROWS;
}

// A dense product's sizes
struct LinearSizes {
    int64_t M, K, N, wide;      // wide: rows of w
};

bool linear_sizes(int64_t rows, int64_t in_features, int64_t out_features, int activation, LinearSizes &d) {
    if (activation < EP_ACT_NONE || activation > EP_ACT_SWIGLU)
        return fail(EP_ERR_INVALID_ARG, "unknown activation %d", activation), false;
    if (rows < 0 || rows > ((int64_t)1 << 30)) return fail(EP_ERR_INVALID_ARG, "rows must be in 0..2^30"), false;
    if (in_features < 8 || in_features % 8 || in_features > (1 << 24))
        return fail(EP_ERR_INVALID_ARG, "in_features must be a multiple of 8, at most 2^24"), false;
    if (out_features < 1 || out_features > (1 << 24))
        return fail(EP_ERR_INVALID_ARG, "out_features must be in 1..2^24"), false;
    d = LinearSizes{rows, in_features, out_features, activation == EP_ACT_SWIGLU ? 2 * out_features : out_features};
    // tiles of 256 x 128 of each product, and the splits of those that are few, are counted in 32 bits
    const auto tiles = [](int64_t a, int64_t b) { return ((a + 255) / 256) * ((b + 127) / 128); };
    if (tiles(d.M, d.wide) > (1 << 26) || tiles(d.M, d.K) > (1 << 26) || tiles(d.wide, d.K) > (1 << 26))
        return fail(EP_ERR_INVALID_ARG, "product too large (over 2^26 tiles of 256 x 128)"), false;
    return true;
}

size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

// The parts of ep_linear_backward's workspace: G [M, wide up to a multiple of 8], sums of its columns by block, and
// the parts of the two products (one after the other)
struct BackwardParts {
    int64_t g_stride;
    int blocks, splits_x, splits_w;
    size_t g, sums, parts, total;
};
BackwardParts backward_parts(const LinearSizes &d) {
    BackwardParts b;
    b.g_stride = (d.wide + 7) / 8 * 8;
    b.blocks = ep::act_grad_blocks(d.M, d.N);
    b.splits_x = ep::linear_splits(d.M, d.K, d.wide);
    b.splits_w = ep::linear_splits(d.wide, d.K, d.M);
    b.g = round16((size_t)d.M * b.g_stride * 2);
    b.sums = round16((size_t)b.blocks * d.wide * 4);
    const size_t px = b.splits_x > 1 ? (size_t)b.splits_x * d.M * d.K * 4 : 0;
    const size_t pw = b.splits_w > 1 ? (size_t)b.splits_w * d.wide * d.K * 4 : 0;
    b.parts = px > pw ? px : pw;
    b.total = b.g + b.sums + b.parts;
    return b;
}

// One product of the backward pass: straight into its output, or in parts that are summed.  order: how it follows the
// launches before it, and how the next may.
cudaError_t backward_product(int form, int64_t R, int64_t C, int64_t L, int splits, const ep::LinearOperand &A,
                             const ep::LinearOperand &B, bool out32, void *out, int64_t out_stride, float *parts,
                             int &order, bool &parts_used, const Manner &how, int32_t *dev_status, cudaStream_t st) {
    ep::LinearArgs a{};
    a.R = R;
    a.C = C;
    a.L = L;
    a.splits = splits;
    a.dev_status = dev_status;
    a.wait_clocks = how.clocks;
    a.out32 = out32;
    a.out = out;
    a.out_stride = out_stride;
    a.out_align = ep::row_align(out, out_stride * (out32 ? 4 : 2));
    a.order = order;
    order = ep::kBeside;       // (what comes next does not read this product)
    if (by_few_rows(how, form, a, ep::linear_time(R, C, L, false, splits)))
        return ep::launch_linear_few(form, a, A, B, st);
    const bool split = splits > 1;
    if (split && parts_used && a.order == ep::kBeside) a.order = ep::kAfter;   // the parts before are being summed
    parts_used |= split;
    a.out32 = split || out32;
    a.out = split ? parts : out;
    a.out_stride = split ? C : out_stride;
    a.split_stride = R * C;
    a.out_align = ep::row_align(a.out, a.out_stride * (a.out32 ? 4 : 2));
    if (cudaError_t e = ep::launch_linear(form, a, A, B, st)) return e;
    if (!split) return cudaSuccess;
    return ep::launch_sum_parts(ep::SumPartsArgs{parts, splits, R, C, out32, out, out_stride, false}, st);
}

int linear_call(const Manner &how, int64_t rows, int64_t in_features, int64_t out_features, int activation,
                const uint16_t *x, int64_t x_stride, const uint16_t *w, const float *bias, const uint16_t *residual,
                int64_t residual_stride, int out_dtype, void *out, int64_t out_stride, uint16_t *pre,
                int32_t *dev_status, ep_stream_t stream) {
    LinearSizes d;
    if (!linear_sizes(rows, in_features, out_features, activation, d)) return EP_ERR_INVALID_ARG;
    if (out_dtype != EP_BF16 && out_dtype != EP_FP32) return fail(EP_ERR_INVALID_ARG, "out must be EP_BF16 or EP_FP32");
    if (x_stride < d.K || x_stride % 8 || x_stride >= (int64_t)1 << 38)
        return fail(EP_ERR_INVALID_ARG, "x_stride must be a multiple of 8, at least in_features");
    if (out_stride < d.N || (residual && residual_stride < d.N))
        return fail(EP_ERR_INVALID_ARG, "out_stride / residual_stride smaller than out_features");
    if (!aligned(dev_status, 4)) return fail(EP_ERR_INVALID_ARG, "dev_status misaligned");
    if (d.M == 0) return EP_OK;
    if (!x || !aligned(x, 16) || !w || !aligned(w, 16))
        return fail(EP_ERR_INVALID_ARG, "x / w NULL or not 16-byte aligned");
    if (!out || !aligned(out, out_dtype == EP_FP32 ? 4 : 2)) return fail(EP_ERR_INVALID_ARG, "out NULL or misaligned");
    if (!aligned(bias, 4) || !aligned(residual, 2) || !aligned(pre, 2))
        return fail(EP_ERR_INVALID_ARG, "bias / residual / pre misaligned");
    ep::LinearArgs a{};
    a.R = d.M;
    a.C = d.N;
    a.L = d.K;
    a.act = activation;
    a.bias = bias;
    a.residual = residual;
    a.residual_stride = residual_stride;
    a.out32 = out_dtype == EP_FP32;
    a.out = out;
    a.out_stride = out_stride;
    a.pre = pre;
    a.pre_stride = d.wide;
    a.out_align = ep::row_align(out, out_stride * (a.out32 ? 4 : 2));
    a.residual_align = ep::row_align(residual, residual_stride * 2);
    // (the up half of a SwiGLU's pre-activations starts at column N)
    a.pre_align = ep::row_align(pre, (activation == EP_ACT_SWIGLU ? d.N : d.wide) * 2);
    a.splits = 1;
    a.dev_status = dev_status;
    a.wait_clocks = how.clocks;
    const ep::LinearOperand X{x, d.M, d.K, x_stride}, W{w, d.wide, d.K, d.K};
    const bool few = by_few_rows(how, ep::kFormForward, a,
                                 ep::linear_time(d.M, d.N, d.K, activation == EP_ACT_SWIGLU, 1));
    cudaError_t e = few ? ep::launch_linear_few(ep::kFormForward, a, X, W, (cudaStream_t)stream)
                        : ep::launch_linear(ep::kFormForward, a, X, W, (cudaStream_t)stream);
    return e ? cuda_fail(e, "ep_linear launch") : EP_OK;
}

int linear_backward_call(const Manner &how, int64_t rows, int64_t in_features, int64_t out_features, int activation,
                         int grad_dtype, const void *grad_out, int64_t grad_stride, const uint16_t *x,
                         int64_t x_stride, const uint16_t *w, const uint16_t *pre, uint16_t *grad_x,
                         int64_t grad_x_stride, int grad_w_dtype, void *grad_w, float *grad_bias, void *workspace,
                         size_t workspace_bytes, int32_t *dev_status, ep_stream_t stream) {
    LinearSizes d;
    if (!linear_sizes(rows, in_features, out_features, activation, d)) return EP_ERR_INVALID_ARG;
    const bool grad32 = grad_dtype == EP_FP32, w32 = grad_w_dtype == EP_FP32;
    if (!grad32 && grad_dtype != EP_BF16) return fail(EP_ERR_INVALID_ARG, "grad_out must be EP_BF16 or EP_FP32");
    if (grad_w && !w32 && grad_w_dtype != EP_BF16) return fail(EP_ERR_INVALID_ARG, "grad_w must be EP_BF16 or EP_FP32");
    if (grad_stride < d.N) return fail(EP_ERR_INVALID_ARG, "grad_stride smaller than out_features");
    if (grad_x && grad_x_stride < d.K) return fail(EP_ERR_INVALID_ARG, "grad_x_stride smaller than in_features");
    if (grad_w && (x_stride < d.K || x_stride % 8 || x_stride >= (int64_t)1 << 38))
        return fail(EP_ERR_INVALID_ARG, "x_stride must be a multiple of 8, at least in_features");
    if (!aligned(dev_status, 4)) return fail(EP_ERR_INVALID_ARG, "dev_status misaligned");
    if (!aligned(grad_w, 16)) return fail(EP_ERR_INVALID_ARG, "grad_w not 16-byte aligned");
    if (!aligned(grad_bias, 4) || !aligned(grad_x, 2)) return fail(EP_ERR_INVALID_ARG, "grad_bias / grad_x misaligned");
    cudaStream_t st = (cudaStream_t)stream;
    if (d.M == 0) {
        cudaError_t e = cudaSuccess;
        if (grad_w) e = cudaMemsetAsync(grad_w, 0, (size_t)d.wide * d.K * (w32 ? 4 : 2), st);
        if (!e && grad_bias) e = cudaMemsetAsync(grad_bias, 0, (size_t)d.wide * 4, st);
        return e ? cuda_fail(e, "ep_linear_backward") : EP_OK;
    }
    if (!grad_x && !grad_w && !grad_bias) return EP_OK;
    if (!grad_out || !aligned(grad_out, grad32 ? 4 : 2))
        return fail(EP_ERR_INVALID_ARG, "grad_out NULL or misaligned");
    if (activation != EP_ACT_NONE && (!pre || !aligned(pre, 2)))
        return fail(EP_ERR_INVALID_ARG, "pre NULL or misaligned");
    if (grad_w && (!x || !aligned(x, 16))) return fail(EP_ERR_INVALID_ARG, "x NULL or not 16-byte aligned");
    if (grad_x && (!w || !aligned(w, 16))) return fail(EP_ERR_INVALID_ARG, "w NULL or not 16-byte aligned");
    const BackwardParts b = backward_parts(d);
    if (!workspace || !aligned(workspace, 16) || workspace_bytes < b.total)
        return fail(EP_ERR_INVALID_ARG, "workspace NULL, not 16-byte aligned or too small (%zu bytes, needs %zu)",
                    workspace_bytes, b.total);
    char *ws = (char *)workspace;
    float *sums = (float *)(ws + b.g), *parts = (float *)(ws + b.g + b.sums);
    // the tensor core reads a bf16 gradient where it lies, if rows start where its copies may
    const bool direct = activation == EP_ACT_NONE && !grad32 && grad_stride % 8 == 0 &&
                        grad_stride < (int64_t)1 << 38 && aligned(grad_out, 16);
    const bool products = grad_x || grad_w;
    int order = ep::kFirst;
    bool parts_used = false;
    cudaError_t e = cudaSuccess;
    if (grad_bias || (products && !direct)) {
        ep::ActGradArgs a{};
        a.M = d.M;
        a.N = d.N;
        a.act = activation;
        a.grad32 = grad32;
        a.grad = grad_out;
        a.grad_stride = grad_stride;
        a.pre = pre;
        a.G = products && !direct ? (uint16_t *)ws : nullptr;
        a.G_stride = b.g_stride;
        a.sums = grad_bias ? sums : nullptr;
        a.blocks = b.blocks;
        a.bias = grad_bias;
        e = ep::launch_act_grad(a, st);
        if (e) return cuda_fail(e, "ep_linear_backward launch");
        // the products need G, not the columns' sums, whose own launch has waited for G
        order = grad_bias ? ep::kBeside : ep::kAfter;
    }
    const ep::LinearOperand G{direct ? (const uint16_t *)grad_out : (const uint16_t *)ws, d.M, d.wide,
                              direct ? grad_stride : b.g_stride};
    if (grad_x)
        e = backward_product(ep::kFormGradX, d.M, d.K, d.wide, b.splits_x, G, ep::LinearOperand{w, d.wide, d.K, d.K},
                             false, grad_x, grad_x_stride, parts, order, parts_used, how, dev_status, st);
    if (!e && grad_w)
        e = backward_product(ep::kFormGradW, d.wide, d.K, d.M, b.splits_w, G, ep::LinearOperand{x, d.M, d.K, x_stride},
                             w32, grad_w, d.K, parts, order, parts_used, how, dev_status, st);
    return e ? cuda_fail(e, "ep_linear_backward launch") : EP_OK;
}

}  // namespace

extern "C" {

int ep_linear(int64_t rows, int64_t in_features, int64_t out_features, int activation, const uint16_t *x,
              int64_t x_stride, const uint16_t *w, const float *bias, const uint16_t *residual,
              int64_t residual_stride, int out_dtype, void *out, int64_t out_stride, uint16_t *pre,
              int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    return linear_call({}, rows, in_features, out_features, activation, x, x_stride, w, bias, residual,
                       residual_stride, out_dtype, out, out_stride, pre, dev_status, stream);
}

size_t ep_linear_backward_workspace_bytes(int64_t rows, int64_t in_features, int64_t out_features, int activation) {
    g_err[0] = 0;
    LinearSizes d;
    return linear_sizes(rows, in_features, out_features, activation, d) ? backward_parts(d).total : 0;
}

int ep_linear_backward(int64_t rows, int64_t in_features, int64_t out_features, int activation, int grad_dtype,
                       const void *grad_out, int64_t grad_stride, const uint16_t *x, int64_t x_stride,
                       const uint16_t *w, const uint16_t *pre, uint16_t *grad_x, int64_t grad_x_stride,
                       int grad_w_dtype, void *grad_w, float *grad_bias, void *workspace, size_t workspace_bytes,
                       int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    return linear_backward_call({}, rows, in_features, out_features, activation, grad_dtype, grad_out, grad_stride, x,
                                x_stride, w, pre, grad_x, grad_x_stride, grad_w_dtype, grad_w, grad_bias, workspace,
                                workspace_bytes, dev_status, stream);
}

int ep_selftest_linear(int kernel, int64_t clocks, int64_t rows, int64_t in_features, int64_t out_features,
                       int activation, const uint16_t *x, int64_t x_stride, const uint16_t *w, const float *bias,
                       const uint16_t *residual, int64_t residual_stride, int out_dtype, void *out,
                       int64_t out_stride, uint16_t *pre, int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    if (!self_test_manner(kernel, clocks, dev_status)) return EP_ERR_INVALID_ARG;
    return linear_call({kernel, clocks}, rows, in_features, out_features, activation, x, x_stride, w, bias, residual,
                       residual_stride, out_dtype, out, out_stride, pre, dev_status, stream);
}

int ep_selftest_linear_backward(int kernel, int64_t clocks, int64_t rows, int64_t in_features, int64_t out_features,
                                int activation, int grad_dtype, const void *grad_out, int64_t grad_stride,
                                const uint16_t *x, int64_t x_stride, const uint16_t *w, const uint16_t *pre,
                                uint16_t *grad_x, int64_t grad_x_stride, int grad_w_dtype, void *grad_w,
                                float *grad_bias, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                                ep_stream_t stream) {
    g_err[0] = 0;
    if (!self_test_manner(kernel, clocks, dev_status)) return EP_ERR_INVALID_ARG;
    return linear_backward_call({kernel, clocks}, rows, in_features, out_features, activation, grad_dtype, grad_out,
                                grad_stride, x, x_stride, w, pre, grad_x, grad_x_stride, grad_w_dtype, grad_w,
                                grad_bias, workspace, workspace_bytes, dev_status, stream);
}

}  // extern "C"

namespace {

// The parts of ep_moe_few's workspace, each from a multiple of 256 bytes on
struct MoeFewParts {
    size_t x, x_scales, h, h_scales, y, arrived, parts, total;
};
bool moe_few_parts(const ep::Dims &d, int64_t I, MoeFewParts &b) {
    if (d.T > ep::kMoeFewTokens)
        return fail(EP_ERR_INVALID_ARG, "ep_moe_few takes at most %d tokens", ep::kMoeFewTokens), false;
    if (d.H % 128 || d.H > (1 << 24)) return fail(EP_ERR_INVALID_ARG, "hidden must be a multiple of 128, at most 2^24"), false;
    if (I < 128 || I % 128 || I > (1 << 23))
        return fail(EP_ERR_INVALID_ARG, "intermediate must be a multiple of 128, at most 2^23"), false;
    if (d.H * I >= (int64_t)1 << 39) return fail(EP_ERR_INVALID_ARG, "hidden * intermediate must be below 2^39"), false;
    const auto round = [](size_t n) { return (n + 255) & ~(size_t)255; };
    const size_t rows = (size_t)d.T * d.k;
    b.x = round((size_t)d.T * d.H);
    b.x_scales = round((size_t)d.T * (d.H / 128) * 4);
    b.h = round(rows * I);
    b.h_scales = round(rows * (I / 128) * 4);
    b.y = round(rows * d.H * 4);
    b.arrived = round(d.H / 128 * 4);
    b.parts = (size_t)ep::kMoeCtas * 2 * ep::moe_part_floats((int)(d.T + 15) / 16 * 16) * 4;
    b.total = b.x + b.x_scales + b.h + b.h_scales + b.y + b.arrived + b.parts + 2 * ep::kMoeCtas * 4;
    return true;
}

int moe_few_call(int64_t clocks, const ep_problem *p, const ep_router *r, int64_t intermediate, const uint16_t *x,
                 int logits_dtype, const void *logits, int64_t logits_row_stride, const float *bias,
                 const uint8_t *gate_up, const float *gate_up_scales, const uint8_t *down, const float *down_scales,
                 const uint16_t *residual, uint16_t *out, int64_t *topk_idx, float *topk_weights, void *workspace,
                 size_t workspace_bytes, int32_t *dev_status, ep_stream_t stream) {
    ep::Dims d;
    MoeFewParts b;
    if (!make_dims(p, d) || !moe_few_parts(d, intermediate, b)) return EP_ERR_INVALID_ARG;
    ep::MoeFewArgs a{};
    const int rc = prepare_route(p, r, logits_dtype, logits, logits_row_stride, dev_status, a.route);
    if (rc != EP_OK || d.T == 0) return rc;
    if (!aligned(bias, 4)) return fail(EP_ERR_INVALID_ARG, "bias misaligned");
    if (!topk_idx || !aligned(topk_idx, 8) || !topk_weights || !aligned(topk_weights, 4))
        return fail(EP_ERR_INVALID_ARG, "topk_idx / topk_weights NULL or misaligned");
    if (!x || !aligned(x, 16) || !gate_up || !aligned(gate_up, 16) || !down || !aligned(down, 16))
        return fail(EP_ERR_INVALID_ARG, "x / gate_up / down NULL or not 16-byte aligned");
    if (!gate_up_scales || !aligned(gate_up_scales, 4) || !down_scales || !aligned(down_scales, 4))
        return fail(EP_ERR_INVALID_ARG, "gate_up_scales / down_scales NULL or misaligned");
    if (!out || !aligned(out, 8) || !aligned(residual, 8))
        return fail(EP_ERR_INVALID_ARG, "out NULL, or out / residual not 8-byte aligned");
    if (!workspace || !aligned(workspace, 256) || workspace_bytes < b.total)
        return fail(EP_ERR_INVALID_ARG, "workspace NULL, not 256-byte aligned or too small (%zu bytes, needs %zu)",
                    workspace_bytes, b.total);
    char *ws = (char *)workspace;
    a.route.bias = bias;
    a.route.topk_idx = topk_idx;
    a.route.topk_weights = topk_weights;
    a.H = d.H;
    a.I = intermediate;
    a.x = x;
    a.residual = residual;
    a.gate_up = gate_up;
    a.down = down;
    a.gate_up_scales = gate_up_scales;
    a.down_scales = down_scales;
    a.xq = (uint8_t *)ws;
    a.x_scales = (float *)(ws += b.x);
    a.h = (uint8_t *)(ws += b.x_scales);
    a.h_scales = (float *)(ws += b.h);
    a.y = (float *)(ws += b.h_scales);
    a.arrived = (unsigned *)(ws += b.y);
    a.parts = (float *)(ws += b.arrived);
    a.split = (unsigned *)(ws + b.parts);
    a.out = out;
    a.wait_clocks = clocks;
    cudaError_t e = ep::launch_moe_few(a, (cudaStream_t)stream);
    return e ? cuda_fail(e, "ep_moe_few launch") : EP_OK;
}

}  // namespace

extern "C" {

size_t ep_moe_few_workspace_bytes(const ep_problem *p, int64_t intermediate) {
    g_err[0] = 0;
    ep::Dims d;
    MoeFewParts b;
    return make_dims(p, d) && moe_few_parts(d, intermediate, b) ? b.total : 0;
}

int ep_moe_few(const ep_problem *p, const ep_router *r, int64_t intermediate, const uint16_t *x, int logits_dtype,
               const void *logits, int64_t logits_row_stride, const float *bias, const uint8_t *gate_up,
               const float *gate_up_scales, const uint8_t *down, const float *down_scales, const uint16_t *residual,
               uint16_t *out, int64_t *topk_idx, float *topk_weights, void *workspace, size_t workspace_bytes,
               int32_t *dev_status, ep_stream_t stream) {
    g_err[0] = 0;
    return moe_few_call(ep::kWaitClocks, p, r, intermediate, x, logits_dtype, logits, logits_row_stride, bias,
                        gate_up, gate_up_scales, down, down_scales, residual, out, topk_idx, topk_weights, workspace,
                        workspace_bytes, dev_status, stream);
}

int ep_selftest_moe_few(int64_t clocks, const ep_problem *p, const ep_router *r, int64_t intermediate,
                        const uint16_t *x, int logits_dtype, const void *logits, int64_t logits_row_stride,
                        const float *bias, const uint8_t *gate_up, const float *gate_up_scales, const uint8_t *down,
                        const float *down_scales, const uint16_t *residual, uint16_t *out, int64_t *topk_idx,
                        float *topk_weights, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                        ep_stream_t stream) {
    g_err[0] = 0;
    if (!self_test_manner(EP_LINEAR_FEW_ROWS, clocks, dev_status)) return EP_ERR_INVALID_ARG;
    return moe_few_call(clocks, p, r, intermediate, x, logits_dtype, logits, logits_row_stride, bias, gate_up,
                        gate_up_scales, down, down_scales, residual, out, topk_idx, topk_weights, workspace,
                        workspace_bytes, dev_status, stream);
}

}  // extern "C"
