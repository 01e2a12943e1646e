"""A mixture-of-experts layer over the library: routing, FP8 dispatch, FP8
experts and combine, with the gradients that reach the router.

``MoeLayer`` keeps the device buffers of one problem and issues, on one stream,

    ep_route -> ep_layout + ep_dispatch (expert-major, FP8) -> ep_expert_swiglu
             -> ep_expert_gemm -> ep_combine

every step in the library's kernels, nothing on the host in between, so that a
forward pass can be recorded into a CUDA graph.  ``router_grad`` is the way back
from the output's gradient to the logits': ep_combine_backward, then
ep_route_backward.  (The experts are served in FP8 and take no gradient.)
"""
from __future__ import annotations

import torch

from . import ep
from .pipeline import EpPipeline


def quantize_blocks(w):
    """(codes, scales) of matrices [.., N, K] in blocks of 128 x 128: e4m3 codes (uint8) of w * 448 / amax and fp32
    scales amax / 448, the format ep_expert_gemm and ep_expert_swiglu read.  K % 128 == 0; done once, when weights
    are loaded."""
    *lead, N, K = w.shape
    if K % 128:
        raise ValueError("the channels must be a multiple of 128")
    nb = -(-N // 128)
    b = torch.zeros(*lead, nb * 128, K, dtype=torch.float32, device=w.device)
    b[..., :N, :] = w
    b = b.view(*lead, nb, 128, K // 128, 128)
    amax = b.abs().amax((-3, -1))
    inv = torch.where(amax > 0, (448.0 / amax).clamp_max(torch.finfo(torch.float32).max), 0.0)
    q = (b * inv[..., :, None, :, None]).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(*lead, nb * 128, K)[..., :N, :].contiguous(), amax / 448.0


class MoeLayer:
    def __init__(self, T: int, H: int, I: int, E: int, k: int, R: int, gate_up, gate_up_scales, down, down_scales,
                 router: ep.ep_router | None = None, bias=None, device="cuda"):
        """T tokens of R source ranks, hidden H, E experts of intermediate size I, k a token.  gate_up [E, 2 I, H]
        and down [E, H, I] are e4m3 codes (uint8) with fp32 scales for 128 x 128 blocks (see quantize_blocks);
        bias [E] fp32 moves the choice of experts (None: no bias)."""
        if tuple(gate_up.shape) != (E, 2 * I, H) or tuple(down.shape) != (E, H, I):
            raise ValueError(f"gate_up must be [{E}, {2 * I}, {H}] and down [{E}, {H}, {I}]")
        self.pipe = EpPipeline(T, H, k, E, R, layout="expert_major", dtype="fp8_e4m3", device=device)
        self.p, self.status = self.pipe.p, self.pipe.status
        self.router = ep.router() if router is None else router
        self.bias = bias
        self.gate_up, self.gate_up_scales, self.down, self.down_scales = gate_up, gate_up_scales, down, down_scales
        self.idx = torch.empty((T, k), dtype=torch.int64, device=device)
        self.weights = torch.empty((T, k), dtype=torch.float32, device=device)
        self.act = torch.empty((self.pipe.rows, I), dtype=torch.uint8, device=device)
        self.act_scales = torch.empty((self.pipe.rows, I // 128), dtype=torch.float32, device=device)
        self.grad_weights = torch.empty((T, k), dtype=torch.float32, device=device)

    def forward(self, x, logits, stream=None, out=None):
        """x [T, H] bf16 and gate logits [T, E] (bf16 or fp32) -> [T, H] bf16.  self.idx, self.weights and
        self.pipe.buf.tokens_per_expert hold the routing; ep_get_status(self.status) tells of bad logits."""
        p, q = self.p, self.pipe
        ep.ep_route(p, self.router, logits, self.bias, self.idx, self.weights, self.status, stream)
        if q.fused:
            q.layout_dispatch_step(x, self.idx, stream)
        else:
            q.layout_step(self.idx, stream)
            q.dispatch_step(x, self.idx, stream)
        counts = q.buf.tokens_per_expert
        ep.ep_expert_swiglu(p, q.recv, q.recv_scales, self.gate_up, self.gate_up_scales, counts, self.act,
                            self.act_scales, self.status, stream)
        ep.ep_expert_gemm(p, self.act, self.act_scales, self.down, self.down_scales, counts, q.y, self.status, stream)
        return q.combine_step(self.idx, self.weights, stream, out)

    def router_grad(self, grad_out, logits, grad_logits, stream=None):
        """After forward: writes the gradient of the loss with respect to the logits [T, E], through the routing
        weights (the choice of experts is a constant), from grad_out [T, H] bf16."""
        p, q = self.p, self.pipe
        ep.ep_combine_backward(p, "expert_major", grad_out, q.y, self.idx, self.weights, q.buf.rank_slot,
                               q.buf.expert_slot, None, self.grad_weights, self.status, stream)
        ep.ep_route_backward(p, self.router, logits, self.idx, self.grad_weights, grad_logits, self.status, stream)
        return grad_logits


def demo(T: int = 256, H: int = 7168, I: int = 2048, E: int = 64, k: int = 8, R: int = 8) -> None:
    """One forward and router-gradient pass over random weights, with its time (python -m
    combine_ep_layout_05_gb300.moe)."""
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)
    layer = MoeLayer(T, H, I, E, k, R, *quantize_blocks(rand(E, 2 * I, H) * H ** -0.5),
                     *quantize_blocks(rand(E, H, I) * I ** -0.5),
                     router=ep.router("sigmoid", num_groups=8, topk_groups=4, group_best=2, scale=2.5),
                     bias=torch.zeros(E, device=dev))
    x, logits, grad = rand(T, H).bfloat16(), rand(T, E), torch.empty(T, E, device=dev)
    for _ in range(3):
        out = layer.forward(x, logits)
        layer.router_grad(out, logits, grad)
    t0, t1, t2 = (torch.cuda.Event(enable_timing=True) for _ in range(3))
    t0.record()
    out = layer.forward(x, logits)
    t1.record()
    layer.router_grad(out, logits, grad)
    t2.record()
    ep_status = ep.ep_get_status(layer.status)
    print(f"{T} tokens, {E} experts of {H} x {I}, top-{k}: forward {t0.elapsed_time(t1) * 1e3:.0f} us, router gradient "
          f"{t1.elapsed_time(t2) * 1e3:.0f} us, status {ep_status}, |out| {float(out.float().abs().mean()):.4f}")


if __name__ == "__main__":
    demo()
