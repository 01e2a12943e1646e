"""A mixture-of-experts layer over the library: the gate, routing, FP8 dispatch,
FP8 experts, combine and a shared expert, with the gradients that reach the
router, the gate and the shared expert.

``MoeLayer`` keeps the device buffers of one problem and issues, on one stream,

    ep_route -> ep_layout + ep_dispatch (expert-major, FP8) -> ep_expert_swiglu
             -> ep_expert_gemm -> ep_combine

every step in the library's kernels, nothing on the host in between, so that a
forward pass can be recorded into a CUDA graph.  The gate (ep_linear: the logits
from the tokens) and a shared expert (two of ep_linear: SwiGLU, and the down
product onto the routed experts' sum) are part of it where the layer has them.
With ``few`` the routed part is one call, ep_moe_few, for up to 64 tokens.
``router_grad`` is the way back from the output's gradient to the logits':
ep_combine_backward, then ep_route_backward; ``gate_grad`` goes on to the gate
and the tokens, ``shared_grad`` through the shared expert.  (The routed experts
are served in FP8 and take no gradient.)
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
                 router: ep.ep_router | None = None, bias=None, device="cuda", gate=None, shared_gate_up=None,
                 shared_down=None, few: bool = False):
        """T tokens of R source ranks, hidden H, E experts of intermediate size I, k a token.  gate_up [E, 2 I, H]
        and down [E, H, I] are e4m3 codes (uint8) with fp32 scales for 128 x 128 blocks (see quantize_blocks);
        bias [E] fp32 moves the choice of experts (None: no bias).  gate [E, H] bf16 makes the logits from the tokens
        (None: forward is given them); shared_gate_up [2 S, H] and shared_down [H, S] bf16 are a shared expert (None:
        none).  few: the routed experts in one call that makes no receive buffers, for T <= 64; such a layer has no
        router_grad."""
        if tuple(gate_up.shape) != (E, 2 * I, H) or tuple(down.shape) != (E, H, I):
            raise ValueError(f"gate_up must be [{E}, {2 * I}, {H}] and down [{E}, {H}, {I}]")
        if gate is not None and tuple(gate.shape) != (E, H):
            raise ValueError(f"gate must be [{E}, {H}]")
        if (shared_gate_up is None) != (shared_down is None):
            raise ValueError("a shared expert has both matrices")
        if shared_down is not None and (shared_down.dim() != 2 or shared_down.shape[0] != H or
                                        tuple(shared_gate_up.shape) != (2 * shared_down.shape[1], H)):
            raise ValueError(f"shared_gate_up must be [2 S, {H}] and shared_down [{H}, S]")
        self.few = few
        buffer = lambda *s, dtype=torch.bfloat16: torch.empty(s, dtype=dtype, device=device)
        if few:
            self.p = ep.problem(T, H, k, E, R)
            bytes_ = ep.ep_moe_few_workspace_bytes(self.p, I)
            if not bytes_:
                raise ValueError(ep.ep_last_error_string())
            self.workspace, self.out = buffer(bytes_, dtype=torch.uint8), buffer(T, H)
            self.status = torch.zeros(1, dtype=torch.int32, device=device)
        else:
            self.pipe = EpPipeline(T, H, k, E, R, layout="expert_major", dtype="fp8_e4m3", device=device)
            self.p, self.status = self.pipe.p, self.pipe.status
            self.act = buffer(self.pipe.rows, I, dtype=torch.uint8)
            self.act_scales = buffer(self.pipe.rows, I // 128, dtype=torch.float32)
            self.grad_weights = buffer(T, k, dtype=torch.float32)
        self.router = ep.router() if router is None else router
        self.bias = bias
        self.gate_up, self.gate_up_scales, self.down, self.down_scales = gate_up, gate_up_scales, down, down_scales
        self.idx = buffer(T, k, dtype=torch.int64)
        self.weights = buffer(T, k, dtype=torch.float32)
        self.gate = gate
        self.logits = None if gate is None else buffer(T, E, dtype=torch.float32)
        self.shared_gate_up, self.shared_down = shared_gate_up, shared_down
        if shared_down is not None:
            S = shared_down.shape[1]
            self.shared_pre, self.shared_act = buffer(T, 2 * S), buffer(T, S)

    def forward(self, x, logits=None, stream=None, out=None):
        """x [T, H] bf16 and gate logits [T, E] (bf16 or fp32; None: the gate's, kept in self.logits) -> [T, H] bf16.
        self.idx, self.weights and (not few) self.pipe.buf.tokens_per_expert hold the routing;
        ep_get_status(self.status) tells of bad logits.  With a shared expert the output is a bf16 number added to another
        in fp32 and rounded: few: the shared expert's output, to the routed sum; else the routed sum, to the shared expert's."""
        if logits is None:
            if self.gate is None:
                raise ValueError("a layer without a gate needs logits")
            logits = self.logits
            ep.ep_linear(x, self.gate, logits, dev_status=self.status, stream=stream)
        shared = self.shared_down is not None
        if shared:
            ep.ep_linear(x, self.shared_gate_up, self.shared_act, pre=self.shared_pre, activation="swiglu",
                         dev_status=self.status, stream=stream)
        if self.few:
            out = self.out if out is None else out
            if shared:
                ep.ep_linear(self.shared_act, self.shared_down, out, dev_status=self.status, stream=stream)
            ep.ep_moe_few(self.p, self.router, x, logits, self.bias, self.gate_up, self.gate_up_scales, self.down,
                          self.down_scales, out, self.idx, self.weights, self.workspace,
                          residual=out if shared else None, dev_status=self.status, stream=stream)
            return out
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
        out = q.combine_step(self.idx, self.weights, stream, out)
        if shared:
            ep.ep_linear(self.shared_act, self.shared_down, out, residual=out, dev_status=self.status, stream=stream)
        return out

    def router_grad(self, grad_out, logits, grad_logits, stream=None):
        """After forward: writes the gradient of the loss with respect to the logits [T, E], through the routing
        weights (the choice of experts is a constant), from grad_out [T, H] bf16."""
        if self.few:
            raise ValueError("a layer with few=True keeps no expert rows: it has no router_grad")
        p, q = self.p, self.pipe
        ep.ep_combine_backward(p, "expert_major", grad_out, q.y, self.idx, self.weights, q.buf.rank_slot,
                               q.buf.expert_slot, None, self.grad_weights, self.status, stream)
        ep.ep_route_backward(p, self.router, logits, self.idx, self.grad_weights, grad_logits, self.status, stream)
        return grad_logits

    def _kept(self, name, make, stream):
        """A buffer of the gradients: made by the first call, on its stream, and kept, so that neither a later call nor a
        graph that holds its address finds it moved.  (Made on another stream it could be memory that writes of that
        stream are still on their way to.)"""
        if name not in self.__dict__:
            if stream is not None and not isinstance(stream, torch.cuda.Stream):    # a handle; 0 and 1: the default stream
                device, handle = self.status.device, int(stream)
                stream = torch.cuda.ExternalStream(handle, device) if handle > 1 else torch.cuda.default_stream(device)
            with torch.cuda.stream(stream):
                setattr(self, name, make())
        return getattr(self, name)

    def _workspace(self, name, w, activation, stream):
        rows, out = self.p.num_tokens, w.shape[0] // 2 if activation == "swiglu" else w.shape[0]
        return self._kept(name, lambda: torch.empty(
            max(16, ep.ep_linear_backward_workspace_bytes(rows, w.shape[1], out, activation)), dtype=torch.uint8,
            device=w.device), stream)

    def gate_grad(self, grad_logits, x, grad_x=None, grad_gate=None, stream=None):
        """Gradients of the logits' product, from router_grad's: grad_x [T, H] bf16 (the tokens', through the gate
        alone) and grad_gate [E, H] bf16 or fp32; None: not computed.  An fp32 grad_logits is rounded to bf16 as the
        products' operand, once, for an fp32 grad_gate too."""
        if self.gate is None:
            raise ValueError("a layer without a gate has no gate_grad")
        ep.ep_linear_backward(grad_logits, x, self.gate, grad_x=grad_x, grad_w=grad_gate,
                              workspace=self._workspace("gate_workspace", self.gate, "none", stream),
                              dev_status=self.status, stream=stream)

    def shared_grad(self, grad_out, x, grad_x=None, grad_gate_up=None, grad_down=None, stream=None):
        """After forward: gradients through the shared expert from grad_out [T, H] bf16: the tokens' (bf16) and its
        matrices' (bf16 or fp32); None: not computed."""
        if self.shared_down is None:
            raise ValueError("a layer without a shared expert has no shared_grad")
        grad_act = None
        if grad_x is not None or grad_gate_up is not None:
            grad_act = self._kept("shared_grad_act", lambda: torch.empty_like(self.shared_act), stream)
        ep.ep_linear_backward(grad_out, self.shared_act, self.shared_down, grad_x=grad_act, grad_w=grad_down,
                              workspace=self._workspace("shared_down_workspace", self.shared_down, "none", stream),
                              dev_status=self.status, stream=stream)
        if grad_act is not None:
            ep.ep_linear_backward(grad_act, x, self.shared_gate_up, grad_x=grad_x, grad_w=grad_gate_up, pre=self.shared_pre,
                                  activation="swiglu",
                                  workspace=self._workspace("shared_up_workspace", self.shared_gate_up, "swiglu", stream),
                                  dev_status=self.status, stream=stream)


def demo(T: int = 256, H: int = 7168, I: int = 2048, E: int = 64, k: int = 8, R: int = 8) -> None:
    """One forward and backward pass of a layer with a gate and a shared expert over random weights, and a decode step of
    8 tokens, with their times (python -m combine_ep_layout_05_gb300.moe)."""
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device=dev)
    experts = (*quantize_blocks(rand(E, 2 * I, H) * H ** -0.5), *quantize_blocks(rand(E, H, I) * I ** -0.5))
    kept = dict(router=ep.router("sigmoid", num_groups=8, topk_groups=4, group_best=2, scale=2.5),
                bias=torch.zeros(E, device=dev), gate=(rand(E, H) * H ** -0.5).bfloat16(),
                shared_gate_up=(rand(2 * I, H) * H ** -0.5).bfloat16(), shared_down=(rand(H, I) * I ** -0.5).bfloat16())
    layer = MoeLayer(T, H, I, E, k, R, *experts, **kept)
    x, grad = rand(T, H).bfloat16(), torch.empty(T, E, device=dev)
    grad_x, grad_gate = torch.empty_like(x), torch.empty_like(kept["gate"])
    grad_up, grad_down = torch.empty_like(kept["shared_gate_up"]), torch.empty_like(kept["shared_down"])

    def backward(out):
        layer.router_grad(out, layer.logits, grad)
        layer.gate_grad(grad, x, grad_x, grad_gate)
        layer.shared_grad(out, x, grad_x, grad_up, grad_down)
    few = MoeLayer(8, H, I, E, k, 1, *experts, **kept, few=True)
    for _ in range(3):
        out = layer.forward(x)
        backward(out)
        few.forward(x[:8])
    t = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    t[0].record()
    out = layer.forward(x)
    t[1].record()
    backward(out)
    t[2].record()
    few.forward(x[:8])
    t[3].record()
    status = ep.ep_get_status(layer.status) | ep.ep_get_status(few.status)
    us = [a.elapsed_time(b) * 1e3 for a, b in zip(t, t[1:])]
    print(f"{T} tokens, {E} experts of {H} x {I}, top-{k}, one shared: forward {us[0]:.0f} us, gradients {us[1]:.0f} us; "
          f"8 tokens {us[2]:.0f} us; status {status}, |out| {float(out.float().abs().mean()):.4f}")


if __name__ == "__main__":
    demo()
