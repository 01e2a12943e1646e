"""Cases that measure the dense products around a mixture-of-experts layer and the layer itself for a few tokens.

Operators: ``linear`` (a bf16 product with bias, activation and residual in its epilogue: the gate that makes the
router's logits, and the shared expert that every token goes through), ``linear_backward`` (the gradients of its
input, matrix and bias) and ``moe_few`` (routing, FP8 experts and weighted sum of up to 64 tokens).  With ``own``
false ``run`` computes them from elementary torch operations in 32 bits; with ``own`` true it calls the library.

x [M, K], w [N, K] (SwiGLU: [2 N, K], gate rows first), out [M, N].  The layer's experts are e4m3 codes with an fp32
scale for each 128 x 128 block, and its activations are cast to e4m3 with a scale for each 128 channels.
"""
import math

import torch

own = False

BLOCK = 128      # channels per FP8 scale
E4M3_MAX = 448.0
GELU_A, GELU_B = math.sqrt(2.0 / math.pi), 0.044715


def listed():
    return [
        # a decode step of 32 tokens through the router's gate: logits in fp32
        dict(name="gate_decode_m32", op="linear", M=32, K=7168, N=256, act="none", bias=False, residual=False,
             out="fp32", pre=False),
        # 8 ranks x 4096 tokens of prefill through the gate
        dict(name="gate_prefill_m32768", op="linear", M=32768, K=7168, N=256, act="none", bias=False, residual=False,
             out="fp32", pre=False),
        # one token through the shared expert's gate and up matrices
        dict(name="shared_up_one_token", op="linear", M=1, K=7168, N=2048, act="swiglu", bias=False, residual=False,
             out="bf16", pre=False),
        # the shared expert's gate and up products of a large batch, in training: what the backward pass needs is kept
        dict(name="shared_up_train_m8192", op="linear", M=8192, K=7168, N=2048, act="swiglu", bias=False,
             residual=False, out="bf16", pre=True),
        # ragged: 1111 tokens through a down product that adds the experts' output
        dict(name="shared_down_ragged_m1111", op="linear", M=1111, K=2048, N=7168, act="none", bias=True,
             residual=True, out="bf16", pre=False),
        # gradients of the gate for 8 x 4096 tokens, the matrix's in fp32
        dict(name="gate_bwd_m32768", op="linear_backward", M=32768, K=7168, N=256, act="none", bias=False,
             grad="bf16", grad_w="fp32"),
        # gradients of the shared expert's gate and up products
        dict(name="shared_up_bwd_m8192", op="linear_backward", M=8192, K=7168, N=2048, act="swiglu", bias=False,
             grad="bf16", grad_w="bf16"),
        # odd sizes: 515 tokens, 1000 -> 1357 channels with GELU and bias
        dict(name="gelu_bwd_ragged_m515", op="linear_backward", M=515, K=1000, N=1357, act="gelu", bias=True,
             grad="fp32", grad_w="bf16"),
        # one token through the layer: grouped sigmoid routing with a balance bias
        dict(name="moe_one_token", op="moe_few", T=1, E=256, k=8, H=7168, I=2048, dtype="fp32", scoring="sigmoid",
             bias=True, groups=8, keep=4, best=2, renorm=True, scale=2.5, padding=0, residual=True),
        # a decode step of 32 tokens
        dict(name="moe_decode_t32", op="moe_few", T=32, E=256, k=8, H=7168, I=2048, dtype="bf16", scoring="sigmoid",
             bias=True, groups=8, keep=4, best=2, renorm=True, scale=2.5, padding=0, residual=True),
        # ragged: 61 tokens, five of them padding, softmax top-6 over 64 experts
        dict(name="moe_ragged_t61", op="moe_few", T=61, E=64, k=6, H=4096, I=1408, dtype="fp32", scoring="softmax",
             bias=False, groups=1, keep=1, best=1, renorm=False, scale=1.0, padding=5, residual=False),
    ]


MOST_FLOPS, MOST_BYTES = 9.6e11, 9.4e8       # of the largest listed products
MOST_EXPERTS = 160 * 2048 * 7168             # codes of the down matrices that the largest listed layer reads


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "moe_few", "moe_few"])
    if op != "moe_few":
        act = rng.choice(["none", "none", "relu", "gelu", "silu", "swiglu"])
        K, N = 8 * _log(rng, 8, 896), _log(rng, 8, 7168)
        wide = 2 * N if act == "swiglu" else N
        times = 2 if op == "linear" else 4
        most = min(32768, MOST_FLOPS / (times * K * wide), MOST_BYTES / (times * (K + wide)))
        c = dict(op=op, M=_log(rng, 1, max(1, int(most))), K=K, N=N, act=act, bias=rng.random() < 0.5)
        if op == "linear":
            c |= dict(residual=rng.random() < 0.5, out=rng.choice(["bf16", "fp32"]), pre=rng.random() < 0.3)
        else:
            # a gradient that is rounded for the products (from fp32, or behind an activation) goes with bf16 results
            g = rng.choice(["bf16", "bf16", "fp32"])
            c |= dict(grad=g, grad_w=rng.choice(["bf16", "fp32"]) if act == "none" and g == "bf16" else "bf16")
        return c
    groups = rng.choice([1, 1, 2, 4, 8])
    E = groups * _log(rng, 2, max(2, 256 // groups))
    H = BLOCK * _log(rng, 2, 56)
    I = BLOCK * _log(rng, 1, max(1, min(16, MOST_EXPERTS // (E * H * BLOCK))))
    T = _log(rng, 1, 64)
    return dict(op=op, T=T, E=E, k=min(rng.randint(1, 10), E // groups), H=H, I=I, dtype=rng.choice(["bf16", "fp32"]),
                scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                keep=rng.randint(1, groups), best=rng.choice([1, 2]), renorm=rng.random() < 0.5,
                scale=rng.choice([1.0, 2.5]), padding=rng.choice([0, 0, T // 8]), residual=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def _keys64(x, bias, scoring):
    z = x.double()
    if scoring == "sigmoid":
        z = torch.where(z == -math.inf, z, torch.sigmoid(z))
    return z if bias is None else z + bias.double()


def _near_ties(x, bias, c):
    """Rows in which a choice hangs on less than a rounding: two different keys, or two groups' scores, nearly equal."""
    key = _keys64(x, bias, c["scoring"])

    def close(v):
        d = (v[:, :-1] - v[:, 1:]).abs()
        return ((d > 0) & (d < 1e-6)).any(1)

    near = close(key.sort(1, descending=True).values)
    if c["groups"] > 1:
        best = key.view(key.shape[0], c["groups"], -1).sort(2, descending=True).values[..., :c["best"]]
        near |= close(torch.where(best > -math.inf, best, 0.0).sum(2).sort(1, descending=True).values)
    return near


def _matrices(E, N, K, g):
    """Expert matrices N(0, 1 / K) as e4m3 codes [E, N, K] with a scale for each 128 x 128 block."""
    w = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, N // BLOCK, K // BLOCK, device="cuda")
    step = max(1, min(E, (1 << 28) // (N * K)))
    for e0 in range(0, E, step):
        n = min(step, E - e0)
        x = torch.randn(n, N // BLOCK, BLOCK, K // BLOCK, BLOCK, generator=g, device="cuda").mul_(K ** -0.5)
        amax = x.abs().amax((2, 4))
        x = x.mul_((E4M3_MAX / amax)[:, :, None, :, None]).clamp_(-E4M3_MAX, E4M3_MAX)
        w[e0:e0 + n] = x.to(torch.float8_e4m3fn).view(torch.uint8).view(n, N, K)
        s[e0:e0 + n] = amax / E4M3_MAX
    return w, s


def _type(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
    st = {"c": c, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if c["op"] == "moe_few":
        T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
        # a balance bias is moved in steps of 0.001
        bias = (rand(E) * 30).round() * 0.001 if c["bias"] else None
        empty = (torch.arange(T, device="cuda") >= T - c["padding"])[:, None]
        x = rand(T, E).to(_type(c["dtype"])).masked_fill_(empty, -math.inf)
        # Rows in which two keys are within a few roundings of each other are drawn again, so that which expert is
        # chosen is the inputs' doing and not a rounding's; equal keys stay.
        for _ in range(6):
            bad = _near_ties(x, bias, c)[:, None] & ~empty
            x = torch.where(bad, rand(T, E).to(x.dtype), x)
        st |= dict(logits=x, bias=bias, x=rand(T, H).bfloat16(), out=torch.empty(T, H, dtype=torch.bfloat16, device="cuda"),
                   idx=torch.empty(T, k, dtype=torch.int64, device="cuda"), w=torch.empty(T, k, device="cuda"),
                   residual=rand(T, H).bfloat16() if c["residual"] else None)
        st["gu"], st["gus"] = _matrices(E, 2 * I, H, g)
        st["dn"], st["dns"] = _matrices(E, H, I, g)
        return st
    M, K, N = c["M"], c["K"], c["N"]
    wide = 2 * N if c["act"] == "swiglu" else N
    st |= dict(x=rand(M, K).bfloat16(), weight=(rand(wide, K) * K ** -0.5).bfloat16(),
               bias=rand(wide) * 0.1 if c["bias"] else None)
    if c["op"] == "linear":
        st |= dict(residual=rand(M, N).bfloat16() if c["residual"] else None,
                   out=torch.empty(M, N, dtype=_type(c["out"]), device="cuda"),
                   pre=torch.empty(M, wide, dtype=torch.bfloat16, device="cuda") if c["pre"] else None)
    else:
        st |= dict(grad=rand(M, N).to(_type(c["grad"])),
                   pre=None if c["act"] == "none" else rand(M, wide).bfloat16(),
                   gx=torch.empty(M, K, dtype=torch.bfloat16, device="cuda"),
                   gw=torch.empty(wide, K, dtype=_type(c["grad_w"]), device="cuda"),
                   gb=torch.empty(wide, device="cuda") if c["bias"] else None)
    return st


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------

def _sigmoid(z):
    return 1.0 / (1.0 + torch.exp(-z))


def _act(z, act):
    if act == "swiglu":
        gate, up = z.chunk(2, 1)
        return gate * _sigmoid(gate) * up
    if act == "silu":
        return z * _sigmoid(z)
    if act == "gelu":
        return z * _sigmoid(2.0 * GELU_A * (z + GELU_B * z * z * z))
    return z.clamp_min(0.0) if act == "relu" else z


def _act_grad(g, z, act):
    """Gradient of the pre-activations z from that of the activations."""
    if act == "swiglu":
        gate, up = z.chunk(2, 1)
        s = _sigmoid(gate)
        return torch.cat([g * up * s * (1.0 + gate * (1.0 - s)), g * gate * s], 1)
    if act == "silu":
        s = _sigmoid(z)
        return g * s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        s = _sigmoid(2.0 * GELU_A * (z + GELU_B * z * z * z))
        return g * s * (1.0 + z * (1.0 - s) * 2.0 * GELU_A * (1.0 + 3.0 * GELU_B * z * z))
    return torch.where(z > 0, g, 0.0) if act == "relu" else g


def _linear(st):
    c = st["c"]
    z = st["x"].float() @ st["weight"].float().t()
    if st["bias"] is not None:
        z = z + st["bias"]
    y = _act(z, c["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    st["out"].copy_(y)
    if st["pre"] is None:
        return {"out": st["out"]}
    st["pre"].copy_(z)
    return {"out": st["out"], "pre": st["pre"]}


def _linear_backward(st):
    g = _act_grad(st["grad"].float(), None if st["pre"] is None else st["pre"].float(), st["c"]["act"])
    st["gx"].copy_(g @ st["weight"].float())
    st["gw"].copy_(g.t() @ st["x"].float())
    if st["gb"] is None:
        return {"grad_x": st["gx"], "grad_w": st["gw"]}
    st["gb"].copy_(g.sum(0))
    return {"grad_x": st["gx"], "grad_w": st["gw"], "grad_bias": st["gb"]}


def _select(c, logits, bias):
    """Expert ids of the k best keys, best first, ties to the lowest id, -1 where fewer are eligible."""
    x = logits.float()
    T, E = x.shape
    key = x if c["scoring"] == "softmax" else _sigmoid(x)
    if bias is not None:
        key = key + bias
    key = torch.where(x > -math.inf, key, -math.inf)
    if c["groups"] > 1:
        best = key.view(T, c["groups"], -1).sort(dim=2, descending=True, stable=True).values[..., :c["best"]]
        ok = best > -math.inf
        score = torch.where(ok.any(2), torch.where(ok, best, 0.0).sum(2), -math.inf)
        kept = score.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, kept, True)
        key = torch.where(keep.repeat_interleave(E // c["groups"], 1), key, -math.inf)
    v, i = key.sort(dim=1, descending=True, stable=True)
    return torch.where(v[:, :c["k"]] > -math.inf, i[:, :c["k"]], -1)


def _route(c, logits, bias):
    idx, x = _select(c, logits, bias), logits.float()
    if c["scoring"] == "sigmoid":
        s = _sigmoid(x)
    else:
        m = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
        s = e / e.sum(1, keepdim=True).clamp_min(1e-38)
    w = torch.where(idx >= 0, s.gather(1, idx.clamp_min(0)), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-38)
    return idx, w * c["scale"]


def _cast(x):
    """x rounded to e4m3 with a scale for each 128 channels: the values the codes stand for.  (Quotients of two
    tensors are rounded once; with a number on one side a reciprocal is taken, and many bf16 inputs lie on the border
    of two codes.)"""
    b = x.view(*x.shape[:-1], -1, BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    most = torch.full_like(amax, E4M3_MAX)
    inv = torch.where(amax > 0, (most / amax).clamp_max(3.4028234663852886e38), 0.0)
    q = (b * inv).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).to(x.dtype)
    return (q * (amax / most)).view(x.shape)


def _widen(q, s):
    b = q.view(torch.float8_e4m3fn).float().view(q.shape[0], s.shape[1], BLOCK, s.shape[2], BLOCK)
    return b.mul_(s[:, :, None, :, None]).view(q.shape)


def _moe_few(st):
    c = st["c"]
    T, E, k, I = c["T"], c["E"], c["k"], c["I"]
    idx, w = _route(c, st["logits"], st["bias"])
    e = idx.clamp_min(0).reshape(-1)
    a = _cast(st["x"].float())
    if T * k < E:          # the chosen experts' matrices, one for each entry
        z = torch.bmm(_widen(st["gu"][e], st["gus"][e]), a.repeat_interleave(k, 0)[..., None])[..., 0]
        h = _cast(_act(z, "swiglu"))
        y = torch.bmm(_widen(st["dn"][e], st["dns"][e]), h[..., None])[..., 0]
    else:                  # every expert's once: its entries' rows, padded to the most a token batch can have
        to = torch.zeros(T, E, dtype=torch.bool, device="cuda").scatter_(1, idx.clamp_min(0), idx >= 0)
        at = (to.cumsum(0) - 1).gather(1, idx.clamp_min(0)).clamp_min(0).reshape(-1)
        z = torch.matmul(a, _widen(st["gu"], st["gus"]).transpose(1, 2))       # [E, T, 2 I]
        t = torch.arange(T, device="cuda").repeat_interleave(k)
        h = torch.zeros(E, T, I, device="cuda")
        live = idx.reshape(-1) >= 0
        h[e[live], at[live]] = _cast(_act(z[e[live], t[live]], "swiglu"))
        y = torch.matmul(h, _widen(st["dn"], st["dns"]).transpose(1, 2))[e, at]
    out = torch.where(idx[..., None] >= 0, w[..., None] * y.view(T, k, -1), 0.0).sum(1)
    if st["residual"] is not None:
        out = out + st["residual"].float()
    st["idx"].copy_(idx)
    st["w"].copy_(w)
    st["out"].copy_(out)
    return {"out": st["out"], "idx": st["idx"], "weights": st["w"]}


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def _run_own(st):
    from combine_ep_layout_05_gb300 import ep
    c, status = st["c"], st["status"]
    if c["op"] == "linear":
        ep.ep_linear(st["x"], st["weight"], st["out"], bias=st["bias"], residual=st["residual"], pre=st["pre"],
                     activation=c["act"], dev_status=status)
        return {"out": st["out"]} if st["pre"] is None else {"out": st["out"], "pre": st["pre"]}
    if c["op"] == "linear_backward":
        if "workspace" not in st:
            st["workspace"] = torch.empty(
                max(16, ep.ep_linear_backward_workspace_bytes(c["M"], c["K"], c["N"], c["act"])), dtype=torch.uint8,
                device="cuda")
        ep.ep_linear_backward(st["grad"], st["x"], st["weight"], grad_x=st["gx"], grad_w=st["gw"], grad_bias=st["gb"],
                              pre=st["pre"], activation=c["act"], workspace=st["workspace"], dev_status=status)
        got = {"grad_x": st["gx"], "grad_w": st["gw"]}
        return got if st["gb"] is None else got | {"grad_bias": st["gb"]}
    p = ep.problem(c["T"], c["H"], c["k"], c["E"], 1)
    r = ep.router(scoring=c["scoring"], num_groups=c["groups"], topk_groups=c["keep"], group_best=c["best"],
                  renormalize=c["renorm"], scale=c["scale"])
    if "workspace" not in st:
        st["workspace"] = torch.empty(ep.ep_moe_few_workspace_bytes(p, c["I"]), dtype=torch.uint8, device="cuda")
    ep.ep_moe_few(p, r, st["x"], st["logits"], st["bias"], st["gu"], st["gus"], st["dn"], st["dns"], st["out"],
                  st["idx"], st["w"], st["workspace"], residual=st["residual"], dev_status=status)
    return {"out": st["out"], "idx": st["idx"], "weights": st["w"]}


def run(state):
    if own:
        return _run_own(state)
    return {"linear": _linear, "linear_backward": _linear_backward, "moe_few": _moe_few}[state["c"]["op"]](state)


# ---------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def _exact_route(c, logits, bias):
    key = _keys64(logits, bias, c["scoring"])
    per = key.shape[1] // c["groups"]
    if c["groups"] > 1:
        score = []
        for i in range(c["groups"]):
            v = key[:, i * per:(i + 1) * per].sort(1, descending=True).values[:, :c["best"]]
            score.append(torch.where(v[:, 0] > -math.inf, torch.where(v > -math.inf, v, 0.0).sum(1), -math.inf))
        order = torch.stack(score, 1).argsort(dim=1, descending=True, stable=True)
        for place in range(c["keep"], c["groups"]):
            for i in range(c["groups"]):
                key[:, i * per:(i + 1) * per][order[:, place] == i] = -math.inf
    order = key.argsort(dim=1, descending=True, stable=True)[:, :c["k"]]
    idx = torch.where(key.gather(1, order) > -math.inf, order, -1)
    z = logits.double()
    s = torch.sigmoid(z) if c["scoring"] == "sigmoid" else torch.nan_to_num(torch.softmax(z, 1), nan=0.0)
    w = s.gather(1, idx.clamp_min(0)) * (idx >= 0)
    if c["renorm"]:
        w = torch.where(idx >= 0, w / w.sum(1, keepdim=True), 0.0)
    return idx, w * c["scale"]


def _exact_cast(v):
    """The cast's values.  Its factor 448 / amax and the product with it are 32-bit numbers by definition, which
    decides the inputs that lie between two codes: bf16 ones often do."""
    top = v.reshape(v.shape[0], -1, BLOCK).abs().amax(2).repeat_interleave(BLOCK, 1)
    inv = (torch.full_like(top, E4M3_MAX) / torch.where(top > 0, top, 1.0)).float()
    return (v * inv.double()).float().to(torch.float8_e4m3fn).double() * top / E4M3_MAX


def exact(case, seed):
    c = dict(case)
    if c["op"] == "moe_few":
        st = prepare(c, seed)
        idx, w = _exact_route(c, st["logits"], st["bias"])
        a = _exact_cast(st["x"].double())
        out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
        scale = lambda s: s.double().repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
        for e in sorted(set(idx.reshape(-1).tolist()) - {-1}):
            share = (w * (idx == e)).sum(1)
            t = (idx == e).any(1).nonzero()[:, 0]
            z = a[t] @ (st["gu"][e].view(torch.float8_e4m3fn).double() * scale(st["gus"][e])).t()
            h = _exact_cast(z[:, :c["I"]] * torch.sigmoid(z[:, :c["I"]]) * z[:, c["I"]:])
            y = h @ (st["dn"][e].view(torch.float8_e4m3fn).double() * scale(st["dns"][e])).t()
            out[t] += share[t, None] * y
        if st["residual"] is not None:
            out += st["residual"].double()
        return {"out": out, "idx": idx, "weights": w}
    if work(c)["flops"] > 4e12:       # double-precision products run at about one TFLOP/s
        return None
    st = prepare(c, seed)
    x, w, N = st["x"].double(), st["weight"].double(), c["N"]
    bias = 0.0 if st["bias"] is None else st["bias"].double()
    u = lambda z: GELU_A * (z + GELU_B * z ** 3)
    if c["op"] == "linear":
        z = torch.mm(x, w.t()) + bias
        y = {"none": lambda: z, "relu": lambda: torch.relu(z), "silu": lambda: z * torch.sigmoid(z),
             "gelu": lambda: 0.5 * z * (1 + torch.tanh(u(z))),
             "swiglu": lambda: z[:, :N] * torch.sigmoid(z[:, :N]) * z[:, N:]}[c["act"]]()
        got = {"out": y if st["residual"] is None else y + st["residual"].double()}
        return got if st["pre"] is None else got | {"pre": z}
    g, z = st["grad"].double(), None if st["pre"] is None else st["pre"].double()
    if c["act"] == "relu":
        g = g * (z > 0)
    elif c["act"] == "silu":
        g = g * (torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z))
    elif c["act"] == "gelu":
        g = g * (0.5 * (1 + torch.tanh(u(z))) + 0.5 * z * GELU_A * (1 + 3 * GELU_B * z * z) / torch.cosh(u(z)) ** 2)
    elif c["act"] == "swiglu":
        p, q = torch.sigmoid(z[:, :N]), z[:, N:]
        g = torch.cat([g * q * (p + z[:, :N] * p * torch.sigmoid(-z[:, :N])), g * z[:, :N] * p], 1)
    got = {"grad_x": torch.mm(g, w), "grad_w": torch.mm(g.t(), x)}
    return got if st["gb"] is None else got | {"grad_bias": g.sum(0)}


# ---------------------------------------------------------------------------------------------------------------
# the least a pass has to move and compute
# ---------------------------------------------------------------------------------------------------------------

def work(case):
    c = dict(case)
    size = lambda name: 2 if name == "bf16" else 4
    if c["op"] == "moe_few":
        T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
        live = T - c["padding"]
        touched = E * (1.0 - (1.0 - k / E) ** live)      # experts with a row, expected under uniform routing
        return {"bytes": touched * 3 * I * H * (1 + 4 / BLOCK ** 2) + T * (H * (6 if c["residual"] else 4) + E * size(c["dtype"]) + k * 12),
                "flops": 6 * live * k * I * H}
    M, K, N = c["M"], c["K"], c["N"]
    wide = 2 * N if c["act"] == "swiglu" else N
    if c["op"] == "linear":
        return {"bytes": 2 * M * K + 2 * wide * K + M * N * (size(c["out"]) + (2 if c["residual"] else 0)) +
                (2 * M * wide if c["pre"] else 0) + (4 * wide if c["bias"] else 0), "flops": 2 * M * wide * K}
    return {"bytes": M * N * size(c["grad"]) + (0 if c["act"] == "none" else 2 * M * wide) + 4 * M * K + 2 * wide * K +
            wide * K * size(c["grad_w"]) + (4 * wide if c["bias"] else 0), "flops": 4 * M * wide * K}
