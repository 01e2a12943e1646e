"""Cases that measure the mixture-of-experts operators around dispatch and combine.

Operators: ``route`` and ``route_backward`` (logits -> expert ids and weights, and the gradient of the logits),
``combine_backward`` (gradients of the expert rows and of the routing weights), ``expert_swiglu`` (FP8 block-scaled
product of the dispatched rows with each expert's gate and up matrices, SwiGLU, FP8 cast) and ``expert_gemm`` (the
FP8 block-scaled product with each expert's down matrix).  With ``own`` false ``run`` computes them from elementary
torch operations in 32 bits; with ``own`` true it calls the library.

T tokens of R source ranks (Tr = T / R each) go to E experts, k each; expert-major receive rows are
(e * R + src) * Tr + slot, rank-major rows (rank * R + src) * Tr + slot.
"""
import math

import torch

own = False

BLOCK = 128      # channels per FP8 scale
E4M3_MAX = 448.0


def listed():
    return [
        # a decode step of 32 tokens through grouped sigmoid routing with a balance bias
        dict(name="route_decode_t32", op="route", T=32, R=4, E=256, k=8, dtype="bf16", scoring="sigmoid", bias=True,
             groups=8, keep=4, best=2, renorm=True, scale=2.5, masked=0.0),
        # 16 ranks x 4096 tokens of prefill with the same routing, one drained rank's experts masked out
        dict(name="route_prefill_t65536", op="route", T=65536, R=16, E=256, k=8, dtype="fp32", scoring="sigmoid",
             bias=True, groups=8, keep=4, best=2, renorm=True, scale=2.5, masked=0.0625),
        # training step of 32768 tokens: softmax over all experts, weights not renormalised, so every logit has a gradient
        dict(name="route_bwd_softmax_t32768", op="route_backward", T=32768, R=8, E=256, k=8, dtype="bf16",
             scoring="softmax", bias=False, groups=1, keep=1, best=1, renorm=False, scale=1.0, masked=0.0),
        # odd sizes: 8 x 515 tokens, 160 experts, top-6, renormalised sigmoid
        dict(name="route_bwd_sigmoid_t4120", op="route_backward", T=4120, R=8, E=160, k=6, dtype="fp32",
             scoring="sigmoid", bias=True, groups=1, keep=1, best=1, renorm=True, scale=1.0, masked=0.0),
        # training step at the low-latency size: one row per (token, expert)
        dict(name="combine_bwd_expert_t1024", op="combine_backward", T=1024, R=8, E=256, k=8, H=7168,
             layout="expert_major"),
        # training step at the prefill size: one row per (token, rank)
        dict(name="combine_bwd_rank_t32768", op="combine_backward", T=32768, R=8, E=256, k=8, H=7168,
             layout="rank_major"),
        # decode: 4 ranks x 8 tokens, most experts have one or two rows
        dict(name="swiglu_decode_t32", op="expert_swiglu", T=32, R=4, E=256, k=8, H=7168, I=2048),
        # the low-latency layout: 8 ranks x 128 tokens, 32 rows an expert on average
        dict(name="swiglu_lowlat_t1024", op="expert_swiglu", T=1024, R=8, E=256, k=8, H=7168, I=2048),
        # a large batch over 32 experts: 2048 rows an expert, bound by the products
        dict(name="swiglu_batch_t8192", op="expert_swiglu", T=8192, R=8, E=32, k=8, H=7168, I=2048),
        # one token through its eight experts
        dict(name="gemm_one_token", op="expert_gemm", T=1, R=1, E=256, k=8, N=7168, K=2048),
        # ragged: 8 x 61 tokens, 128 experts, 4096 channels
        dict(name="gemm_ragged_t488", op="expert_gemm", T=488, R=8, E=128, k=8, N=4096, K=1536),
        # the large batch's down product
        dict(name="gemm_batch_t8192", op="expert_gemm", T=8192, R=8, E=32, k=8, N=7168, K=2048),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "combine_backward", "expert_swiglu", "expert_gemm", "expert_swiglu",
                     "expert_gemm"])
    R = rng.choice([1, 2, 3, 4, 5, 8, 16])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = R * groups * _log(rng, 2, max(2, 1024 // (R * groups)))
        k = min(rng.randint(1, 10), E // groups)
        return dict(op=op, T=R * _log(rng, 1, 65536 // R), R=R, E=E, k=k, dtype=rng.choice(["bf16", "fp32"]),
                    scoring=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    keep=rng.randint(1, groups), best=rng.choice([1, 2]), renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.0, 0.125]))
    if op == "combine_backward":
        layout = rng.choice(["expert_major", "rank_major"])
        E = R * _log(rng, 1, 256 // R)
        H = 8 * _log(rng, 32, 896)
        blocks = E if layout == "expert_major" else R   # blocks of T rows in the receive buffer
        T = R * _log(rng, 1, max(1, min(32768, 1_800_000_000 // (blocks * H)) // R))
        return dict(op=op, T=T, R=R, E=E, k=min(rng.randint(1, 8), E), H=H, layout=layout)
    E = R * _log(rng, 1, 256 // R)
    k = min(rng.randint(1, 8), E)
    K = BLOCK * _log(rng, 2, 56 if op == "expert_swiglu" else 16)
    I = BLOCK * _log(rng, 1, 16)
    N = 8 * _log(rng, 16, 896)
    wide = 2 * I if op == "expert_swiglu" else N
    most = min(8192, 1_500_000_000 // (E * max(K, wide)), int(3.5e12 / (2 * k * K * wide)))
    T = R * _log(rng, 1, max(1, most // R))
    if op == "expert_swiglu":
        return dict(op=op, T=T, R=R, E=E, k=k, H=K, I=I)
    return dict(op=op, T=T, R=R, E=E, k=k, N=N, K=K)


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
    T, E = key.shape
    near = torch.zeros(T, dtype=torch.bool, device=x.device)

    def close(v):
        d = (v[:, :-1] - v[:, 1:]).abs()
        return ((d > 0) & (d < 1e-6)).any(1)

    if c["groups"] > 1:
        best = key.view(T, c["groups"], -1).sort(2, descending=True).values[..., :c["best"]]
        score = torch.where(best > -math.inf, best, 0.0).sum(2)
        near |= close(score.sort(1, descending=True).values)
        # groups are not looked at one by one: every pair of neighbouring keys has to be apart
        return near | close(key.sort(1, descending=True).values[:, :min(E, c["k"] * c["groups"] + 1)])
    return near | close(key.sort(1, descending=True).values[:, :c["k"] + 1])


def _logits(c, g):
    """Gate outputs N(0, 1).  Rows in which two keys are within a few roundings of each other (about one in a
    hundred) are drawn again, so that which expert is chosen is the inputs' doing and not a rounding's; equal keys stay."""
    T, E, dev = c["T"], c["E"], "cuda"
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    # a balance bias is moved in steps of 0.001
    bias = (torch.randn(E, generator=g, device=dev) * 30).round() * 0.001 if c["bias"] else None
    off = torch.zeros(E, dtype=torch.bool, device=dev)
    off[:int(E * c["masked"])] = True      # experts of a drained rank
    empty = torch.arange(T, device=dev) >= (T if c["masked"] == 0 else T - T // 64)   # padding tokens
    mask = off[None, :] | empty[:, None]
    x = torch.randn(T, E, generator=g, device=dev).to(dt).masked_fill_(mask, -math.inf)
    for _ in range(6):
        bad = torch.cat([_near_ties(p, bias, c) for p in x.split(16384)])
        x = torch.where(bad[:, None] & ~mask, torch.randn(T, E, generator=g, device=dev).to(dt), x)
    return x, bias


def _topk_routing(c, g):
    """k distinct experts a token: the largest of E uniform logits (uniform routing), softmax weights."""
    x = torch.randn(c["T"], c["E"], generator=g, device="cuda")
    v, i = x.topk(c["k"], dim=1)
    return i, torch.softmax(v, 1)


def _slots(group, src, n):
    """Number of earlier entries of the same (group, src), in the order given."""
    key = group * n + src
    order = torch.argsort(key, stable=True)
    s = key[order]
    first = torch.searchsorted(s, s, right=False)
    slot = torch.empty_like(key)
    slot[order] = torch.arange(key.numel(), device=key.device) - first
    return slot


def _expert_layout(c, idx):
    """(expert_slot [T, k], tokens_per_expert [R, E]) of a routing."""
    T, R, E = c["T"], c["R"], c["E"]
    src = (torch.arange(T, device="cuda") // (T // R))[:, None].expand_as(idx).reshape(-1)
    e = idx.reshape(-1)
    slot = _slots(e, src, R).view_as(idx)
    count = torch.bincount(src * E + e, minlength=R * E).view(R, E)
    return slot.int(), count.int()


def _rank_layout(c, idx):
    """rank_slot [T, R]: the token's place among those of its source that go to the rank, -1 where it does not."""
    T, R, E = c["T"], c["R"], c["E"]
    to = torch.zeros(T, R, dtype=torch.bool, device="cuda")
    to.scatter_(1, idx // (E // R), True)
    before = to.view(R, T // R, R).long().cumsum(1).view(T, R) - 1
    return torch.where(to, before, -1).int()


def _cast_rows(x):
    """e4m3 codes and scales of 1 x 128 blocks."""
    b = x.view(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(2)
    q = (b * (E4M3_MAX / amax.clamp_min(1e-30))[..., None]).clamp_(-E4M3_MAX, E4M3_MAX)
    return q.to(torch.float8_e4m3fn).view(torch.uint8).view(x.shape), amax / E4M3_MAX


def _weights(E, N, K, g):
    """Expert matrices N(0, 1 / K) as e4m3 codes [E, N, K] with a scale for each 128 x 128 block."""
    nb, kb = -(-N // BLOCK), K // BLOCK
    w = torch.empty(E, N, K, dtype=torch.uint8, device="cuda")
    s = torch.empty(E, nb, kb, device="cuda")
    step = max(1, min(E, (1 << 28) // (nb * BLOCK * K)))
    for e0 in range(0, E, step):
        n = min(step, E - e0)
        x = torch.randn(n, nb, BLOCK, kb, BLOCK, generator=g, device="cuda").mul_(K ** -0.5)
        amax = x.abs().amax((2, 4))
        x = x.mul_((E4M3_MAX / amax)[:, :, None, :, None]).clamp_(-E4M3_MAX, E4M3_MAX)
        w[e0:e0 + n] = x.to(torch.float8_e4m3fn).view(torch.uint8).view(n, nb * BLOCK, K)[:, :N]
        s[e0:e0 + n] = amax / E4M3_MAX
    return w, s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, T, R, E, k = c["op"], c["T"], c["R"], c["E"], c["k"]
    st = {"c": c, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if op in ("route", "route_backward"):
        st["logits"], st["bias"] = _logits(c, g)
        st["idx"] = torch.empty(T, k, dtype=torch.int64, device="cuda")
        st["w"] = torch.empty(T, k, device="cuda")
        if op == "route_backward":
            st["idx"] = _select(c, st["logits"], st["bias"])
            st["gw"] = torch.randn(T, k, generator=g, device="cuda")
            st["gx"] = torch.empty_like(st["logits"])
        return st
    st["idx"], st["w"] = _topk_routing(c, g)
    if op == "combine_backward":
        major = c["layout"] == "expert_major"
        rows = (E if major else R) * T
        st["eslot"], _ = _expert_layout(c, st["idx"])
        st["rslot"] = _rank_layout(c, st["idx"])
        st["y"] = torch.empty(rows, c["H"], dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        st["dout"] = torch.randn(T, c["H"], generator=g, device="cuda").bfloat16()
        st["gy"] = torch.zeros_like(st["y"])
        st["gw"] = torch.zeros(T, k, device="cuda")
        return st
    N, K = (2 * c["I"], c["H"]) if op == "expert_swiglu" else (c["N"], c["K"])
    slot, st["count"] = _expert_layout(c, st["idx"])
    src = (torch.arange(T, device="cuda") // (T // R))[:, None]
    row = ((st["idx"] * R + src) * (T // R) + slot).view(-1)
    q, s = _cast_rows(torch.randn(T, K, generator=g, device="cuda"))
    st["a"] = torch.zeros(E * T, K, dtype=torch.uint8, device="cuda")
    st["as"] = torch.zeros(E * T, K // BLOCK, device="cuda")
    st["a"][row] = q.repeat_interleave(k, 0)
    st["as"][row] = s.repeat_interleave(k, 0)
    st["W"], st["Ws"] = _weights(E, N, K, g)
    if op == "expert_swiglu":
        st["q"] = torch.zeros(E * T, c["I"], dtype=torch.uint8, device="cuda")
        st["qs"] = torch.zeros(E * T, c["I"] // BLOCK, device="cuda")
    else:
        st["y"] = torch.zeros(E * T, N, dtype=torch.bfloat16, device="cuda")
    return st


# ---------------------------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------------------------

def _select(c, logits, bias):
    """Expert ids of the k best keys, best first, ties to the lowest id, -1 where fewer are eligible."""
    x = logits.float()
    T, E = x.shape
    fit = x > -math.inf
    key = x if c["scoring"] == "softmax" else 1.0 / (1.0 + torch.exp(-x))
    if bias is not None:
        key = key + bias
    key = torch.where(fit, key, -math.inf)
    if c["groups"] > 1:
        best = key.view(T, c["groups"], -1).sort(dim=2, descending=True, stable=True).values[..., :c["best"]]
        ok = best > -math.inf
        score = torch.where(ok, best, 0.0).sum(2)
        score = torch.where(ok.any(2), score, -math.inf)
        kept = score.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, kept, True)
        key = torch.where(keep.repeat_interleave(E // c["groups"], 1), key, -math.inf)
    v, i = key.sort(dim=1, descending=True, stable=True)
    return torch.where(v[:, :c["k"]] > -math.inf, i[:, :c["k"]], -1)


def _scores(c, x):
    if c["scoring"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    return e / e.sum(1, keepdim=True).clamp_min(1e-38)


def _route(st):
    c, x = st["c"], st["logits"].float()
    idx = _select(c, st["logits"], st["bias"])
    w = torch.where(idx >= 0, _scores(c, x).gather(1, idx.clamp_min(0)), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-38)
    st["idx"].copy_(idx)
    st["w"].copy_(w * c["scale"])
    return {"idx": st["idx"], "weights": st["w"]}


def _route_backward(st):
    c, x = st["c"], st["logits"].float()
    idx, live = st["idx"].clamp_min(0), st["idx"] >= 0
    g = torch.where(live, st["gw"], 0.0) * c["scale"]
    s = _scores(c, x)
    sj = torch.where(live, s.gather(1, idx), 0.0)
    if c["renorm"]:
        total = sj.sum(1, keepdim=True).clamp_min(1e-38)
        ds = (g - (g * sj).sum(1, keepdim=True) / total) / total
    else:
        ds = g
    ds = torch.zeros_like(x).scatter_add_(1, idx, torch.where(live, ds, 0.0))
    if c["scoring"] == "sigmoid":
        dx = ds * s * (1.0 - s)
    else:
        dx = s * (ds - (ds * s).sum(1, keepdim=True))
    st["gx"].copy_(dx)
    return {"grad_logits": st["gx"]}


def _combine_backward(st):
    c = st["c"]
    T, R, E, H = c["T"], c["R"], c["E"], c["H"]
    src = (torch.arange(T, device="cuda") // (T // R))[:, None]
    if c["layout"] == "expert_major":
        row, w = (st["idx"] * R + src) * (T // R) + st["eslot"], st["w"]
        live = torch.ones_like(row, dtype=torch.bool)
        col = torch.arange(c["k"], device="cuda").expand_as(row)
    else:
        live = st["rslot"] >= 0
        row = (torch.arange(R, device="cuda") * R + src) * (T // R) + st["rslot"]
        col = st["idx"] // (E // R)
        w = torch.zeros(T, R, device="cuda").scatter_add_(1, col, st["w"])
    t, _ = live.nonzero(as_tuple=True)
    at = row[live]
    dout = st["dout"].float()[t]
    st["gy"][at] = (dout * w[live][:, None]).bfloat16()
    dot = torch.zeros(row.shape, device="cuda")
    dot[live] = (dout * st["y"][at].float()).sum(1)
    st["gw"].copy_(dot.gather(1, col))
    return {"grad_y": st["gy"], "grad_weights": st["gw"]}


def _product(st, N, K):
    """(fp32 product [live rows, N], their rows): the rows of each expert, padded to the most, times its matrix."""
    c = st["c"]
    E, T, R = c["E"], c["T"], c["R"]
    live = torch.arange(T // R, device="cuda") < st["count"].t()[..., None]
    row = live.reshape(-1).nonzero()[:, 0]
    m = st["count"].sum(0)
    place = torch.arange(int(m.max()), device="cuda")
    has = place < m[:, None]
    at = row[((m.cumsum(0) - m)[:, None] + place).clamp_max(row.numel() - 1)]
    a = st["a"][at].view(torch.float8_e4m3fn).float().view(E, -1, K // BLOCK, BLOCK)
    a = (a * st["as"][at][..., None]).view(E, -1, K)
    w = st["W"].view(torch.float8_e4m3fn).float().view(E, N, K // BLOCK, BLOCK)
    w = w.mul_(st["Ws"].repeat_interleave(BLOCK, 1)[:, :N, :, None]).view(E, N, K)
    return torch.bmm(a, w.transpose(1, 2))[has], row


def _expert_swiglu(st):
    I = st["c"]["I"]
    y, row = _product(st, 2 * I, st["c"]["H"])
    gate, up = y[:, :I], y[:, I:]
    h = (gate / (1.0 + torch.exp(-gate)) * up).view(-1, I // BLOCK, BLOCK)
    amax = h.abs().amax(2)
    inv = torch.where(amax > 0, (E4M3_MAX / amax).clamp_max(3.4028234663852886e38), 0.0)
    q = (h * inv[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    st["q"][row] = q.view(torch.uint8).view(-1, I)
    st["qs"][row] = amax / E4M3_MAX
    return {"q": st["q"].view(torch.float8_e4m3fn), "scales": st["qs"]}


def _expert_gemm(st):
    y, row = _product(st, st["c"]["N"], st["c"]["K"])
    st["y"][row] = y.bfloat16()
    return {"y": st["y"]}


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def _run_own(st):
    from combine_ep_layout_05_gb300 import ep
    c, status = st["c"], st["status"]
    op = c["op"]
    H = c["H"] if "H" in c else c["N"] if "N" in c else 128
    p = ep.problem(c["T"], H, c["k"], c["E"], c["R"])
    if op in ("route", "route_backward"):
        r = ep.router(scoring=c["scoring"], num_groups=c["groups"], topk_groups=c["keep"], group_best=c["best"],
                      renormalize=c["renorm"], scale=c["scale"])
        if op == "route":
            ep.ep_route(p, r, st["logits"], st["bias"], st["idx"], st["w"], status)
            return {"idx": st["idx"], "weights": st["w"]}
        ep.ep_route_backward(p, r, st["logits"], st["idx"], st["gw"], st["gx"], status)
        return {"grad_logits": st["gx"]}
    if op == "combine_backward":
        ep.ep_combine_backward(p, c["layout"], st["dout"], st["y"], st["idx"], st["w"], st["rslot"], st["eslot"],
                               st["gy"], st["gw"], status)
        return {"grad_y": st["gy"], "grad_weights": st["gw"]}
    if op == "expert_swiglu":
        ep.ep_expert_swiglu(p, st["a"], st["as"], st["W"], st["Ws"], st["count"], st["q"], st["qs"], status)
        return {"q": st["q"].view(torch.float8_e4m3fn), "scales": st["qs"]}
    ep.ep_expert_gemm(p, st["a"], st["as"], st["W"], st["Ws"], st["count"], st["y"], status)
    return {"y": st["y"]}


def run(state):
    if own:
        return _run_own(state)
    return {"route": _route, "route_backward": _route_backward, "combine_backward": _combine_backward,
            "expert_swiglu": _expert_swiglu, "expert_gemm": _expert_gemm}[state["c"]["op"]](state)


# ---------------------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------

def _exact_route(c, x, bias):
    key = _keys64(x, bias, c["scoring"])
    per = key.shape[1] // c["groups"]
    if c["groups"] > 1:
        score = []
        for i in range(c["groups"]):
            v = key[:, i * per:(i + 1) * per].sort(1, descending=True).values[:, :c["best"]]
            score.append(torch.where(v[:, 0] > -math.inf, torch.where(v > -math.inf, v, 0.0).sum(1), -math.inf))
        score = torch.stack(score, 1)
        order = score.argsort(dim=1, descending=True, stable=True)
        for place in range(c["keep"], c["groups"]):
            drop = order[:, place]
            for i in range(c["groups"]):
                key[:, i * per:(i + 1) * per][drop == i] = -math.inf
    order = key.argsort(dim=1, descending=True, stable=True)[:, :c["k"]]
    return torch.where(key.gather(1, order) > -math.inf, order, -1)


def _exact_scores(c, x):
    z = x.double()
    if c["scoring"] == "sigmoid":
        return torch.sigmoid(z)
    return torch.nan_to_num(torch.softmax(z, 1), nan=0.0)


def exact(case, seed):
    c = dict(case)
    op, T, R, E, k = c["op"], c["T"], c["R"], c["E"], c["k"]
    if op.startswith("expert"):
        N, K = (2 * c["I"], c["H"]) if op == "expert_swiglu" else (c["N"], c["K"])
        if 2.0 * T * k * N * K > 4e12:      # double-precision products run at about one TFLOP/s
            return None
    st = prepare(c, seed)
    if op == "route":
        x = st["logits"]
        idx = _exact_route(c, x, st["bias"])
        w = _exact_scores(c, x).gather(1, idx.clamp_min(0)) * (idx >= 0)
        if c["renorm"]:
            w = torch.where(idx >= 0, w / w.sum(1, keepdim=True), 0.0)
        return {"idx": idx, "weights": w * c["scale"]}
    if op == "route_backward":
        s, live, idx = _exact_scores(c, st["logits"]), st["idx"] >= 0, st["idx"].clamp_min(0)
        sel = torch.zeros_like(s).scatter_add_(1, idx, live.double())
        gd = torch.zeros_like(s).scatter_add_(1, idx, st["gw"].double() * live) * c["scale"]
        if c["renorm"]:
            tot = (s * sel).sum(1, keepdim=True)
            tot = torch.where(tot > 0, tot, 1.0)
            gd = sel * (gd / tot - (gd * s).sum(1, keepdim=True) / tot ** 2)
        dx = gd * s * (1 - s) if c["scoring"] == "sigmoid" else s * gd - s * (s * gd).sum(1, keepdim=True)
        return {"grad_logits": dx}
    if op == "combine_backward":
        gy, gw = torch.zeros_like(st["y"], dtype=torch.float64 if st["y"].numel() < 2e9 else torch.float32), []
        for t0 in range(0, T, 2048):
            t = torch.arange(t0, min(T, t0 + 2048), device="cuda")
            idx, d, w = st["idx"][t], st["dout"][t].double(), st["w"][t].double()
            dst = idx // (E // R)
            if c["layout"] == "expert_major":
                at = (idx * R + (t // (T // R))[:, None]) * (T // R) + st["eslot"][t]
                share = w
            else:
                at = (dst * R + (t // (T // R))[:, None]) * (T // R) + st["rslot"][t].gather(1, dst)
                share = ((dst[:, :, None] == dst[:, None, :]) * w[:, None, :]).sum(2)
            dots = []
            for j in range(k):
                dots.append((st["y"][at[:, j]].double() * d).sum(1))
                gy[at[:, j]] = (share[:, j:j + 1] * d).to(gy.dtype)
            gw.append(torch.stack(dots, 1))
        return {"grad_y": gy, "grad_weights": torch.cat(gw)}
    out = torch.zeros(E * T, N // 2 if op == "expert_swiglu" else N, dtype=torch.float64, device="cuda")
    sc = torch.zeros(E * T, out.shape[1] // BLOCK if op == "expert_swiglu" else 1, dtype=torch.float64, device="cuda")
    count = st["count"].tolist()
    for e in range(E):
        at = [(e * R + s) * (T // R) + i for s in range(R) for i in range(count[s][e])]
        if not at:
            continue
        at = torch.tensor(at, device="cuda")
        a = st["a"][at].view(torch.float8_e4m3fn).double() * st["as"][at].double().repeat_interleave(BLOCK, 1)
        w = st["W"][e].view(torch.float8_e4m3fn).double()
        w *= st["Ws"][e].double().repeat_interleave(BLOCK, 1).repeat_interleave(BLOCK, 0)[:N]
        y = a @ w.t()
        if op == "expert_swiglu":
            h = y[:, :N // 2] * torch.sigmoid(y[:, :N // 2]) * y[:, N // 2:]
            top = h.view(len(at), -1, BLOCK).abs().amax(2)
            sc[at] = top / E4M3_MAX
            # the codes stand for h over the block's scale
            y = h / torch.where(top > 0, top / E4M3_MAX, 1.0).repeat_interleave(BLOCK, 1)
        out[at] = y
    return {"q": out, "scales": sc} if op == "expert_swiglu" else {"y": out}


# ---------------------------------------------------------------------------------------------------------------
# the least a pass has to move and compute
# ---------------------------------------------------------------------------------------------------------------

def _touched(c):
    """Experts with at least one row, expected under uniform routing."""
    return c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])


def work(case):
    c = dict(case)
    op, T, R, E, k = c["op"], c["T"], c["R"], c["E"], c["k"]
    if op in ("route", "route_backward"):
        b = 2 if c["dtype"] == "bf16" else 4
        if op == "route":
            return {"bytes": T * E * b + T * k * 12 + (E * 4 if c["bias"] else 0), "flops": 8 * T * E}
        dense = c["scoring"] == "softmax" and not c["renorm"]
        return {"bytes": T * (E if dense else k) * b + T * E * b + T * k * 12, "flops": 8 * T * (E if dense else k)}
    if op == "combine_backward":
        H = c["H"]
        if c["layout"] == "expert_major":
            rows, slots = T * k, k
        else:
            miss = math.prod((E - E // R - i) / (E - i) for i in range(k)) if E - E // R >= k else 0.0
            rows, slots = T * R * (1.0 - miss), R
        return {"bytes": rows * H * 4 + T * H * 2 + T * (k * 16 + slots * 4), "flops": 3 * rows * H}
    N, K = (2 * c["I"], c["H"]) if op == "expert_swiglu" else (c["N"], c["K"])
    out = c["I"] * (1 + 4 / BLOCK) if op == "expert_swiglu" else 2 * N
    scales = -(-N // BLOCK) * (K // BLOCK) * 4
    return {"bytes": _touched(c) * (N * K + scales) + T * k * (K * (1 + 4 / BLOCK) + out) + R * E * 4,
            "flops": 2 * T * k * N * K}
