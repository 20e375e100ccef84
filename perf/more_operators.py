"""The library's 8-bit and mixture-of-experts operators, as they are measured.

quantize    from x [M, K]: scale_m = max_k |x_mk| / 127; q_mk = the integer nearest to 127 x_mk / max_k |x_mk| (ties to even)
i8          out_mn = a_scale_m b_scale_n sum_k a_mk b_nk, a [M, K] and b [N, K] in 8-bit integers, out in 16 bits
moe         z = x Wr^T [M, E]; the top_k experts of a token by z (ties to the lowest), p = their softmax probabilities
            (over all experts, or over the chosen ones where `normalize` is set);
            y_m = sum_j p_mj Wd[e_mj] (act(Wg[e_mj] x_m) * (Wu[e_mj] x_m)), experts and p are returned too;
            the experts' weights in the type of x, or in 8-bit integers with a scale for each row

Matrices are row-major; x is [M, K] in binary16 or bfloat16, Wg and Wu [E, F, K], Wd [E, K, F].
"""
import math

import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # the activations of a batch of tokens before an 8-bit product: latency
        {"name": "quantize_tokens", "op": "quantize", "type": "bf16", "M": 64, "K": 4096},
        # a weight matrix quantized when a model is loaded: bandwidth
        {"name": "quantize_weights", "op": "quantize", "type": "f16", "M": 16384, "K": 8192},
        # one new token through a projection: the weights' bytes
        {"name": "i8_token", "op": "i8", "type": "bf16", "M": 1, "K": 4096, "N": 16384},
        # a batch of tokens, one per sequence being served: the weights' bytes
        {"name": "i8_batch", "op": "i8", "type": "f16", "M": 32, "K": 4096, "N": 16384},
        # the library's ragged problem: rows that no 16-byte boundary holds
        {"name": "i8_ragged", "op": "i8", "type": "f16", "M": 4000, "K": 2050, "N": 3000},
        # a whole prompt, the library's large cube
        {"name": "i8_prompt", "op": "i8", "type": "bf16", "M": 8192, "K": 8192, "N": 8192},
        # one new token through a small layer: latency
        {"name": "moe_token", "op": "moe", "type": "bf16", "M": 1, "K": 1024, "F": 512, "E": 32, "top_k": 4, "act": "silu",
         "normalize": True, "i8": False},
        # one new token through a wide layer: six experts' bytes
        {"name": "moe_token_wide", "op": "moe", "type": "f16", "M": 1, "K": 4096, "F": 2048, "E": 64, "top_k": 6, "act": "silu",
         "normalize": False, "i8": False},
        # a few tokens with every size odd or unaligned
        {"name": "moe_ragged", "op": "moe", "type": "f16", "M": 7, "K": 1030, "F": 731, "E": 12, "top_k": 3, "act": "gelu",
         "normalize": False, "i8": False},
        # a batch of sequences over many experts, few tokens for each
        {"name": "moe_batch", "op": "moe", "type": "bf16", "M": 16, "K": 4096, "F": 1536, "E": 64, "top_k": 8, "act": "silu",
         "normalize": True, "i8": False},
        # the same in 8 bits
        {"name": "moe_batch_i8", "op": "moe", "type": "bf16", "M": 32, "K": 4096, "F": 2048, "E": 32, "top_k": 4, "act": "silu",
         "normalize": True, "i8": True},
        # few experts, each with many of the tokens
        {"name": "moe_crowded", "op": "moe", "type": "f16", "M": 64, "K": 2048, "F": 4096, "E": 8, "top_k": 2, "act": "gelu",
         "normalize": True, "i8": False},
    ]


def _spread(rng, lo, hi):
    """A size, evenly spread over its logarithm; any value, an odd one, or a multiple of 8 or 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    kind = rng.random()
    if kind < 0.2:
        v |= 1
    elif kind < 0.5:
        v = (v + 7) // 8 * 8
    elif kind < 0.8 and v >= 64:
        v = (v + 63) // 64 * 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["quantize", "i8", "i8", "moe", "moe", "moe"])
    like = [work(c) for c in listed() if c["op"] == op]
    most = {k: max(w[k] for w in like) for k in ("bytes", "flops")}
    while True:
        c = {"op": op, "type": rng.choice(["f16", "bf16"])}
        if op == "quantize":
            c.update(M=_spread(rng, 1, 32768), K=_spread(rng, 16, 16384))
        elif op == "i8":
            c.update(M=_spread(rng, 1, 8192), K=_spread(rng, 64, 16384), N=_spread(rng, 64, 16384))
        else:
            c.update(M=_spread(rng, 1, 64), K=_spread(rng, 256, 4096), F=_spread(rng, 128, 4096), E=_spread(rng, 4, 128))
            c.update(top_k=rng.randint(1, min(8, c["E"])), act=rng.choice(["silu", "gelu"]),
                     normalize=rng.random() < 0.5, i8=rng.random() < 0.4)
            if c["E"] * c["F"] * c["K"] > 64 * 1536 * 4096:
                continue
        w = work(c)
        if all(w[k] <= most[k] for k in most):
            return c


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "quantize":
        return {"bytes": 3 * M * K + 4 * M, "flops": 3 * M * K}
    if case["op"] == "i8":
        N = case["N"]
        return {"bytes": (M + N) * (K + 4) + 2 * M * N, "flops": 2 * M * N * K}
    F, E, top_k = case["F"], case["E"], case["top_k"]
    # the experts that M tokens choose between them, on average
    chosen = E * (1 - (1 - top_k / E) ** M)
    expert = 3 * F * K + 4 * (2 * F + K) if case["i8"] else 6 * F * K
    return {"bytes": int(4 * M * K + 2 * E * K + 8 * M * top_k + chosen * expert),
            "flops": 2 * M * E * K + 6 * M * top_k * F * K}


def _rows8(w):
    """A matrix (or a stack of them) in 8-bit integers with a scale for each row."""
    top = w.abs().amax(dim=-1, keepdim=True)
    return torch.round(127 * w / top).to(torch.int8), (top / 127).squeeze(-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = _TYPES[case["type"]]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda").mul_(std)

    M, K = case["M"], case["K"]
    state = {"case": dict(case)}
    if case["op"] == "quantize":
        # tokens after a norm, or rows of weights; sizes differ from row to row
        state["x"] = (normal(M, K) * torch.exp(normal(M, 1))).to(dtype)
    elif case["op"] == "i8":
        state["a"], state["a_scale"] = _rows8(normal(M, K))
        state["b"], state["b_scale"] = _rows8(normal(case["N"], K, std=1 / math.sqrt(K)))
        state["dtype"] = dtype
    else:
        F, E = case["F"], case["E"]
        state["x"] = normal(M, K).to(dtype)
        state["w_router"] = normal(E, K, std=1.5 / math.sqrt(K)).to(dtype)
        for name, shape in (("w_gate", (E, F, K)), ("w_up", (E, F, K)), ("w_down", (E, K, F))):
            w = normal(*shape, std=1 / math.sqrt(shape[2]))
            if case["i8"]:
                state[name], state[name + "_scale"] = _rows8(w)
            else:
                state[name] = w.to(dtype)
    return state


def _act(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _plain_moe(state):
    case, x = state["case"], state["x"]
    M, top_k = case["M"], case["top_k"]
    # logits in 64 bits: which of two near ones is larger decides a token's experts
    z = x.double() @ state["w_router"].double().t()
    experts = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top_k]
    chosen = z.gather(1, experts)
    e = (chosen - z.amax(dim=1, keepdim=True)).exp()
    over = e if case["normalize"] else (z - z.amax(dim=1, keepdim=True)).exp()
    p = (e / over.sum(dim=1, keepdim=True)).float()

    def weight(name, which=None):
        w = state[name] if which is None else state[name][which]
        if not case["i8"]:
            return w.float()
        scale = state[name + "_scale"] if which is None else state[name + "_scale"][which]
        return w.float() * scale.unsqueeze(-1)

    xf = x.float()
    if M * top_k < case["E"]:
        # the chosen experts' weights, one copy for each choice
        which = experts.reshape(-1)
        rows = xf.repeat_interleave(top_k, dim=0).unsqueeze(2)
        h = _act(torch.bmm(weight("w_gate", which), rows), case["act"]) * torch.bmm(weight("w_up", which), rows)
        y = (torch.bmm(weight("w_down", which), h).view(M, top_k, -1) * p.unsqueeze(2)).sum(dim=1)
    else:
        # every expert for every token, weighted by p, or by 0 where it is not chosen
        share = torch.zeros(M, case["E"], device=x.device).scatter_(1, experts, p).t().unsqueeze(2)
        rows = xf.t().unsqueeze(0).expand(case["E"], -1, -1)
        h = _act(torch.bmm(weight("w_gate"), rows), case["act"]) * torch.bmm(weight("w_up"), rows)
        y = (torch.bmm(weight("w_down"), h).transpose(1, 2) * share).sum(dim=0)
    return {"y": y.to(x.dtype), "experts": experts.int(), "weights": p}


def _plain(state):
    case = state["case"]
    if case["op"] == "moe":
        return _plain_moe(state)
    if case["op"] == "i8":
        total = state["a"].float() @ state["b"].float().t()
        return {"out": (total * state["a_scale"].unsqueeze(1) * state["b_scale"]).to(state["dtype"])}
    x = state["x"].float()
    top = x.abs().amax(dim=1, keepdim=True)
    q = torch.where(top > 0, torch.round(127 * x / top), torch.zeros((), device=x.device))
    return {"q": q.to(torch.int8), "scale": (top / 127).squeeze(1)}


def _own(state):
    import pipelined_warp_specialized_gb300 as pws
    case = state["case"]
    if case["op"] == "quantize":
        q, scale = pws.gemm_i8_quantize(state["x"])
        return {"q": q, "scale": scale}
    if case["op"] == "i8":
        return {"out": pws.gemm_i8_nt(state["a"], state["b"], state["a_scale"], state["b_scale"], dtype=state["dtype"])}
    scales = (state["w_gate_scale"], state["w_up_scale"], state["w_down_scale"]) if case["i8"] else None
    y, experts, weights = pws.gemm_moe_nt(state["x"], state["w_router"], state["w_gate"], state["w_up"], state["w_down"],
                                          case["top_k"], scales=scales, act=case["act"], normalize=case["normalize"])
    return {"y": y, "experts": experts, "weights": weights}


def run(state):
    return _own(state) if own else _plain(state)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        x = s["x"].double()
        top = x.abs().max(dim=1).values
        safe = torch.where(top > 0, top, torch.ones_like(top))
        return {"q": torch.round(x * 127.0 / safe[:, None]).to(torch.int8), "scale": top / 127.0}
    if case["op"] == "i8":
        b = s["b"].double()
        rows = [torch.einsum("mk,nk->mn", a.double(), b) * u.double()[:, None] * s["b_scale"].double()[None, :]
                for a, u in zip(s["a"].split(1024), s["a_scale"].split(1024))]
        return {"out": torch.cat(rows)}
    x, top_k = s["x"].double(), case["top_k"]
    z = torch.einsum("mk,ek->me", x, s["w_router"].double())
    order = torch.argsort(-z, dim=1, stable=True)[:, :top_k]
    picked = torch.gather(z, 1, order)
    p = torch.exp(picked - torch.logsumexp(picked if case["normalize"] else z, dim=1, keepdim=True))
    inner = math.sqrt(2 / math.pi)
    y = torch.zeros_like(x)
    for e in range(case["E"]):
        token, slot = torch.nonzero(order == e, as_tuple=True)
        if token.numel() == 0:
            continue
        w = {n: s[n][e].double() for n in ("w_gate", "w_up", "w_down")}
        if case["i8"]:
            w = {n: v * s[n + "_scale"][e].double()[:, None] for n, v in w.items()}
        g, u = torch.einsum("tk,fk->tf", x[token], w["w_gate"]), torch.einsum("tk,fk->tf", x[token], w["w_up"])
        gate = g / (1 + torch.exp(-g)) if case["act"] == "silu" else g * (1 + torch.tanh(inner * g * (1 + 0.044715 * g ** 2))) / 2
        y.index_add_(0, token, torch.einsum("tf,kf->tk", gate * u, w["w_down"]) * p[token, slot][:, None])
    return {"y": y, "experts": order.int(), "weights": p}
