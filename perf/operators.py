"""The operators around the library's products, as they are measured: a gated feed-forward block and a softmax cross
entropy over a linear head, each with its backward pass, and the backward pass of a linear layer.

gated       h = act(x Wg^T) * (x Wu^T), optionally keeping g = x Wg^T and u = x Wu^T for the backward pass
gated_bwd   from dh, g, u, x, Wg, Wu: dg = dh u act'(g), du = dh act(g);
            dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x
xent        z = x W^T; lse_i = log sum_v exp z_iv; loss_i = lse_i - z_i,target(i), 0 for ignored rows
xent_step   the same, then with dloss: D_iv = dloss_i (exp(z_iv - lse_i) - [v = target(i)]), 0 for ignored rows;
            dx = D W, dW = D^T x
linear_bwd  from dy, x, W of y = x W^T: dx = dy W, dW = dy^T x

Matrices are row-major; x is [M, K], weights are [rows, K], in binary16 or bfloat16.  Losses are float32.
"""
import math

import torch

own = False

IGNORE = -100
_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
# float64 products of more work than this take too long for exact()
_EXACT_FLOPS = 2.5e12


def listed():
    return [
        # one new token through a small model's feed-forward block: latency and the weights' bytes
        {"name": "gated_token", "op": "gated", "type": "bf16", "M": 1, "K": 1024, "F": 4096, "act": "silu", "save": False},
        # a batch of tokens, one per sequence being served: the weights' bytes
        {"name": "gated_batch", "op": "gated", "type": "f16", "M": 32, "K": 4096, "F": 16384, "act": "silu", "save": False},
        # training forward on rows that no 16-byte boundary holds (the library's ragged 4000 x 3000 x 2050 problem)
        {"name": "gated_ragged", "op": "gated", "type": "f16", "M": 4000, "K": 2050, "F": 3000, "act": "gelu", "save": True},
        # training forward, 8192 tokens
        {"name": "gated_train", "op": "gated", "type": "bf16", "M": 8192, "K": 4096, "F": 8192, "act": "silu", "save": True},
        # training backward with every size odd or unaligned
        {"name": "gated_bwd_ragged", "op": "gated_bwd", "type": "f16", "M": 1000, "K": 1030, "F": 2731, "act": "gelu"},
        # training backward, 8192 tokens
        {"name": "gated_bwd_train", "op": "gated_bwd", "type": "bf16", "M": 8192, "K": 4096, "F": 8192, "act": "silu"},
        # scoring the few tokens of an answer over an odd vocabulary: the head's bytes
        {"name": "xent_score", "op": "xent", "type": "bf16", "M": 5, "K": 2048, "V": 50001, "ignored": 0.0},
        # evaluation of a batch over a large vocabulary
        {"name": "xent_eval", "op": "xent", "type": "bf16", "M": 4096, "K": 4096, "V": 131072, "ignored": 0.05},
        # a small training step, every size odd or unaligned, a third of the rows padding
        {"name": "xent_step_ragged", "op": "xent_step", "type": "f16", "M": 777, "K": 1030, "V": 32003, "ignored": 0.33},
        # a training step's loss and gradients, 8192 tokens
        {"name": "xent_step_train", "op": "xent_step", "type": "bf16", "M": 8192, "K": 4096, "V": 65536, "ignored": 0.1},
        # the backward pass of the library's small square product
        {"name": "linear_bwd_1024", "op": "linear_bwd", "type": "f16", "M": 1024, "K": 1024, "N": 1024},
        # the backward pass of a feed-forward block's second product, 8192 tokens
        {"name": "linear_bwd_train", "op": "linear_bwd", "type": "bf16", "M": 8192, "K": 8192, "N": 4096},
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
    op = rng.choice(["gated", "gated", "gated_bwd", "xent", "xent_step", "linear_bwd"])
    most = max(work(c)["flops"] for c in listed() if c["op"] == op)
    while True:
        c = {"op": op, "type": rng.choice(["f16", "bf16"]), "M": _spread(rng, 1, 8192), "K": _spread(rng, 256, 8192)}
        if op in ("gated", "gated_bwd"):
            c.update(F=_spread(rng, 256, 16384), act=rng.choice(["silu", "gelu"]))
            if op == "gated":
                c["save"] = rng.random() < 0.5
        elif op in ("xent", "xent_step"):
            c.update(V=_spread(rng, 1000, 131072), ignored=rng.choice([0.0, 0.1, 0.5, 1.0]))
        else:
            c.update(N=_spread(rng, 256, 8192))
        if work(c)["flops"] <= most:
            return c


def work(case):
    M, K = case["M"], case["K"]
    e = 2    # bytes of an element
    if case["op"] == "gated":
        F = case["F"]
        return {"bytes": e * (M * K + 2 * F * K + M * F * (3 if case["save"] else 1)), "flops": 4 * M * F * K}
    if case["op"] == "gated_bwd":
        F = case["F"]
        return {"bytes": e * (3 * M * F + 2 * M * K + 4 * F * K), "flops": 8 * M * F * K}
    if case["op"] == "xent":
        V = case["V"]
        return {"bytes": e * (M * K + V * K) + 8 * M + 8 * M, "flops": 2 * M * V * K}
    if case["op"] == "xent_step":
        V = case["V"]
        return {"bytes": e * 2 * (M * K + V * K) + 12 * M + 8 * M, "flops": 6 * M * V * K}
    N = case["N"]
    return {"bytes": e * (M * N + 2 * M * K + 2 * N * K), "flops": 4 * M * N * K}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = _TYPES[case["type"]]

    def normal(rows, cols, std=1.0):
        return (torch.randn(rows, cols, generator=gen, device="cuda") * std).to(dtype)

    M, K = case["M"], case["K"]
    state = {"case": dict(case)}
    if case["op"] in ("gated", "gated_bwd"):
        # activations after a norm; weights of a usual initialisation
        F = case["F"]
        state["x"] = normal(M, K)
        state["w_gate"] = normal(F, K, 1 / math.sqrt(K))
        state["w_up"] = normal(F, K, 1 / math.sqrt(K))
        if case["op"] == "gated_bwd":
            # what the forward pass kept, and a (scaled) gradient from above
            state["g"] = (state["x"].float() @ state["w_gate"].float().t()).to(dtype)
            state["u"] = (state["x"].float() @ state["w_up"].float().t()).to(dtype)
            state["dh"] = normal(M, F, 0.02)
    elif case["op"] in ("xent", "xent_step"):
        # logits spread by about 2.5; every other row leans towards its target, as a trained model's does
        V = case["V"]
        state["w"] = normal(V, K, 2.5 / math.sqrt(K))
        target = torch.randint(0, V, (M,), generator=gen, device="cuda")
        lean = torch.randint(0, 2, (M, 1), generator=gen, device="cuda").float()
        x = torch.randn(M, K, generator=gen, device="cuda") + 3.0 * lean * state["w"][target].float() / 2.5
        state["x"] = x.to(dtype)
        ignored = torch.rand(M, generator=gen, device="cuda") < case["ignored"]
        state["target"] = torch.where(ignored, torch.full_like(target, IGNORE), target)
        if case["op"] == "xent_step":
            # the gradient of the mean loss over the rows that count, with the loss scale that binary16 trains with
            count = (~ignored).sum().clamp(min=1).float()
            scale = 1024.0 if case["type"] == "f16" else 1.0
            state["dloss"] = torch.where(ignored, torch.zeros((), device="cuda"), scale / count)
    else:
        N = case["N"]
        state["x"] = normal(M, K)
        state["w"] = normal(N, K, 1 / math.sqrt(K))
        state["dy"] = normal(M, N, 0.02)
    return state


def _act(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _plain(state):
    case = state["case"]
    dtype = state["x"].dtype
    x = state["x"].float()
    if case["op"] == "gated":
        g = x @ state["w_gate"].float().t()
        u = x @ state["w_up"].float().t()
        h = (_act(g, case["act"]) * u).to(dtype)
        return {"h": h, "g": g.to(dtype), "u": u.to(dtype)} if case["save"] else {"h": h}
    if case["op"] == "gated_bwd":
        g, u, dh = state["g"].float(), state["u"].float(), state["dh"].float()
        dg = dh * u * _act_grad(g, case["act"])
        du = dh * _act(g, case["act"])
        dx = dg @ state["w_gate"].float() + du @ state["w_up"].float()
        return {"dx": dx.to(dtype), "dw_gate": (dg.t() @ x).to(dtype), "dw_up": (du.t() @ x).to(dtype)}
    if case["op"] in ("xent", "xent_step"):
        w, target = state["w"].float(), state["target"]
        z = x @ w.t()
        top = z.max(dim=1, keepdim=True).values
        lse = (top + (z - top).exp().sum(dim=1, keepdim=True).log())
        counts = target != IGNORE
        at = torch.where(counts, target, torch.zeros_like(target)).unsqueeze(1)
        loss = torch.where(counts, (lse - z.gather(1, at)).squeeze(1), torch.zeros((), device=x.device))
        if case["op"] == "xent":
            return {"loss": loss, "lse": lse.squeeze(1)}
        d = (z - lse).exp()
        d.scatter_add_(1, at, torch.full_like(at, -1, dtype=d.dtype))
        d *= torch.where(counts, state["dloss"], torch.zeros((), device=x.device)).unsqueeze(1)
        return {"loss": loss, "dx": (d @ w).to(dtype), "dw": (d.t() @ x).to(dtype)}
    dy = state["dy"].float()
    return {"dx": (dy @ state["w"].float()).to(dtype), "dw": (dy.t() @ x).to(dtype)}


def _own(state):
    import pipelined_warp_specialized_gb300 as pws
    case = state["case"]
    if case["op"] == "gated":
        if case["save"]:
            h, g, u = pws.gemm_gated_nt(state["x"], state["w_gate"], state["w_up"], act=case["act"], save=True)
            return {"h": h, "g": g, "u": u}
        return {"h": pws.gemm_gated_nt(state["x"], state["w_gate"], state["w_up"], act=case["act"])}
    if case["op"] == "gated_bwd":
        dx, dw_gate, dw_up = pws.gemm_gated_nt_bwd(state["dh"], state["g"], state["u"], state["x"], state["w_gate"],
                                                   state["w_up"], act=case["act"])
        return {"dx": dx, "dw_gate": dw_gate, "dw_up": dw_up}
    if case["op"] == "xent":
        loss, lse = pws.gemm_xent_nt(state["x"], state["w"], state["target"], ignore_index=IGNORE)
        return {"loss": loss, "lse": lse}
    if case["op"] == "xent_step":
        loss, lse = pws.gemm_xent_nt(state["x"], state["w"], state["target"], ignore_index=IGNORE)
        dx, dw = pws.gemm_xent_nt_bwd(state["x"], state["w"], state["target"], lse, state["dloss"],
                                      ignore_index=IGNORE)
        return {"loss": loss, "dx": dx, "dw": dw}
    dx, dw = pws.gemm_nt_bwd(state["dy"], state["x"], state["w"])
    return {"dx": dx, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


def exact(case, seed):
    if work(case)["flops"] > _EXACT_FLOPS:
        return None
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v
         for k, v in prepare(case, seed).items()}
    if case["op"] in ("gated", "gated_bwd"):
        inner = math.sqrt(2 / math.pi)

        def act(v):         # the value and its derivative
            if case["act"] == "silu":
                e = torch.exp(-v)
                return v / (1 + e), (1 + e + v * e) / (1 + e) ** 2
            th = torch.tanh(inner * v * (1 + 0.044715 * v ** 2))
            return v * (1 + th) / 2, (1 + th) / 2 + v / 2 * (1 - th ** 2) * inner * (1 + 0.134145 * v ** 2)

        if case["op"] == "gated":
            g, u = torch.einsum("mk,fk->mf", s["x"], s["w_gate"]), torch.einsum("mk,fk->mf", s["x"], s["w_up"])
            h = act(g)[0] * u
            return {"h": h, "g": g, "u": u} if case["save"] else {"h": h}
        value, slope = act(s["g"])
        dg, du = s["dh"] * s["u"] * slope, s["dh"] * value
        return {"dx": torch.einsum("mf,fk->mk", dg, s["w_gate"]) + torch.einsum("mf,fk->mk", du, s["w_up"]),
                "dw_gate": torch.einsum("mf,mk->fk", dg, s["x"]), "dw_up": torch.einsum("mf,mk->fk", du, s["x"])}
    if case["op"] in ("xent", "xent_step"):
        x, w, target = s["x"], s["w"], s["target"]
        losses, lses, dxs = [], [], []
        dw = torch.zeros_like(w) if case["op"] == "xent_step" else None
        for a in range(0, case["M"], 512):      # rows at a time: the float64 logits of all rows are large
            z = torch.einsum("mk,vk->mv", x[a:a + 512], w)
            t = target[a:a + 512]
            lse = torch.logsumexp(z, dim=1)
            keep = t != IGNORE
            hit = torch.zeros_like(z)
            rows = torch.nonzero(keep).squeeze(1)
            hit[rows, t[rows]] = 1.0
            losses.append(torch.where(keep, lse - (z * hit).sum(dim=1), torch.zeros_like(lse)))
            lses.append(lse)
            if dw is not None:
                d = (torch.exp(z - lse[:, None]) - hit) * (s["dloss"][a:a + 512] * keep)[:, None]
                dxs.append(torch.einsum("mv,vk->mk", d, w))
                dw += torch.einsum("mv,mk->vk", d, x[a:a + 512])
        if dw is None:
            return {"loss": torch.cat(losses), "lse": torch.cat(lses)}
        return {"loss": torch.cat(losses), "dx": torch.cat(dxs), "dw": dw}
    return {"dx": torch.einsum("mn,nk->mk", s["dy"], s["w"]), "dw": torch.einsum("mn,mk->nk", s["dy"], s["x"])}
