"""A language model's last block and head, trained and served with the
library's operators:

    h      = silu(x Wg^T) * (x Wu^T)          gemm_gated_nt
    y      = x + h Wd^T                       gemm_f16_nt
    loss   = cross entropy of y W^T           gemm_xent_nt (the logits are never kept)

    backward: gemm_xent_nt_bwd -> gemm_nt_bwd -> gemm_gated_nt_bwd

Trains on one synthetic batch with plain gradient descent (binary16 weights
from float32 masters, a loss scale), prints the loss of each step and checks the
first step's gradients against autograd; then scores one token.

    python examples/language_model_block.py [--tokens 2048] [--steps 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import pipelined_warp_specialized_gb300 as pws  # noqa: E402

IGNORE = -100
LOSS_SCALE = 1024.0


def make(tokens, width, inner, vocabulary, seed=0):
    """Inputs, targets (a tenth of them padding) and float32 master weights."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(rows, cols, std):
        return torch.randn(rows, cols, generator=gen, device="cuda") * std

    x = normal(tokens, width, 1.0).half()
    target = torch.randint(0, vocabulary, (tokens,), generator=gen, device="cuda")
    target[torch.rand(tokens, generator=gen, device="cuda") < 0.1] = IGNORE
    masters = {"gate": normal(inner, width, width ** -0.5), "up": normal(inner, width, width ** -0.5),
               "down": normal(width, inner, inner ** -0.5), "head": normal(vocabulary, width, width ** -0.5)}
    return x, target, masters


def forward_backward(x, target, w):
    """Mean loss over the rows that count, and the gradients of LOSS_SCALE
    times it (x's and each weight's)."""
    h, g, u = pws.gemm_gated_nt(x, w["gate"], w["up"], save=True)
    y = x + pws.gemm_f16_nt(h, w["down"])
    loss, lse = pws.gemm_xent_nt(y, w["head"], target, ignore_index=IGNORE)
    count = (target != IGNORE).sum().clamp(min=1)

    dloss = (LOSS_SCALE / count).expand(len(target)).contiguous()
    dy, d_head = pws.gemm_xent_nt_bwd(y, w["head"], target, lse, dloss, ignore_index=IGNORE)
    dh, d_down = pws.gemm_nt_bwd(dy, h, w["down"])
    dx, d_gate, d_up = pws.gemm_gated_nt_bwd(dh, g, u, x, w["gate"], w["up"])
    return loss.sum() / count, {"x": dx + dy, "gate": d_gate, "up": d_up, "down": d_down, "head": d_head}


def autograd(x, target, w):
    """The same in float32 by torch."""
    leaves = {k: v.float().requires_grad_() for k, v in {"x": x, **w}.items()}
    h = torch.nn.functional.silu(leaves["x"] @ leaves["gate"].t()) * (leaves["x"] @ leaves["up"].t())
    y = leaves["x"] + h @ leaves["down"].t()
    loss = torch.nn.functional.cross_entropy(y @ leaves["head"].t(), target, ignore_index=IGNORE)
    (LOSS_SCALE * loss).backward()
    return loss.detach(), {k: v.grad for k, v in leaves.items()}


def train(x, target, masters, steps, rate=2.0):
    losses = []
    for _ in range(steps):
        w = {k: v.half() for k, v in masters.items()}
        loss, grads = forward_backward(x, target, w)
        for k in masters:
            masters[k] -= rate * grads[k].float() / LOSS_SCALE
        losses.append(loss)
    return [float(v) for v in losses]


def score(x, target, w):
    """Log probability of each row's target: one token, or a few."""
    y = x + pws.gemm_f16_nt(pws.gemm_gated_nt(x, w["gate"], w["up"]), w["down"])
    loss, _ = pws.gemm_xent_nt(y, w["head"], target, ignore_index=IGNORE)
    return -loss


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=2816)
    ap.add_argument("--vocabulary", type=int, default=32000)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    x, target, masters = make(a.tokens, a.width, a.inner, a.vocabulary)
    w = {k: v.half() for k, v in masters.items()}
    loss, grads = forward_backward(x, target, w)
    want, want_grads = autograd(x, target, w)
    print(f"loss {float(loss):.5f}, by autograd {float(want):.5f}")
    for k, g in want_grads.items():
        off = float((grads[k].float() - g).norm() / g.norm())
        print(f"  gradient of {k:5s} off by {off:.2e} of its norm")
    print("losses:", " ".join(f"{v:.4f}" for v in train(x, target, masters, a.steps)))
    w = {k: v.half() for k, v in masters.items()}
    print(f"log probability of one token after training: {float(score(x[:1], target[:1].clamp(min=0), w)):.4f}")
    if pws.gemm_device_status() != pws.GEMM_OK:
        raise SystemExit("a device wait timed out")


if __name__ == "__main__":
    main()
