"""The mixture-of-experts half of a transformer block over a prompt.

One pass: residual addition and norm (bf16 rows for the router, MXFP8 rows for
the experts), router, routed experts on the tensor cores, weighted sum back
onto the residual stream. Weights and inputs are synthetic. With --shared the
block has a norm behind the attention too, a router in FP32 with sigmoid scores,
a balancing bias and groups of experts, and a shared expert whose output the
routed ones are added to.

    python examples/prompt_block.py [--tokens 4096] [--format mxfp8|mxfp4]
        [--experts 128] [--topk 8] [--hidden 2048] [--intermediate 768] [--shared]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from sparse_expert_gemv_gb300 import (DenseProduct, MoEDecode, add_rms_norm,  # noqa: E402
                                      norm_add_norm)


class PromptBlock:
    """Norm weight, router matrix and expert layer of one block."""

    def __init__(self, layer: MoEDecode, norm_weight: torch.Tensor, router: torch.Tensor,
                 eps: float = 1e-6):
        self.layer, self.norm_weight, self.router, self.eps = layer, norm_weight, router, eps

    def __call__(self, x: torch.Tensor, residual: torch.Tensor | None) -> torch.Tensor:
        """The residual stream after the block, bf16 [T, H], from the block's
        input x (the attention's output) and the stream before it."""
        n = add_rms_norm(x, self.norm_weight, residual, eps=self.eps, bf16=True, mxfp8=True)
        logits = (n.y @ self.router.T).float()
        ids, w = self.layer.route(logits)
        return self.layer.prompt(n.codes, n.scales, ids, w,
                                 residual=x if n.sum is None else n.sum)


class SharedBlock:
    """The same with a shared expert, a norm behind the block's input and grouped,
    biased routing."""

    def __init__(self, layer: MoEDecode, post_weight: torch.Tensor, norm_weight: torch.Tensor,
                 router: torch.Tensor, bias: torch.Tensor, shared_gate_up: torch.Tensor,
                 shared_down: torch.Tensor, groups: int = 8, top_groups: int = 4, scale: float = 2.5):
        self.layer, self.post_weight, self.norm_weight = layer, post_weight, norm_weight
        self.router = DenseProduct(router)
        self.gate_up = DenseProduct(shared_gate_up, activation="silu_mul")
        self.down = DenseProduct(shared_down)
        self.routing = dict(score="sigmoid", bias=bias, groups=groups, top_groups=top_groups,
                            group_score="top2", scale=scale)

    def __call__(self, x: torch.Tensor, residual: torch.Tensor) -> torch.Tensor:
        n = norm_add_norm(x, residual, self.post_weight, self.norm_weight, mxfp8=True)
        ids, w = self.layer.route(self.router(n.y, float32=True), **self.routing)
        shared = self.down(self.gate_up(n.y), n.sum)
        return self.layer.prompt(n.codes, n.scales, ids, w, residual=shared)


def random_layer(E, k, H, I, fmt, max_T, seed=0, device="cuda") -> MoEDecode:
    """A layer with random codes and scales near 2^-8 of MXFP8's range (of
    MXFP4's 2^-5): weights of about 0.02."""
    g = torch.Generator(device=device).manual_seed(seed)

    def codes(*shape):
        c = torch.randint(0, 256, shape, dtype=torch.uint8, device=device, generator=g)
        return torch.where(c % 128 >= 120, c - 16, c) if fmt == "mxfp8" else c   # no NaN codes

    def scales(*shape):
        return torch.full(shape, 115 if fmt == "mxfp8" else 120, dtype=torch.uint8, device=device)

    per = 1 if fmt == "mxfp8" else 2
    return MoEDecode(codes(E, 2 * I, H // per), scales(E, 2 * I, H // 32),
                     codes(E, H, I // per), scales(E, H, I // 32), k=k, max_T=max_T, fmt=fmt)


def main(argv=None) -> float:
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, default=4096)
    p.add_argument("--experts", type=int, default=128)
    p.add_argument("--topk", type=int, default=8)
    p.add_argument("--hidden", type=int, default=2048)
    p.add_argument("--intermediate", type=int, default=768)
    p.add_argument("--format", choices=("mxfp8", "mxfp4"), default="mxfp8")
    p.add_argument("--shared", action="store_true")
    a = p.parse_args(argv)
    T, E, H = a.tokens, a.experts, a.hidden
    g = torch.Generator(device="cuda").manual_seed(1)
    layer = random_layer(E, a.topk, H, a.intermediate, a.format, max_T=T)
    ones = torch.ones(H, dtype=torch.bfloat16, device="cuda")

    def weight(n, k):
        return torch.randn(n, k, device="cuda", generator=g).mul_(k ** -0.5).bfloat16()

    if a.shared:
        bias = 0.1 * torch.randn(E, device="cuda", generator=g)
        block = SharedBlock(layer, ones, ones, weight(E, H), bias, weight(2 * a.intermediate, H),
                            weight(H, a.intermediate), groups=4 if E % 4 == 0 else 1,
                            top_groups=2 if E % 4 == 0 else 1)
    else:
        block = PromptBlock(layer, ones, weight(E, H))
    x, residual = (torch.randn(T, H, device="cuda", generator=g).bfloat16() for _ in range(2))
    for _ in range(3):
        out = block(x, residual)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(20):
        out = block(x, residual)
    end.record()
    torch.cuda.synchronize()
    us = begin.elapsed_time(end) * 1e3 / 20
    assert out.isfinite().all() and layer.get_error() == 0
    shared = " and a shared expert" if a.shared else ""
    print(f"{T} tokens, E={E} k={a.topk} H={H} I={a.intermediate} {a.format}{shared}: {us:.1f} us a block, "
          f"{T / us:.2f} tokens a us")
    return us


if __name__ == "__main__":
    main()
