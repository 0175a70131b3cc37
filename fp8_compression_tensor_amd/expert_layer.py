"""A layer of experts trained on compressed operands: the products and the transposed compress in use.

Tokens, sorted by the expert a router gave them, go through one linear layer per expert.  Every
product of the training step reads E4M3 codes:

  forward    y  = x W_e^T       x compressed along k, W along k          (compress, matmul_grouped)
  backward   dx = dy W_e        dy compressed along n, W^T along n       (compress_t, matmul_grouped)
             dW = dy_e^T x_e    both compressed along the expert's rows  (compress_t, matmul_grouped_t)

and the weight gradients of the micro-batches are added up in a compressed main gradient
(accumulate: the AGoQ page, "AGoQ: Activation and Gradient Quantization for Memory-Efficient
Distributed Training of LLMs", section 2.B).  A linear head, matmul, reads the result of one token.

Usage: python -m fp8_compression_tensor_amd.expert_layer [--tokens 4096] [--steps 20] ...
trains a student layer to follow a teacher's outputs and prints the loss before and after, the
gradients' distance from the float32 ones, and the time of a step, as one JSON line.
"""
from __future__ import annotations

import argparse
import json
import sys
import time

import torch
from torch.autograd.function import once_differentiable

from . import (accumulate, compress, compress_t, decompress, matmul, matmul_grouped,
               matmul_grouped_t)

BLOCK = 128


class CompressedWeights:
    """The experts' weights [experts, n, k], compressed along k for the forward product and along n
    for the one that passes gradients back; laid out once per update."""

    def __init__(self, weight: torch.Tensor, block: int = BLOCK):
        experts, n, k = weight.shape
        if n % block or k % block:
            raise ValueError(f"{n} and {k} must be multiples of the block size {block}")
        w = weight.detach()
        codes, alpha, scale = compress(w, block)
        self.rows = (codes, alpha.view(experts, n, -1), scale.view(experts, n, -1))
        parts = [compress_t(w[e], block) for e in range(experts)]
        self.columns = tuple(torch.stack(t) for t in zip(*parts))
        self.block = block


class ExpertLinear(torch.autograd.Function):
    """y[r] = x[r] W_e(r)^T for rows sorted by expert; gradients for x and for the weights."""

    @staticmethod
    def forward(ctx, x, weight, compressed, offsets):
        block = compressed.block
        codes, alpha, scale = compress(x, block)
        ctx.save_for_backward(x, offsets)
        ctx.compressed = compressed
        ctx.wdtype = weight.dtype
        return matmul_grouped((codes, alpha, scale), compressed.rows, offsets, block, x.dtype)

    @staticmethod
    @once_differentiable  # the products record no graph: a second derivative is refused, not dropped
    def backward(ctx, dy):
        x, offsets = ctx.saved_tensors
        w, block = ctx.compressed, ctx.compressed.block
        dy = dy.contiguous()
        dx = dw = None
        if ctx.needs_input_grad[0]:
            dx = matmul_grouped(compress(dy, block), w.columns, offsets, block, x.dtype)
        if ctx.needs_input_grad[1]:
            dw = matmul_grouped_t(compress_t(dy, block, offsets=offsets),
                                  compress_t(x, block, offsets=offsets), offsets, x.shape[0],
                                  block, ctx.wdtype)
        return dx, dw, None, None


def expert_linear(x: torch.Tensor, weight: torch.Tensor, compressed: CompressedWeights,
                  offsets: torch.Tensor) -> torch.Tensor:
    """x [rows, k] with the rows of expert e at [offsets[e], offsets[e + 1]); weight [experts, n, k]
    (its gradient is the dense weight gradient), compressed = CompressedWeights(weight)."""
    return ExpertLinear.apply(x, weight, compressed, offsets)


def route(rows: int, experts: int, gen: torch.Generator) -> torch.Tensor:
    """The offsets of rows sorted by a random, uneven choice of expert."""
    share = 1.0 / torch.arange(1, experts + 1, device=gen.device, dtype=torch.float32) ** 0.3
    e = torch.multinomial(share, rows, replacement=True, generator=gen)
    counts = torch.bincount(e, minlength=experts)
    return torch.cat([counts.new_zeros(1), counts.cumsum(0)])


def plain_gradients(x, weight, dy, offsets):
    """dx and dW of the uncompressed layer, in float32."""
    off = offsets.tolist()
    dx, dw = torch.zeros_like(x, dtype=torch.float32), torch.zeros_like(weight, dtype=torch.float32)
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        dx[lo:hi] = dy[lo:hi].float() @ weight[e].float()
        dw[e] = dy[lo:hi].float().t() @ x[lo:hi].float()
    return dx, dw


def train(tokens: int, experts: int, width: int, steps: int, micro: int, rate: float,
          seed: int = 0) -> dict:
    """What the command prints; ms_per_step is the mean of the steps after the first, None where
    there is none."""
    if steps < 1 or micro < 1:
        raise ValueError(f"{steps} steps of {micro} micro-batches: at least one of each")
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *s: torch.randn(*s, device=dev, generator=gen)
    teacher = normal(experts, width, width) * width ** -0.5
    weight = torch.zeros_like(teacher).requires_grad_()
    wanted = CompressedWeights(teacher)

    def micro_batch(compressed):
        """Forward and backward of one batch: its loss, input, routing and outputs' gradient."""
        x = normal(tokens, width).to(torch.bfloat16).requires_grad_()
        offsets = route(tokens, experts, gen)
        with torch.no_grad():
            want = expert_linear(x, teacher, wanted, offsets)
        y = expert_linear(x, weight, compressed, offsets)
        diff = (y - want).float()
        loss = diff.square().mean()
        loss.backward()
        return loss.detach(), x, offsets, (2 / diff.numel() * diff.detach()).to(torch.bfloat16)

    losses = []
    begun = None
    for step in range(steps):
        if step == 1:
            torch.cuda.synchronize()
            begun = time.perf_counter()
        compressed = CompressedWeights(weight)
        main = None  # the compressed main gradient
        loss = 0.0
        for _ in range(micro):
            part = micro_batch(compressed)[0]
            grad, weight.grad = weight.grad, None
            if main is None:
                main = compress(grad, BLOCK)
            else:
                accumulate(*main, grad, BLOCK, inplace=True)
            loss = loss + part / micro
        with torch.no_grad():  # the loss is a mean over [tokens, width], of which an expert has a share
            weight -= rate * width * experts / micro * decompress(*main, BLOCK)
        losses.append(loss)
    torch.cuda.synchronize()
    ms = None if begun is None else round((time.perf_counter() - begun) / (steps - 1) * 1e3, 3)
    # the gradients of one more batch against the uncompressed layer's
    _, x, offsets, dy = micro_batch(CompressedWeights(weight))
    dx, dw = plain_gradients(x.detach(), weight.detach(), dy, offsets)
    off_dw = float((weight.grad - dw).norm() / dw.norm())
    off_dx = float((x.grad.float() - dx).norm() / dx.norm())
    token = compress(normal(1, width).to(torch.bfloat16), BLOCK)
    head = compress(weight.detach()[0], BLOCK)
    logits = matmul(token, head, BLOCK, torch.float32)
    return {"tokens": tokens, "experts": experts, "width": width, "steps": steps,
            "loss_first": float(losses[0]), "loss_last": float(losses[-1]),
            "dw_rel_l2": off_dw, "dx_rel_l2": off_dx, "ms_per_step": ms,
            "logits": list(logits.shape)}


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--micro", type=int, default=2, help="micro-batches a step")
    ap.add_argument("--rate", type=float, default=0.4)
    a = ap.parse_args(argv)
    print(json.dumps(train(a.tokens, a.experts, a.width, a.steps, a.micro, a.rate)))
    return 0


if __name__ == "__main__":
    sys.exit(main())
