"""A layer of experts trained on compressed operands: the products and the transposed compress in use.

Tokens, sorted by the expert a router gave them, go through one linear layer per expert.  Every
product of the training step reads E4M3 codes:

  forward    y  = x W_e^T       x compressed along k, W along k          (compress, matmul_grouped)
  backward   dx = dy W_e        dy compressed along n, W^T along n       (compress_t, matmul_grouped)
             dW = dy_e^T x_e    both compressed along the expert's rows  (compress_t, matmul_grouped_t)

and the weight gradients of the micro-batches are added up in a compressed main gradient
(accumulate: the AGoQ page, "AGoQ: Activation and Gradient Quantization for Memory-Efficient
Distributed Training of LLMs", section 2.B).  A linear head, matmul, reads the result of one token.

GatedExperts is the whole of such a layer, W2 (silu(W1 x) * (W3 x)) behind a router: its step takes the
compressed main gradients (grad_norm, adamw), which leaves the weights' codes for the next products, and
it answers for a few tokens from those codes (moe_layer).

Usage: python -m fp8_compression_tensor_amd.expert_layer [--tokens 4096] [--steps 20] [--gated] ...
trains a student layer to follow a teacher's outputs and prints the loss before and after, the
gradients' distance from the float32 ones, and the time of a step, as one JSON line; with --gated, a
student GatedExperts, its loss, its answers' distance from its training form, and both times.
"""
from __future__ import annotations

import argparse
import json
import sys
import time

import torch
from torch.autograd.function import once_differentiable

from . import (accumulate, adamw, adamw_state, compress, compress_t, decompress, grad_norm, matmul,
               matmul_grouped, matmul_grouped_t, moe_layer)

BLOCK = 128


class CompressedWeights:
    """The experts' weights [experts, n, k], compressed along k for the forward product and along n
    for the one that passes gradients back; laid out once per update.  rows: (codes, alpha, scale) of
    the weights where they are there already, as adamw leaves them."""

    def __init__(self, weight: torch.Tensor, block: int = BLOCK, rows=None):
        experts, n, k = weight.shape
        if n % block or k % block:
            raise ValueError(f"{n} and {k} must be multiples of the block size {block}")
        w = weight.detach()
        codes, alpha, scale = compress(w, block) if rows is None else rows
        codes = codes.view(w.shape)
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


class GatedExperts:
    """A router [experts, k] and gated experts: up [experts, 2 f, k] holds W1's rows before W3's, down
    [experts, k, f]; float32, with a state of 8 or 32 bits.  Each token takes the top_k experts with the
    largest logits, weighted by their softmax."""

    def __init__(self, router, up, down, top_k: int, block: int = BLOCK, bits: int = 8, seed: int = 0):
        if not 1 <= top_k <= len(router):
            raise ValueError(f"top_k must be 1 to {len(router)}, got {top_k}")
        self.params = [p.detach().clone().requires_grad_() for p in (router, up, down)]
        self.top_k, self.block, self.seed = top_k, block, seed
        self.state = adamw_state(self.params, bits, block)
        self.steps = torch.zeros((), dtype=torch.int64, device=self.params[0].device)  # that were taken
        self.rows = [compress(p.detach(), block) for p in self.params[1:]]
        self._lay_out()

    def _lay_out(self):
        self.compressed = [CompressedWeights(p, self.block, rows)
                           for p, rows in zip(self.params[1:], self.rows)]

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        """[tokens, k] -> [tokens, k], with gradients: tokens sorted by expert, products of compressed
        operands."""
        router, up, down = self.params
        f = down.shape[-1]
        top, ids = torch.sort(x.float() @ router.t(), dim=-1, descending=True, stable=True)
        gates = torch.softmax(top[:, :self.top_k], -1)
        ids = ids[:, :self.top_k].reshape(-1)
        order = torch.argsort(ids, stable=True)
        counts = torch.bincount(ids, minlength=router.shape[0])
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
        a = expert_linear(x[order // self.top_k], up, self.compressed[0], offsets)
        h = (torch.nn.functional.silu(a[:, :f].float()) * a[:, f:].float()).to(x.dtype)
        y = expert_linear(h, down, self.compressed[1], offsets)
        back = torch.empty_like(order).scatter_(0, order, torch.arange(len(order), device=x.device))
        y = y[back].view(len(x), self.top_k, y.shape[-1]).float()
        return (y * gates[..., None]).sum(1).to(x.dtype)

    def step(self, grads, rate: float, max_norm: float = 1.0, decay: float = 0.0) -> torch.Tensor:
        """One AdamW step from the parameters' gradients, dense or compressed, clipped together; returns
        their norm.  The step writes the weights' new codes.  Where the norm is infinite or NaN it is left out,
        and does not count: the number of steps lies on the GPU, which alone knows."""
        norm, scale = grad_norm(grads, max_norm, self.block)
        steps = self.steps + torch.isfinite(scale)
        adamw([p.detach() for p in self.params], grads, self.state, rate, (0.9, 0.99),
              weight_decay=decay, step=steps, block=self.block, scale=scale,
              copies=[None, *self.rows], seed=self.seed)
        self.steps = steps
        self._lay_out()
        return norm

    def answer(self, x: torch.Tensor) -> torch.Tensor:
        """The layer for a few tokens (at most MOE_TOKENS), without gradients, from the weights' codes."""
        up, down = (c.rows for c in self.compressed)
        return moe_layer(x, self.params[0].detach(), up, down, self.top_k, self.block, dtype=x.dtype)


def train_gated(tokens: int, experts: int, width: int, hidden: int, top_k: int, steps: int, micro: int,
                rate: float, seed: int = 0) -> dict:
    """What the command prints with --gated."""
    if steps < 1 or micro < 1:
        raise ValueError(f"{steps} steps of {micro} micro-batches: at least one of each")
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)
    normal = lambda *s: torch.randn(*s, device=dev, generator=gen)
    make = lambda: GatedExperts(normal(experts, width) * width ** -0.5,
                                normal(experts, 2 * hidden, width) * width ** -0.5,
                                normal(experts, width, hidden) * hidden ** -0.5, top_k, seed=seed)
    teacher, student = make(), make()
    losses, begun = [], None
    for step in range(steps):
        if step == 1:
            torch.cuda.synchronize()
            begun = time.perf_counter()
        main, loss = None, 0.0
        for _ in range(micro):
            x = normal(tokens, width).to(torch.bfloat16)
            with torch.no_grad():
                want = teacher(x)
            part = (student(x) - want).float().square().mean()
            part.backward()
            grads = [p.grad for p in student.params]
            for p in student.params:
                p.grad = None
            if main is None:  # the router's gradient stays dense, the experts' are compressed
                main = [grads[0], *(compress(g, student.block) for g in grads[1:])]
            else:
                main[0] += grads[0]
                for m, g in zip(main[1:], grads[1:]):
                    accumulate(*m, g, student.block, inplace=True)
            loss = loss + part.detach() / micro
        student.step(main, rate)
        losses.append(loss)
    torch.cuda.synchronize()
    ms = None if begun is None else round((time.perf_counter() - begun) / (steps - 1) * 1e3, 3)
    few = normal(min(tokens, 8), width).to(torch.bfloat16)
    with torch.no_grad():
        want, got = student(few).float(), student.answer(few).float()
    student.answer(few[:1])
    torch.cuda.synchronize()
    begun = time.perf_counter()
    for _ in range(20):
        student.answer(few[:1])
    torch.cuda.synchronize()
    answer_us = (time.perf_counter() - begun) / 20 * 1e6
    return {"tokens": tokens, "experts": experts, "width": width, "hidden": hidden, "top_k": top_k,
            "steps": steps, "loss_first": float(losses[0]), "loss_last": float(losses[-1]),
            "ms_per_step": ms, "answer_rel_l2": float((got - want).norm() / want.norm()),
            "answer_us_per_token": round(answer_us, 1)}


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--micro", type=int, default=2, help="micro-batches a step")
    ap.add_argument("--rate", type=float, default=None, help="0.4; with --gated 0.002")
    ap.add_argument("--gated", action="store_true", help="gated experts behind a router, AdamW")
    ap.add_argument("--hidden", type=int, default=512, help="of a gated expert")
    ap.add_argument("--top-k", type=int, default=2, help="experts a token, with --gated")
    a = ap.parse_args(argv)
    if a.gated:
        print(json.dumps(train_gated(a.tokens, a.experts, a.width, a.hidden, a.top_k, a.steps, a.micro,
                                     0.002 if a.rate is None else a.rate)))
        return 0
    a.rate = 0.4 if a.rate is None else a.rate
    print(json.dumps(train(a.tokens, a.experts, a.width, a.steps, a.micro, a.rate)))
    return 0


if __name__ == "__main__":
    sys.exit(main())
