"""Helpers of the tests of the products of compressed operands and of the transposed compress: seeded
operands, the products in float64 from the definition, and the bound their results are held to."""
from __future__ import annotations

import numpy as np
import torch

DEV = "cuda:0"

E4M3 = np.array([(-1.0 if c & 128 else 1.0) * ((c & 7) * 2.0 ** -9 if not c & 0x78
                 else (8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10)) for c in range(256)])


def random_operand(rows, k, block, rng, spread=3.0, zero_blocks=0.05):
    """(codes, alpha, scale) on the host: finite random codes and scales over a few octaves, as
    compress may write them, with all-zero blocks (alpha 1, scale 0, codes 0) among them."""
    codes = rng.integers(0, 256, (rows, k), dtype=np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0
    nb = k // block
    alpha = np.exp2(rng.uniform(-spread, spread, (rows, nb))).astype(np.float32)
    scale = np.exp2(rng.uniform(-spread, spread, (rows, nb)) - 8).astype(np.float32)
    z = rng.random((rows, nb)) < zero_blocks
    alpha[z], scale[z] = 1, 0
    codes.reshape(rows, nb, block)[z] = 0
    return codes, alpha, scale


def to_gpu(op):
    return tuple(torch.from_numpy(np.ascontiguousarray(t)).to(DEV) for t in op)


def rotated_values(op, block):
    """r dec(q) of every code, in float64: the operand in the rotated basis."""
    codes, alpha, scale = op
    r = scale.astype(np.float64).reshape(-1) / alpha.astype(np.float64).reshape(-1)
    return (E4M3[codes].reshape(-1, block) * r[:, None]).reshape(codes.shape)


def exact_product(a, b):
    """(A B^T, |A| |B|^T, the root of the sum of the squared products) in float64."""
    return a @ b.T, np.abs(a) @ np.abs(b).T, np.sqrt((a * a) @ (b * b).T)


def bound(exact, mag, mag2, k, bf16):
    """How far a product may be off, from the kernels' arithmetic.

    float32 output.  Every product of two codes is exact in float32 (4 + 4 significant bits).  A
    block's sum has 128 of them a step; each addition errs by at most 2^-23 (one unit, rounded or cut
    off) of the largest partial sum, which is at most the sum of magnitudes: 128 * 2^-23.  The two
    quotients and their product round thrice (2^-24 each), and the running sum once a step: k / 128 *
    2^-24.  What lies below float32's normal range is left out by the factor's own rounding (2^-126 a
    step).

    bfloat16 output.  The 8-bit matrix instructions drop what lies more than 13 binary places below
    the largest of eight products, so each of the other seven errs by less than 2^-13 of it; taken
    as independent, that is a root mean square of at most sqrt(7) 2^-13 mag2, and six of those bound
    it.  bfloat16 has 8 significant bits, so that rounding to nearest once errs by at most 2^-8."""
    steps = max(k // 128, 1)
    e = mag * (128 * 2.0 ** -23 + (steps + 3) * 2.0 ** -24) + steps * 2.0 ** -126
    if bf16:
        e = e + 6 * 7 ** 0.5 * 2.0 ** -13 * mag2
        e = e + (np.abs(exact) + e) * 2.0 ** -8 + 2.0 ** -134
    return e


def assert_product(got, want, k, what):
    exact, mag, mag2 = want
    bf16 = got.dtype == torch.bfloat16
    g = got.detach().to(torch.float64).cpu().numpy()
    assert g.shape == exact.shape, (what, g.shape, exact.shape)
    off = np.abs(g - exact)
    e = bound(exact, mag, mag2, k, bf16)
    bad = ~(off <= e)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(),
                           float(np.nanmax(off / np.maximum(e, 1e-300))))
    return float(np.max(off / np.maximum(e, 1e-300), initial=0.0))


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)


def padded_length(rows, groups, block):
    return (rows + groups * (block - 1)) // block * block


def padded_transpose(x, offsets, block):
    """x^T with each group's columns starting at a multiple of the block, zeros between."""
    groups = len(offsets) - 1
    out = np.zeros((x.shape[1], padded_length(x.shape[0], groups, block)), x.dtype)
    at = 0
    for lo, hi in zip(offsets, offsets[1:]):
        out[:, at:at + hi - lo] = x[lo:hi].T
        at += (hi - lo + block - 1) // block * block
    return out
