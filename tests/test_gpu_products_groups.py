"""Grouped products and the transposed compress where the offsets do not start at the first row, end at
the last one, or ascend."""
import numpy as np
import pytest
import torch

import fp8_compression_tensor_amd as tfp8
from gpu_helpers import say
from product_helpers import (DEV, assert_product, exact_product, padded_length, random_operand,
                             rotated_values, to_gpu)

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def gpu(off):
    return torch.tensor([int(o) for o in off], dtype=torch.int64, device=DEV)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("off,rows", [([3, 3, 20], 33), ([40, 60, 60, 200], 200),
                                      ([300, 431, 800], 900), ([70] * 5, 70), ([70] * 5, 100),
                                      (list(range(9, 80)), 90)])
@pytest.mark.parametrize("n,k,block", [(40, 256, 128), (1000, 512, 256)])
def test_rows_of_no_group_become_zeros(off, rows, n, k, block, dt):
    """The offsets of some of the experts, taken with their weights out of a longer vector."""
    say(f"matmul_grouped offsets {off[:4]} of {rows} rows, n {n} k {k} block {block} {dt}")
    groups = len(off) - 1
    rng = np.random.default_rng(rows + n)
    a, w = random_operand(rows, k, block, rng), random_operand(groups * n, k, block, rng)
    av, wv = rotated_values(a, block), rotated_values(w, block).reshape(groups, n, k)
    wg = tuple(t.view(groups, n, -1) for t in to_gpu(w))
    out = torch.full((rows, n), float("nan"), dtype=DTYPES[dt], device=DEV)
    tfp8.matmul_grouped(to_gpu(a), wg, gpu(off), block, DTYPES[dt], out=out)
    assert not out[:off[0]].any() and not out[off[-1]:].any()
    for g, (lo, hi) in enumerate(zip(off, off[1:])):
        assert_product(out[lo:hi], exact_product(av[lo:hi], wv[g]), k, f"group {g}")


@pytest.mark.parametrize("off", [[90, 20, 80, 10], [0, 60, 30, 100, 10, 100], [-9, 200, 50, 1 << 62],
                                 [0, -5, 1 << 40, 100], [55, 0, 0, 70]])
def test_offsets_out_of_order_count_as_the_largest_before_them(off):
    say(f"offsets {off}")
    rows, n, k, block = 100, 48, 256, 128
    groups = len(off) - 1
    kept = np.maximum.accumulate(np.clip(np.array(off), 0, rows))
    rng = np.random.default_rng(len(off))
    a = to_gpu(random_operand(rows, k, block, rng))
    w = tuple(t.view(groups, n, -1) for t in to_gpu(random_operand(groups * n, k, block, rng)))
    x = torch.randn(rows, 24, device=DEV)

    def all_of(o):
        out = torch.full((rows, n), float("nan"), device=DEV)
        tfp8.matmul_grouped(a, w, gpu(o), block, torch.float32, out=out)
        ct = tfp8.compress_t(x, offsets=gpu(o))
        return out, *ct, tfp8.matmul_grouped_t(ct, ct, gpu(o), rows)

    for got, want in zip(all_of(off), all_of(kept)):
        assert not want.isnan().any() and torch.equal(got, want)


@pytest.mark.parametrize("off", [[40, 60, 60, 200], [0, 10, 150], [129, 131, 132, 200]])
def test_gradients_leave_rows_of_no_group_out(off):
    say(f"compress_t and matmul_grouped_t, offsets {off}")
    rows, m, n, block = 200, 64, 40, 128
    rng = np.random.default_rng(off[0])
    x, y = (torch.from_numpy(rng.standard_normal((rows, c)).astype(np.float32)).to(DEV)
            for c in (m, n))
    groups, kp = len(off) - 1, padded_length(rows, len(off) - 1, block)
    xt, yt = tfp8.compress_t(x, block, offsets=gpu(off)), tfp8.compress_t(y, block, offsets=gpu(off))
    assert xt[0].shape == (m, kp)
    got = tfp8.matmul_grouped_t(xt, yt, gpu(off), rows, block)
    for g, (lo, hi) in enumerate(zip(off, off[1:])):
        if lo == hi:
            assert not got[g].any()
            continue
        xg, yg = tfp8.compress_t(x[lo:hi], block), tfp8.compress_t(y[lo:hi], block)
        assert torch.equal(got[g], tfp8.matmul_grouped_t(xg, yg, gpu([0, hi - lo]), hi - lo, block)[0])
