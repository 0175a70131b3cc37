"""Products and the transposed compress with operands and outputs past 4 GiB, in the kernels for many rows,
for groups and along the depth: rows are a short operand's again and again, so that a float64
product of it says what every part of the output holds."""
import numpy as np
import pytest
import torch

import fp8_compression_tensor_amd as tfp8
from gpu_helpers import say
from product_helpers import DEV, assert_product, exact_product, random_operand, rotated_values, to_gpu

pytestmark = pytest.mark.gpu


def need(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"less than {gib} GiB of free device memory")


def again(op, rows):
    """op's rows from the first on until there are `rows`."""
    n = op[0].shape[0]
    return tuple(torch.cat([t.repeat(rows // n, 1), t[:rows % n]]) for t in op)


def operand(rows, k, block, seed):
    op = random_operand(rows, k, block, np.random.default_rng(seed))
    return to_gpu(op), rotated_values(op, block)


def assert_repeats(out, dim, n, what):
    """Slices of n along dim are equal, the last one cut off."""
    first = out.narrow(dim, 0, n)
    for at in range(n, out.shape[dim], n):
        c = min(n, out.shape[dim] - at)
        assert torch.equal(out.narrow(dim, at, c), first.narrow(dim, 0, c)), (what, at)


def test_tiles_of_a_large_operand():
    say("matmul 130 x 1148576 x 4096: 4.7 GB of codes in b")
    need(24)
    m, n, k, block = 130, (1 << 20) + 100000, 4096, 256
    a, av = operand(m, k, block, 1)
    t, tv = operand(1000, k, block, 2)
    got = tfp8.matmul(a, again(t, n), block)
    assert_product(got[:, :1000], exact_product(av, tv), k, "first columns")
    assert_repeats(got, 1, 1000, "columns")


@pytest.mark.parametrize("dtype,m", [(torch.bfloat16, 66100), (torch.float32, 33100)])
def test_tiles_of_a_large_output(dtype, m):
    say(f"matmul {m} x 33000 x 256 {dtype}: 4.4 GB of output")
    need(24)
    n, k, block = 33000, 256, 128
    a, av = operand(1000, k, block, 3)
    b, bv = operand(n, k, block, 4)
    got = tfp8.matmul(again(a, m), b, block, dtype)
    assert got.numel() * got.element_size() > 1 << 32
    assert_product(got[:200], exact_product(av[:200], bv), k, "first rows")
    assert_repeats(got, 0, 1000, "rows")


@pytest.mark.parametrize("each", [3, 70])  # the kernels for few rows, and tiles
def test_groups_of_large_weights(each):
    say(f"matmul_grouped, {each} rows in each of 35 groups, 4.7 GB of codes in b")
    need(24)
    groups, n, k, block = 35, 32768, 4096, 512
    a, av = operand(each, k, block, 5)
    t, tv = operand(1024, k, block, 6)
    w = tuple(x.view(groups, n, -1) for x in again(t, groups * n))
    off = torch.arange(groups + 1, device=DEV) * each
    got = tfp8.matmul_grouped(again(a, groups * each), w, off, block, torch.float32)
    assert_product(got[:each, :1024], exact_product(av, tv), k, "first group")
    assert_repeats(got, 0, each, "groups")
    assert_repeats(got, 1, 1024, "columns")


def test_gradients_of_large_weights():
    say("matmul_grouped_t, 16 groups of 8300 x 8300 float32: 4.4 GB of output")
    need(24)
    groups, c, each, block = 16, 8300, 40, 128
    rows = groups * each
    x = torch.randn(each, c, device=DEV)
    off = torch.arange(groups + 1, device=DEV) * each
    xt = tfp8.compress_t(x.repeat(groups, 1), block, offsets=off)
    got = tfp8.matmul_grouped_t(xt, xt, off, rows, block)
    assert got.numel() * 4 > 1 << 32
    xv = rotated_values(tuple(t[:300, :w].cpu().numpy() for t, w in zip(xt, (block, 1, 1))), block)
    assert_product(got[0, :300, :300], exact_product(xv, xv), block, "first group")
    assert_repeats(got.view(groups * c, c), 0, c, "groups")


def test_compress_t_of_a_large_matrix():
    say("compress_t 66100 x 66000 bfloat16: 8.7 GB, 4.4 GB of codes")
    need(48)
    rows, cols, block = 66100, 66000, 128
    x = torch.randn(1000, cols, device=DEV).to(torch.bfloat16).repeat(67, 1)[:rows]
    codes, alpha, scale = tfp8.compress_t(x, block)
    assert codes.numel() > 1 << 32
    for lo, hi in ((0, 200), (cols // 2, cols // 2 + 64), (cols - 130, cols)):
        want = tfp8.compress_t(x[:, lo:hi].contiguous(), block)
        for g, w in zip((codes, alpha, scale), want):
            assert torch.equal(g[lo:hi], w), (lo, hi)
    off = torch.tensor([0, 33000, 65990], device=DEV)
    codes, alpha, scale = tfp8.compress_t(x, block, offsets=off)
    want = tfp8.compress_t(x[:, -70:].contiguous(), block, offsets=off)
    for g, w in zip((codes, alpha, scale), want):
        assert torch.equal(g[-70:], w)
