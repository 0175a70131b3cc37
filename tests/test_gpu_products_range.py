"""Products of operands whose magnitudes lie far apart: blocks near 2^-135 or 2^-128, whose factor s / alpha is
below float32's normal range, by blocks near 2^60, with results well inside it.  The sizes reach every
kernel on 256 compute units (the comments, as in test_gpu_products_kernels.py)."""
import numpy as np
import pytest
import torch

import fp8_compression_tensor_amd as tfp8
from gpu_helpers import say
from product_helpers import DEV, assert_product, offsets_of, rotated_values

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def values(rows, cols, block, powers, seed):
    """Normal values times a power of two: that of row i and block j is powers[(i + i // 3 * j) % len]."""
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal((rows, cols)))
    i, j = torch.arange(rows)[:, None], torch.arange(cols)[None] // block
    e = torch.tensor(powers, dtype=torch.float64)[(i + i // 3 * j) % len(powers)]
    return (x * torch.exp2(e)).to(torch.float32).to(DEV)  # rounded once, also where it is subnormal


def as_float64(op, block):
    codes, alpha, scale = (t.cpu().numpy() for t in op)
    return torch.from_numpy(rotated_values((codes, alpha, scale), block)).to(DEV)


def exact(a, b):
    """As product_helpers.exact_product, in float64 on the GPU."""
    return tuple(t.cpu().numpy() for t in (a @ b.T, a.abs() @ b.abs().T, ((a * a) @ (b * b).T).sqrt()))


TINY, LARGE = [-135, 0, -128], [60, 0]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k,block", [
    (5, 100, 256, 128),      # few16 / few16
    (33, 4200, 1536, 512),   # few32 / few32
    (28, 10300, 1280, 256),  # few48 / few48
    (90, 9000, 1152, 128),   # 64+ / 64
    (200, 2600, 1280, 128),  # 64+ / 64+
    (777, 2561, 640, 128),   # 64 / 64
    (1537, 2561, 640, 128),  # 128 / 128
    (2300, 4100, 768, 256),  # 256 / 128
])
@pytest.mark.parametrize("tiny_first", [True, False])
def test_matmul_of_tiny_by_large_blocks(m, n, k, block, tiny_first, dt):
    say(f"matmul {m}x{n}x{k} block {block} {dt}, tiny values in {'a' if tiny_first else 'b'}")
    pa, pb = (TINY, LARGE) if tiny_first else (LARGE, TINY)
    a = tfp8.compress(values(m, k, block, pa, 1), block)
    b = tfp8.compress(values(n, k, block, pb, 2), block)
    want = exact(as_float64(a, block), as_float64(b, block))
    assert_product(tfp8.matmul(a, b, block, DTYPES[dt]), want, k, f"{m}x{n}x{k}")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("counts,n,k,block", [([3, 0, 9], 200, 512, 128), ([300, 1, 0, 200], 500, 512, 256)])
def test_matmul_grouped_of_tiny_by_large_blocks(counts, n, k, block, dt):
    say(f"matmul_grouped {counts} n {n} k {k} block {block} {dt}, tiny values in a")
    rows, groups, off = sum(counts), len(counts), offsets_of(counts)
    a = tfp8.compress(values(rows, k, block, TINY, 3), block)
    w = tfp8.compress(values(groups * n, k, block, LARGE, 4), block)
    av, wv = as_float64(a, block), as_float64(w, block).view(groups, n, k)
    w = (w[0].view(groups, n, k), *(t.view(groups, n, -1) for t in w[1:]))
    got = tfp8.matmul_grouped(a, w, torch.from_numpy(off).to(DEV), block, DTYPES[dt])
    for g, (lo, hi) in enumerate(zip(off, off[1:])):
        assert_product(got[lo:hi], exact(av[lo:hi], wv[g]), k, f"group {g}")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("counts,m,n,block", [([200, 0, 130], 100, 70, 128), ([300, 700], 600, 300, 256)])
def test_matmul_grouped_t_of_tiny_by_large_blocks(counts, m, n, block, dt):
    say(f"matmul_grouped_t {counts} {m}x{n} block {block} {dt}, tiny values in a")
    rows, off = sum(counts), offsets_of(counts)
    og = torch.from_numpy(off).to(DEV)
    # the blocks run along the rows: powers by column and by block of rows
    x = values(m, rows, block, TINY, 5).t().contiguous()
    y = values(n, rows, block, LARGE, 6).t().contiguous()
    xt, yt = (tfp8.compress_t(t, block, offsets=og) for t in (x, y))
    xv, yv = as_float64(xt, block), as_float64(yt, block)
    got = tfp8.matmul_grouped_t(xt, yt, og, rows, block, DTYPES[dt])
    at = 0
    for g, c in enumerate(counts):
        to = at + (c + block - 1) // block * block
        assert_product(got[g], exact(xv[:, at:to], yv[:, at:to]), to - at, f"group {g}")
        at = to


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k", [(5, 100, 256), (300, 300, 640)])
def test_subnormal_gradients_by_ordinary_values(m, n, k, dt):
    """bfloat16-subnormal blocks beside ordinary ones, by values around 1: what the r of the former loses is
    below 2^-123 for each 128 codes, where the smallest normal float32 is 2^-126."""
    say(f"matmul {m}x{n}x{k} {dt} with subnormal blocks")
    a = values(m, k, 128, [-8, -130, -8, -8], 7).to(torch.bfloat16)
    a, b = tfp8.compress(a), tfp8.compress(values(n, k, 128, [0], 8).to(torch.bfloat16))
    e, mag, mag2 = exact(as_float64(a, 128), as_float64(b, 128))
    got = tfp8.matmul(a, b, 128, DTYPES[dt])
    # as a part of the magnitudes that the bound counts at 2^-16 and more of them
    mag = mag + k // 128 * 2.0 ** (16 - 123)
    assert_product(got, (e, mag, mag2), k, f"{m}x{n}x{k}")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k", [(5, 100, 256), (90, 9000, 1152), (300, 300, 640), (1537, 2561, 640)])
def test_huge_values_that_do_not_meet(m, n, k, dt):
    """Without the rotation, one value of 2^80 to 2^99 a block, at other places in a than in b: the
    product of the factors leaves float32's range, and the sums are 0."""
    say(f"matmul {m}x{n}x{k} {dt}, huge values at different places")
    block, off = 128, tfp8.FLAG_NO_ROTATION
    a, b = torch.zeros(m, k, device=DEV), torch.zeros(n, k, device=DEV)
    a[:, 3::block] = torch.exp2(80 + torch.arange(m, device=DEV) % 20).float()[:, None]
    b[:, 70::block] = -torch.exp2(99 - torch.arange(n, device=DEV) % 20).float()[:, None]
    a, b = tfp8.compress(a, block, flags=off), tfp8.compress(b, block, flags=off)
    assert not tfp8.matmul(a, b, block, DTYPES[dt]).any()
