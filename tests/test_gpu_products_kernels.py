"""Products of compressed operands at sizes that reach every kernel a product may be sent to.

A product goes to the kernel whose rounds of workgroups are estimated to be done first, so that each
appears only at sizes of its own.  The comment on each case names what an MI355X (256 compute units)
takes for it, bfloat16 / float32: `256`, `128` and `64` the tiles of so many rows and columns, `64+` the last with two teams, `few16`, `few32`, `few48` the kernels for few rows by their
columns.  On another number of compute units the cases stay right and reach other kernels."""
import numpy as np
import pytest
import torch

import fp8_compression_tensor_amd as tfp8
from gpu_helpers import say
from product_helpers import (DEV, assert_product, offsets_of, padded_length, random_operand,
                             rotated_values, to_gpu)

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def exact_on_gpu(a, b):
    """exact_product of float64 arrays, computed in float64 on the GPU."""
    a, b = torch.from_numpy(a).to(DEV), torch.from_numpy(b).to(DEV)
    return tuple(t.cpu().numpy() for t in (a @ b.T, a.abs() @ b.abs().T, ((a * a) @ (b * b).T).sqrt()))


def framed(m, n, dtype):
    """(buffer, an [m, n] view within it whose rows start at odd elements)."""
    buf = torch.full((m + 2, n + 37), 5.0, dtype=dtype, device=DEV)
    return buf, buf[1:m + 1, 1:n + 1]


def assert_frame(buf, out, what):
    out.fill_(5.0)
    assert (buf == 5.0).all(), f"{what}: written outside the output"


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k,block", [
    (260, 100, 8448, 128),    # few16 / few16, 66 blocks: scales refilled
    (260, 1100, 8448, 128),   # few32 / few32, refilled
    (33, 4200, 4608, 512),    # few32 / few32
    (28, 10300, 2560, 256),   # few48 / few48
    (20, 11000, 8448, 128),   # few48 / few48, refilled
    (90, 9000, 2176, 128),    # 64+ / 64, the teams' steps uneven, 17 blocks: refilled
    (200, 2600, 4352, 256),   # 64+ / 64+, refilled
    (130, 4200, 4608, 512),   # 64+ / few48
    (777, 2561, 2176, 128),   # 64 / 64, refilled
    (777, 2561, 2560, 512),   # 64 / 64
    (1537, 2561, 1152, 128),  # 128 / 128
    (1537, 2561, 2560, 256),  # 128 / 128
    (2100, 4100, 1152, 128),  # 256 / 128
    (2300, 4100, 1280, 256),  # 256 / 128
    (2300, 4100, 1536, 512),  # 256 / 128
    (4100, 4300, 640, 128),   # 128 / 128
    (4100, 4300, 1280, 256),  # 128 / 128
    (4100, 4300, 1536, 512),  # 128 / 128
])
def test_matmul_in_every_kernel(m, n, k, block, dt):
    say(f"matmul {m}x{n}x{k} block {block} {dt}")
    rng = np.random.default_rng(m + n + k)
    a, b = random_operand(m, k, block, rng), random_operand(n, k, block, rng)
    want = exact_on_gpu(rotated_values(a, block), rotated_values(b, block))
    buf, out = framed(m, n, DTYPES[dt])
    tfp8.matmul(to_gpu(a), to_gpu(b), block, DTYPES[dt], out=out)
    assert_product(out, want, k, f"{m}x{n}x{k}")
    assert_frame(buf, out, f"{m}x{n}x{k}")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("counts,n,k,block", [
    ([10, 0, 20], 1000, 8448, 128),            # few16 / few16, refilled
    ([14, 0, 9], 5100, 8448, 128),             # few16 / few16, refilled
    ([100, 1, 159], 1000, 2176, 128),          # few32 / few48
    ([20, 12, 30], 5000, 8448, 128),           # few32 / few32, refilled
    ([33], 9000, 1024, 256),                   # few48 / few48
    ([40] * 5, 2305, 8448, 128),               # 64+ / few48, refilled
    ([100, 1, 159], 3000, 2176, 128),          # 64+ / 64+
    ([300, 0, 777, 1, 500], 1793, 2176, 128),  # 64 / 64, refilled
    ([300, 0, 777, 1, 500], 2561, 1536, 512),  # 128 / 128
    ([2100, 0, 3, 400], 2561, 1152, 128),      # 128 / 128
    ([2100, 0, 3, 400], 4100, 1280, 256),      # 256 / 128
    ([1] * 200 + [0] * 60 + [300, 2], 300, 384, 128),  # more groups than a wavefront has lanes
])
def test_matmul_grouped_in_every_kernel(counts, n, k, block, dt):
    say(f"matmul_grouped {counts}, n {n} k {k} block {block} {dt}")
    rng = np.random.default_rng(sum(counts) + n + k)
    groups, rows, off = len(counts), sum(counts), offsets_of(counts)
    a, w = random_operand(rows, k, block, rng), random_operand(groups * n, k, block, rng)
    av, wv = rotated_values(a, block), rotated_values(w, block).reshape(groups, n, k)
    parts = [exact_on_gpu(av[lo:hi], wv[g]) for g, (lo, hi) in enumerate(zip(off, off[1:]))]
    want = tuple(np.concatenate(t) for t in zip(*parts))
    wg = tuple(t.view(groups, n, -1) for t in to_gpu(w))
    buf, out = framed(rows, n, DTYPES[dt])
    tfp8.matmul_grouped(to_gpu(a), wg, torch.from_numpy(off).to(DEV), block, DTYPES[dt], out=out)
    assert_product(out, want, k, str(counts))
    assert_frame(buf, out, str(counts))


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("counts,m,n,block", [
    ([1300], 260, 1793, 128),                       # 64+ / 64+
    ([2500], 260, 1793, 128),                       # 64+ / 64+, refilled
    ([2200, 0, 2100], 260, 2561, 128),              # 64 / 64, refilled
    ([0, 1000, 793], 520, 2049, 256),               # 64 / 64
    ([300, 0, 777, 1, 500], 260, 3001, 512),        # 128 / 128
    ([300, 0, 777, 1, 500], 520, 2049, 128),        # 128 / 128
    ([300, 0, 777, 1, 500], 2050, 2561, 128),       # 256 / 128
])
def test_matmul_grouped_t_in_every_kernel(counts, m, n, block, dt):
    say(f"matmul_grouped_t {counts}, {m}x{n} block {block} {dt}")
    rng = np.random.default_rng(sum(counts) + n + m)
    groups, rows, off = len(counts), sum(counts), offsets_of(counts)
    kp = padded_length(rows, groups, block)
    a, b = random_operand(m, kp, block, rng), random_operand(n, kp, block, rng)
    av, bv = rotated_values(a, block), rotated_values(b, block)
    got = tfp8.matmul_grouped_t(to_gpu(a), to_gpu(b), torch.from_numpy(off).to(DEV), rows, block,
                                DTYPES[dt])
    at = 0
    for g, c in enumerate(counts):
        to = at + (c + block - 1) // block * block
        want = exact_on_gpu(av[:, at:to], bv[:, at:to])
        assert_product(got[g], want, to - at, f"{counts} group {g}")
        at = to


@pytest.mark.parametrize("m,n,k", [(90, 9000, 2176), (260, 1100, 8448), (777, 2561, 2176),
                                   (1537, 2561, 1152), (2300, 4100, 1152)])
def test_large_products_repeat_bit_for_bit(m, n, k):
    say(f"matmul {m}x{n}x{k} four times")
    rng = np.random.default_rng(k)
    a, b = to_gpu(random_operand(m, k, 128, rng)), to_gpu(random_operand(n, k, 128, rng))
    for dtype in DTYPES.values():
        first = tfp8.matmul(a, b, 128, dtype)
        assert all(torch.equal(first, tfp8.matmul(a, b, 128, dtype)) for _ in range(3))


@pytest.mark.parametrize("rows,groups,used", [(3, 200, 2), (40, 40, 40), (41, 40, 30), (100, 5000, 60)])
def test_matmul_grouped_with_more_groups_than_tiles_of_rows(rows, groups, used):
    """One row to each of `used` groups spread over all of them, the rest past the last group."""
    say(f"matmul_grouped {rows} rows, {used} of {groups} groups with one")
    n, k, block = 48, 256, 128
    rng = np.random.default_rng(groups)
    counts = np.zeros(groups, np.int64)
    counts[np.sort(rng.choice(groups, used, replace=False))] = 1
    off = offsets_of(counts)
    a, w = random_operand(rows, k, block, rng), random_operand(groups * n, k, block, rng)
    av, wv = rotated_values(a, block), rotated_values(w, block).reshape(groups, n, k)
    rep = np.repeat(np.arange(groups), counts)
    wg = tuple(t.view(groups, n, -1) for t in to_gpu(w))
    out = torch.full((rows, n), 7.0, device=DEV)
    tfp8.matmul_grouped(to_gpu(a), wg, torch.from_numpy(off).to(DEV), block, torch.float32, out=out)
    parts = [exact_on_gpu(av[i:i + 1], wv[g]) for i, g in enumerate(rep)]
    assert_product(out[:used], tuple(np.concatenate(t) for t in zip(*parts)), k, "groups of one row")
    assert not out[used:].any()
