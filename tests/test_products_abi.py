"""Argument checks of the products and of the transposed compress: every refusal comes before any
HIP call, so these run without a GPU."""
import numpy as np
import pytest
import torch

import fp8_compression_tensor_amd as tfp8

F = 0x7F0000000000  # an aligned address that is never dereferenced here
G = 1 << 30         # far enough apart for every buffer below
A = (F, 512, F + G, F + 2 * G, 4)
B = (F + 3 * G, 512, F + 4 * G, F + 5 * G, 4)
OUT, OFF = F + 6 * G, F + 7 * G
BIG = 1 << 31


def put(t, i, v):
    return t[:i] + (v,) + t[i + 1:]


def dense(a=A, b=B, m=8, n=16, k=512, block=128, out=OUT, dt=0, ldc=16):
    return tfp8.matmul_raw(a, b, m, n, k, block, out, dt, ldc)


def grouped(a=A, b=B, off=OFF, g=4, m=8, n=16, k=512, block=128, out=OUT, dt=0, ldc=16):
    return tfp8.matmul_grouped_raw(a, b, off, g, m, n, k, block, out, dt, ldc)


def grouped_t(a=A, b=B, off=OFF, g=2, rows=258, m=8, n=16, block=128, out=OUT, dt=0):
    return tfp8.matmul_grouped_t_raw(a, b, off, g, rows, m, n, block, out, dt)


def transpose(x=F, dt=0, rows=300, cols=40, ldx=40, off=None, g=1, block=128, target=1.0,
              codes=F + G, alpha=F + 2 * G, scale=F + 3 * G, flags=0):
    return tfp8.compress_t_raw(x, dt, rows, cols, ldx, off, g, block, target, codes, alpha, scale,
                               0, flags)


@pytest.mark.parametrize("call", [dense, grouped, grouped_t])
def test_products_refuse_what_they_share(call):
    for block in (0, 64, 96, 1024, -128):
        assert call(block=block) == -3
    assert call(dt=2) == -4
    assert call(m=-1) == -2 and call(n=-1) == -2 and call(m=BIG, n=0) == -2
    for i in (0, 2, 3):
        assert call(a=put(A, i, None)) == -1 and call(b=put(B, i, None)) == -1
    assert call(out=None) == -1
    assert call(a=put(A, 1, 496)) == -6 and call(b=put(B, 1, 511)) == -6
    assert call(a=put(A, 4, 3)) == -6 and call(b=put(B, 4, 3)) == -6
    assert call(a=put(A, 1, (1 << 22) + 16)) == -2 and call(b=put(B, 4, (1 << 20) + 1)) == -2
    assert call(a=put(A, 1, 520)) == -5 and call(a=put(A, 0, F + 8)) == -5
    assert call(b=put(B, 2, B[2] + 2)) == -5 and call(out=OUT + 1) == -5
    assert call(out=OUT + 2, dt=1) == -5
    for p in (A[0], A[2], A[3], B[0], B[2], B[3]):
        assert call(out=p) == -6  # the output over an input
    assert call(m=0) == 0 and call(n=0) == 0


def test_dense_and_grouped_sizes():
    for call in (dense, grouped):
        assert call(k=500) == -2 and call(k=-128) == -2 and call(k=(1 << 22) + 128) == -2
        assert call(ldc=15) == -6 and call(ldc=1 << 40) == -2
    # k = 0 reads nothing, so no operand pointer is asked for; the output still is
    none = (None, 0, None, None, 0)
    assert dense(a=none, b=none, k=0, out=None) == -1
    assert dense(a=none, b=none, k=0, m=0, out=None) == 0


def test_group_arguments():
    for call in (grouped, grouped_t):
        for g in (0, -1, tfp8.MAX_GROUPS + 1):
            assert call(g=g) == -6
        assert call(off=None) == -1 and call(off=OFF + 4) == -5
        assert call(off=OUT) == -6  # the output over the offsets
    assert grouped(n=1 << 30, ldc=1 << 30, m=0) == -2  # 4 x 2^30 rows of weights
    assert grouped_t(rows=-1) == -2 and grouped_t(rows=BIG) == -2
    assert grouped_t(rows=600) == -6  # rows that need a longer operand than ld


def test_compress_t_arguments():
    for block in (64, 96, 1024, 0):
        assert transpose(block=block) == -3
    assert transpose(rows=-1) == -2 and transpose(cols=-1) == -2 and transpose(rows=BIG) == -2
    assert transpose(cols=BIG) == -2 and transpose(dt=3) == -4
    for t in (0.0, -1.0, float("inf"), float("nan"), 2.0 ** 70, 2.0 ** -70):
        assert transpose(target=t) == -6
    assert transpose(flags=tfp8.FLAG_INT8) == -6 and transpose(flags=8) == -6
    assert transpose(g=0) == -6 and transpose(g=2) == -6 and transpose(off=OFF, g=1 << 17) == -6
    assert transpose(ldx=39) == -6
    assert transpose(rows=1 << 30, cols=1 << 30, ldx=1 << 30) == -2
    assert transpose(rows=1 << 20, ldx=1 << 30) == -2
    assert transpose(x=None) == -1 and transpose(codes=None) == -1
    assert transpose(alpha=None) == -1 and transpose(scale=None) == -1
    assert transpose(x=F + 1) == -5 and transpose(x=F + 2, dt=1) == -5
    assert transpose(codes=F + G + 8) == -5 and transpose(scale=F + 3 * G + 2) == -5
    assert transpose(off=OFF + 4) == -5
    assert transpose(codes=F + 1024) == -6 and transpose(alpha=F + G) == -6
    assert transpose(off=F + G) == -6
    assert transpose(cols=0, ldx=0, x=None, codes=None, alpha=None, scale=None) == 0
    assert transpose(rows=0, x=None, codes=None, alpha=None, scale=None) == 0


def test_padded_rows():
    L = tfp8.lib()
    rng = np.random.default_rng(0)
    for block in tfp8.PRODUCT_BLOCKS:
        assert tfp8.padded_rows(0, 1, block) == 0 and tfp8.padded_rows(1, 1, block) == block
        for _ in range(50):
            counts = rng.integers(0, 400, int(rng.integers(1, 9)))
            total = int(((counts + block - 1) // block * block).sum())
            p = tfp8.padded_rows(int(counts.sum()), len(counts), block)
            assert p % block == 0 and p >= total
            assert L.tfp8_padded_rows(int(counts.sum()), len(counts), block) == p
    # one row in every group is the longest that rows and groups can come to
    assert tfp8.padded_rows(7, 7, 128) == 7 * 128
    assert L.tfp8_padded_rows(-1, 1, 128) == 0 and L.tfp8_padded_rows(1, 0, 128) == 0
    with pytest.raises(ValueError):
        tfp8.padded_rows(1, 0, 128)


def test_wrappers_refuse_cpu_tensors():
    t = (torch.zeros(4, 128, dtype=torch.uint8), torch.ones(4, 1), torch.ones(4, 1))
    for call in (lambda: tfp8.matmul(t, t), lambda: tfp8.compress_t(torch.zeros(4, 4)),
                 lambda: tfp8.matmul_grouped(t, t, torch.zeros(2, dtype=torch.int64)),
                 lambda: tfp8.matmul_grouped_t(t, t, torch.zeros(2, dtype=torch.int64), 4)):
        with pytest.raises(ValueError, match="GPU"):
            call()
