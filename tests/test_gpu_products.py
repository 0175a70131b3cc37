"""Products of compressed operands and the transposed compress on the GPU, against float64."""
import numpy as np
import pytest
import torch

import fp8_compression_tensor_amd as tfp8
from gpu_helpers import assert_scales, say
from product_helpers import (DEV, assert_product, exact_product, offsets_of, padded_length,
                             padded_transpose, random_operand, rotated_values, to_gpu)
from tiecheck import assert_codes_match

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def bits_of(x):
    """float32 -> bfloat16 bit patterns, by truncation (any bfloat16 values will do as inputs)."""
    return (np.ascontiguousarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def bits_to_f32(b):
    return (b.astype(np.uint32) << 16).view(np.float32)


# ------------------------------------------------------------------------------------ compress_t

def check_compress_t(oracle, x, offsets, block, dtype, target=1.0, flags=0, what=""):
    """x: float32 values exact in dtype, [rows, cols]."""
    groups = 1 if offsets is None else len(offsets) - 1
    rows, cols = x.shape
    kp = padded_length(rows, groups, block)
    off = offsets_of([rows]) if offsets is None else offsets
    xt = padded_transpose(x, off, block)
    src = bits_of(xt) if dtype == torch.bfloat16 else xt
    rq, ra, rs, rt = oracle.compress(np.ascontiguousarray(src).reshape(-1), block, target,
                                     with_quot=True, flags=flags)
    xg = torch.from_numpy(x).to(DEV).to(dtype)
    og = None if offsets is None else torch.from_numpy(offsets).to(DEV)
    codes, alpha, scale = tfp8.compress_t(xg, block, target, offsets=og, flags=flags)
    assert codes.shape == (cols, kp) and alpha.shape == scale.shape == (cols, kp // block)
    # a tie decided the other way is admissible; on a few thousand elements the usual cap of a
    # fraction of them would be less than one element
    assert_codes_match(codes.cpu().numpy().reshape(-1), rq, rt, what=what,
                       max_frac=max(1e-2 if flags else 1e-4, 2.0 / max(rq.size, 1)))
    assert_scales(alpha.cpu().numpy(), scale.cpu().numpy(), ra, rs, what)
    return codes, alpha, scale


def tp_values(rng, rows, cols, dtype):
    x = (rng.standard_normal((rows, cols)) * np.exp(0.7 * rng.standard_normal(cols))).astype(
        np.float32)
    x[rng.random((rows, cols)) < 1e-3] *= 40
    return bits_to_f32(bits_of(x)) if dtype == torch.bfloat16 else x


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("block", tfp8.PRODUCT_BLOCKS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 64), (127, 3), (128, 64), (129, 65), (517, 33),
                                       (1024, 256), (300, 130)])
def test_compress_t_matches_the_oracle(oracle, rows, cols, block, dt):
    say(f"compress_t {rows}x{cols} block {block} {dt}")
    rng = np.random.default_rng(rows * 1000 + cols + block)
    x = tp_values(rng, rows, cols, DTYPES[dt])
    x[:, cols // 2] = 0  # a column of zero blocks
    check_compress_t(oracle, x, None, block, DTYPES[dt], what=f"{rows}x{cols}")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("block", tfp8.PRODUCT_BLOCKS)
def test_compress_t_without_the_rotation(oracle, block, dt):
    say(f"compress_t without rotation, block {block} {dt}")
    x = tp_values(np.random.default_rng(5), 700, 40, DTYPES[dt])
    check_compress_t(oracle, x, None, block, DTYPES[dt], target=3.0,
                     flags=tfp8.FLAG_NO_ROTATION, what="no rotation")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("block", [128, 512])
@pytest.mark.parametrize("counts", [[5, 0, 128, 1, 200], [0, 0, 3], [300], [1] * 70, [0] * 3,
                                    [0] * 65 + [130] + [0] * 63 + [1]])
def test_compress_t_of_groups(oracle, counts, block, dt):
    say(f"compress_t groups {len(counts)} rows {sum(counts)} block {block} {dt}")
    x = tp_values(np.random.default_rng(len(counts)), sum(counts), 20, DTYPES[dt])
    check_compress_t(oracle, x, offsets_of(counts), block, DTYPES[dt], what=str(counts[:5]))


def test_compress_t_leaves_rows_past_the_groups_out(oracle):
    say("compress_t rows past the last group")
    x = tp_values(np.random.default_rng(3), 400, 24, torch.float32)
    codes, _, scale = check_compress_t(oracle, x, np.array([0, 100, 260]), 128, torch.float32)
    assert not codes[:, 384:].any() and not scale[:, 3:].any()


@pytest.mark.parametrize("k", [-140, -100, 80, 99])
@pytest.mark.parametrize("block", [128, 256])
def test_compress_t_of_tiny_and_huge_values(oracle, block, k):
    say(f"compress_t of values near 2^{k}, block {block}")
    rng = np.random.default_rng(k + 500)
    x = np.ldexp(rng.uniform(0.5, 0.99, (block + 9, 16)), k).astype(np.float32)
    check_compress_t(oracle, x, None, block, torch.float32, what=f"2^{k}")


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("ld,col", [(97, 0), (97, 1), (128, 8), (100, 4)])
def test_compress_t_of_strided_rows(oracle, ld, col, dt):
    say(f"compress_t rows {ld} apart from column {col} {dt}")
    big = torch.from_numpy(tp_values(np.random.default_rng(9), 260, ld, DTYPES[dt])).to(DEV)
    big = big.to(DTYPES[dt])
    x = big[:, col:col + 80]
    got = tfp8.compress_t(x, 128)
    want = tfp8.compress_t(x.contiguous(), 128)
    assert all(torch.equal(g, w) for g, w in zip(got, want))


def test_compress_t_agrees_with_compress_of_the_transpose():
    say("compress_t against compress of a transposed copy")
    x = torch.randn(1024, 320, device=DEV).to(torch.bfloat16)
    codes, alpha, scale = tfp8.compress_t(x, 256)
    c2, a2, s2 = tfp8.compress(x.t().contiguous(), 256)
    assert (codes != c2).float().mean() < 1e-4
    assert torch.allclose(alpha.view(-1), a2, rtol=1e-6) and torch.allclose(scale.view(-1), s2,
                                                                           rtol=1e-6)


# ---------------------------------------------------------------------------------------- matmul

@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n,k,block", [
    (1, 1, 128, 128), (1, 17, 256, 256), (2, 64, 512, 512), (3, 1000, 1280, 128),
    (16, 16, 384, 128), (17, 33, 640, 128), (31, 100, 2560, 256), (33, 65, 1024, 512),
    (64, 128, 4096, 128), (65, 127, 128, 128), (127, 129, 768, 256), (128, 128, 1536, 128),
    (200, 257, 512, 128), (256, 256, 128, 128), (257, 255, 1024, 256), (300, 520, 2048, 512),
    (1, 4099, 5120, 128), (5, 640, 10240, 128), (700, 3, 896, 128), (48, 300, 128, 128)])
def test_matmul_matches_float64(m, n, k, block, dt):
    say(f"matmul {m}x{n}x{k} block {block} {dt}")
    rng = np.random.default_rng(m * 7919 + n * 31 + k)
    a, b = random_operand(m, k, block, rng), random_operand(n, k, block, rng)
    want = exact_product(rotated_values(a, block), rotated_values(b, block))
    got = tfp8.matmul(to_gpu(a), to_gpu(b), block, DTYPES[dt])
    assert_product(got, want, k, f"{m}x{n}x{k}")


@pytest.mark.parametrize("dt", DTYPES)
def test_matmul_is_the_product_of_the_decompressed_operands(dt):
    say(f"matmul of compressed tensors against their reconstructions {dt}")
    x = torch.randn(200, 1024, device=DEV).to(torch.bfloat16)
    w = torch.randn(333, 1024, device=DEV).to(torch.bfloat16)
    for flags in (0, tfp8.FLAG_NO_ROTATION):
        a, b = tfp8.compress(x, 128, flags=flags), tfp8.compress(w, 128, 2.0, flags=flags)
        xh = tfp8.decompress(*a, 128, flags=flags).double().cpu()
        wh = tfp8.decompress(*b, 128, flags=flags).double().cpu()
        # products in the rotated basis: their magnitudes sum to at most |x| |w| (Cauchy-Schwarz);
        # the reconstructions are rounded to float32, 2^-24 of each factor: two more steps
        mag = np.outer(xh.norm(dim=1), wh.norm(dim=1))
        got = tfp8.matmul(a, b, 128, DTYPES[dt])
        assert_product(got, ((xh @ wh.t()).numpy(), mag, mag), 1024 + 128 * 2, "decompressed")


def test_matmul_of_no_depth_and_no_rows():
    say("matmul with k = 0, m = 0, n = 0")
    e = lambda r, k: (torch.empty(r, k, dtype=torch.uint8, device=DEV),
                      torch.empty(r, k // 128, device=DEV), torch.empty(r, k // 128, device=DEV))
    assert torch.equal(tfp8.matmul(e(5, 0), e(40, 0)).float(), torch.zeros(5, 40, device=DEV))
    assert tfp8.matmul(e(0, 256), e(40, 256)).shape == (0, 40)
    assert tfp8.matmul(e(7, 256), e(0, 256)).shape == (7, 0)


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("m,n", [(1, 100), (40, 129), (300, 300)])
def test_matmul_of_strided_operands_into_a_strided_output(m, n, dt):
    say(f"matmul with row strides {m}x{n} {dt}")
    k, block = 640, 128
    rng = np.random.default_rng(m + n)

    def strided(rows):
        """Rows of one receive buffer: [codes | alpha | scale] per row, and a gap."""
        op = to_gpu(random_operand(rows, k, block, rng))
        nb = k // block
        ld = (k + 8 * nb + 15) // 16 * 16 + 48
        buf = torch.full((rows, ld), 0x77, dtype=torch.uint8, device=DEV)
        buf[:, :k] = op[0]
        f = buf.view(torch.float32)
        f[:, k // 4:k // 4 + nb], f[:, k // 4 + nb:k // 4 + 2 * nb] = op[1], op[2]
        return op, (buf[:, :k], f[:, k // 4:k // 4 + nb], f[:, k // 4 + nb:k // 4 + 2 * nb])

    (a, av), (b, bv) = strided(m), strided(n)
    want = tfp8.matmul(a, b, block, DTYPES[dt])
    for shift in (0, 1):  # an output row at any alignment
        buf = torch.full((m + 2, n + 37), 5.0, dtype=DTYPES[dt], device=DEV)
        out = buf[1:m + 1, shift:shift + n]
        tfp8.matmul(av, bv, block, DTYPES[dt], out=out)
        assert torch.equal(out, want)
        out.fill_(5.0)
        assert (buf == 5.0).all()  # nothing outside the view was written


def test_matmul_keeps_the_range_of_its_scales():
    say("matmul of operands with very small and very large scales")
    k, block = 256, 128
    rng = np.random.default_rng(8)
    a, b = (random_operand(20, k, block, rng, zero_blocks=0.0) for _ in range(2))
    a = (a[0], np.full_like(a[1], 2.0 ** 90), a[2])   # r about 2^-98
    b = (b[0], np.full_like(b[1], 2.0 ** -80), b[2])  # r about 2^72
    want = exact_product(rotated_values(a, block), rotated_values(b, block))
    assert_product(tfp8.matmul(to_gpu(a), to_gpu(b), block, torch.float32), want, k, "range")


def test_matmul_past_32_bit_offsets():
    say("matmul with 4.6 GB of codes in one operand")
    k, n, m, block = 4096, 1 << 20, 24, 256
    n += 100000
    need = n * k + n * m * 4 + (2 << 30)
    if torch.cuda.mem_get_info()[0] < 2 * need:
        pytest.skip("not enough free device memory")
    rng = np.random.default_rng(4)
    a = random_operand(m, k, block, rng)
    tile = random_operand(1000, k, block, rng)
    t = to_gpu(tile)
    b = tuple(torch.cat([x.repeat(n // 1000, 1), x[:n % 1000]]) for x in t)
    got = tfp8.matmul(to_gpu(a), b, block, torch.float32)
    want = exact_product(rotated_values(a, block), rotated_values(tile, block))
    assert_product(got[:, :1000], want, k, "first rows")
    last = (n - 1000) // 1000 * 1000
    assert last * k > 1 << 32
    assert_product(got[:, last:last + 1000], want, k, "last rows")
    assert torch.equal(got[:, :1000].repeat(1, n // 1000 + 1)[:, :n], got)


def test_products_on_another_stream_and_in_a_graph():
    say("products on a stream of their own and replayed from a graph")
    rng = np.random.default_rng(12)
    a, b = to_gpu(random_operand(70, 1024, 128, rng)), to_gpu(random_operand(500, 1024, 128, rng))
    w = to_gpu(random_operand(4 * 130, 1024, 128, rng))
    w = tuple(t.view(4, 130, -1) for t in w)
    off = torch.tensor([0, 10, 10, 60, 70], device=DEV)
    x = torch.randn(70, 200, device=DEV)
    y = torch.randn(70, 90, device=DEV)

    def step():
        ct, dt = tfp8.compress_t(x, offsets=off), tfp8.compress_t(y, offsets=off)
        return (tfp8.matmul(a, b), tfp8.matmul_grouped(a, w, off), *ct,
                tfp8.matmul_grouped_t(ct, dt, off, 70))

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(g, t) for g, t in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, t) for g, t in zip(out, want)), i
        assert all(torch.equal(g, t) for g, t in zip(step(), want)), i


def test_products_repeat_bit_for_bit():
    say("products twice on the same inputs")
    rng = np.random.default_rng(13)
    for m, n, k in [(1, 4096, 4096), (24, 1000, 5120), (500, 700, 2560)]:
        a, b = to_gpu(random_operand(m, k, 128, rng)), to_gpu(random_operand(n, k, 128, rng))
        first = tfp8.matmul(a, b, 128, torch.float32)
        assert all(torch.equal(first, tfp8.matmul(a, b, 128, torch.float32)) for _ in range(3))


# --------------------------------------------------------------------------------------- grouped

COUNTS = [[7, 0, 130, 1, 300], [0, 0, 5], [64], [1] * 70, [0, 200, 0], [33, 31, 64, 128, 129],
          [0] * 65 + [40] + [0] * 66 + [3]]


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("n,k,block", [(16, 128, 128), (130, 640, 128), (65, 1024, 512)])
def test_matmul_grouped_matches_float64(counts, n, k, block, dt):
    say(f"matmul_grouped {len(counts)} groups, {sum(counts)} rows, n {n} k {k} block {block} {dt}")
    rng = np.random.default_rng(n + k + len(counts))
    groups, rows = len(counts), sum(counts)
    a, w = random_operand(rows, k, block, rng), random_operand(groups * n, k, block, rng)
    off = offsets_of(counts)
    av, wv = rotated_values(a, block), rotated_values(w, block).reshape(groups, n, k)
    parts = [exact_product(av[lo:hi], wv[g]) for g, (lo, hi) in enumerate(zip(off, off[1:]))]
    want = tuple(np.concatenate(t) for t in zip(*parts))
    wg = tuple(t.view(groups, n, -1) for t in to_gpu(w))
    got = tfp8.matmul_grouped(to_gpu(a), wg, torch.from_numpy(off).to(DEV), block, DTYPES[dt])
    assert_product(got, want, k, str(counts[:5]))


def test_matmul_grouped_writes_zeros_past_the_last_group():
    say("matmul_grouped rows past the last group")
    rng = np.random.default_rng(2)
    a, w = to_gpu(random_operand(300, 256, 128, rng)), to_gpu(random_operand(2 * 50, 256, 128, rng))
    w = tuple(t.view(2, 50, -1) for t in w)
    out = torch.full((300, 50), 9.0, device=DEV)
    off = torch.tensor([0, 20, 90], device=DEV)
    tfp8.matmul_grouped(a, w, off, 128, torch.float32, out=out)
    assert not out[90:].any() and out[:90].abs().sum(1).gt(0).all()


def test_offsets_out_of_range_touch_nothing_outside():
    # the offsets are clamped on the device: whatever they hold, the call ends and stays inside
    say("offsets that break the rules")
    rng = np.random.default_rng(6)
    a, w = to_gpu(random_operand(100, 256, 128, rng)), to_gpu(random_operand(3 * 40, 256, 128, rng))
    w = tuple(t.view(3, 40, -1) for t in w)
    x = torch.randn(100, 24, device=DEV)
    for bad in ([0, -5, 1 << 40, 100], [-9, 200, 50, 1 << 62], [90, 20, 80, 10]):
        off = torch.tensor(bad, device=DEV)
        buf = torch.full((104, 40), 3.0, device=DEV)
        tfp8.matmul_grouped(a, w, off, 128, torch.float32, out=buf[2:102])
        ct = tfp8.compress_t(x, offsets=off)
        tfp8.matmul_grouped_t(ct, ct, off, 100)
        torch.cuda.synchronize()
        assert (buf[:2] == 3).all() and (buf[102:] == 3).all()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("m,n,block", [(16, 16, 128), (130, 65, 128), (7, 200, 512)])
def test_matmul_grouped_t_matches_float64(counts, m, n, block, dt):
    say(f"matmul_grouped_t {len(counts)} groups, {sum(counts)} rows, {m}x{n} block {block} {dt}")
    rng = np.random.default_rng(n + m + len(counts))
    groups, rows, off = len(counts), sum(counts), offsets_of(counts)
    kp = padded_length(rows, groups, block)
    # random codes everywhere, also past the last group's end: those are not to be read as a group's
    a, b = random_operand(m, kp, block, rng), random_operand(n, kp, block, rng)
    av, bv = rotated_values(a, block), rotated_values(b, block)
    got = tfp8.matmul_grouped_t(to_gpu(a), to_gpu(b), torch.from_numpy(off).to(DEV), rows, block,
                                DTYPES[dt])
    at = 0
    for g, c in enumerate(counts):
        to = at + (c + block - 1) // block * block
        want = exact_product(av[:, at:to], bv[:, at:to])
        assert_product(got[g], want, to - at, f"{counts[:5]} group {g}")
        at = to


# ------------------------------------------------------------------------------------- gradients

def test_gradients_of_a_grouped_linear_layer_against_formula_and_differences():
    """dX = dY W and dW = dY^T X of y = x W^T by expert, from compressed operands, against the
    formulas on the decompressed values, and against differences of the float64 loss <dY, x W^T>."""
    say("gradients of a grouped linear layer")
    rng = np.random.default_rng(21)
    counts, n, k = [70, 0, 130, 5], 256, 384
    off, rows, groups = offsets_of(counts), sum(counts), len(counts)
    x = rng.standard_normal((rows, k)).astype(np.float32)
    w = (rng.standard_normal((groups, n, k)) * 0.05).astype(np.float32)
    dy = rng.standard_normal((rows, n)).astype(np.float32)
    gpu = lambda t: torch.from_numpy(t).to(DEV)
    og = gpu(off)
    xg, wg, dyg = gpu(x), gpu(w), gpu(dy)
    # dX: dY compressed along n, each expert's W^T compressed along n
    wt = [tfp8.compress_t(wg[g]) for g in range(groups)]
    wt = tuple(torch.stack(t) for t in zip(*wt))
    dyc = tfp8.compress(dyg)
    dx = tfp8.matmul_grouped(dyc, wt, og, dtype=torch.float32)
    # dW: both compressed along the tokens
    dyt, xt = tfp8.compress_t(dyg, offsets=og), tfp8.compress_t(xg, offsets=og)
    dw = tfp8.matmul_grouped_t(dyt, xt, og, rows)
    dec = lambda t: tfp8.decompress(*(u.contiguous() for u in t)).double().cpu().numpy()
    dyh, wth, dyth, xth = dec(dyc), dec(wt), dec(dyt), dec(xt)
    at = 0
    loss = lambda xx, ww, d: sum(float((d[lo:hi] * (xx[lo:hi] @ ww[g].T)).sum())
                                 for g, (lo, hi) in enumerate(zip(off, off[1:])))
    for g, (lo, hi) in enumerate(zip(off, off[1:])):
        to = at + (hi - lo + 127) // 128 * 128
        norm = lambda t: np.linalg.norm(t, axis=-1)
        mag = np.outer(norm(dyh[lo:hi]), norm(wth[g]))
        assert_product(dx[lo:hi], (dyh[lo:hi] @ wth[g].T, mag, mag), n + 256, f"dX {g}")
        mag = np.outer(norm(dyth[:, at:to]), norm(xth[:, at:to]))
        assert_product(dw[g], (dyth[:, at:to] @ xth[:, at:to].T, mag, mag), to - at + 256,
                       f"dW {g}")
        at = to
    # differences along random directions: the loss is linear in x and in w, so a central difference
    # is the exact directional derivative.  E4M3 rounds a value by 2.6% (root mean square: a step of
    # 2^-3, uniform, over a binade), so a product of two rounded operands is off by 3.7% of its norm,
    # and its part along a direction of independent normal values is normal with that deviation:
    # six of them
    for _ in range(4):
        v = rng.standard_normal(x.shape)
        d = (loss(x + 0.5 * v, w, dy) - loss(x - 0.5 * v, w, dy))
        got = float((dx.double().cpu().numpy() * v).sum())
        assert abs(got - d) <= 6 * 0.037 * np.linalg.norm(dx.cpu().numpy())
        v = rng.standard_normal(w.shape)
        d = (loss(x, w + 0.5 * v, dy) - loss(x, w - 0.5 * v, dy))
        got = float((dw.double().cpu().numpy() * v).sum())
        assert abs(got - d) <= 6 * 0.037 * np.linalg.norm(dw.cpu().numpy())


# --------------------------------------------------------------------------------------- refusals

def test_wrappers_refuse_bad_operands():
    rng = np.random.default_rng(1)
    a, b = to_gpu(random_operand(8, 512, 128, rng)), to_gpu(random_operand(9, 512, 128, rng))
    off = torch.tensor([0, 8], device=DEV)
    w = tuple(t.view(1, 9, -1) for t in b)
    cases = [
        (lambda: tfp8.matmul(a, b, 64), "block must be"),
        (lambda: tfp8.matmul(a, b, 128, torch.float16), "output dtype"),
        (lambda: tfp8.matmul((a[0][:, :500], a[1], a[2]), b), "multiple of the block"),
        (lambda: tfp8.matmul((a[0].view(torch.int8), a[1], a[2]), b), "codes of a must be"),
        (lambda: tfp8.matmul((a[0], a[1][:, :3], a[2]), b), "alpha of a must have"),
        (lambda: tfp8.matmul((a[0].cpu(), a[1], a[2]), b), "GPU tensors only"),
        (lambda: tfp8.matmul((a[0].t(), a[1], a[2]), b), "multiple of the block|contiguous"),
        (lambda: tfp8.matmul(a, (b[0][:, :256], b[1][:, :2], b[2][:, :2])), "512 and 256"),
        (lambda: tfp8.matmul(a, b, out=torch.empty(8, 8, device=DEV)), "out must be"),
        (lambda: tfp8.matmul_grouped(a, b, off), "3 dimensions"),
        (lambda: tfp8.matmul_grouped(a, w, off.int()), "int64"),
        (lambda: tfp8.matmul_grouped(a, w, torch.tensor([0, 4, 8], device=DEV)), "2 groups"),
        (lambda: tfp8.matmul_grouped(a, w, off.cpu()), "GPU tensors only"),
        (lambda: tfp8.matmul_grouped_t(a, b, off, 8), "128 elements a row"),
        (lambda: tfp8.compress_t(torch.zeros(4, 4)), "GPU tensors only"),
        (lambda: tfp8.compress_t(torch.zeros(4, device=DEV)), "must be"),
        (lambda: tfp8.compress_t(torch.zeros(4, 4, device=DEV).half()), "input dtype"),
        (lambda: tfp8.compress_t(torch.zeros(4, 4, device=DEV), 64), "block must be"),
        (lambda: tfp8.compress_t(torch.zeros(4, 6, device=DEV).t()), "contiguous"),
    ]
    for i, (call, text) in enumerate(cases):
        with pytest.raises(ValueError, match=text):
            call()
    with pytest.raises(tfp8.TFP8Error, match="TFP8_E_ARG"):
        tfp8.compress_t(torch.zeros(4, 4, device=DEV), flags=tfp8.FLAG_INT8)
    with pytest.raises(tfp8.TFP8Error, match="TFP8_E_ALIGN"):
        tfp8.matmul((torch.zeros(8 * 520, dtype=torch.uint8, device=DEV).view(8, 520)[:, :512],
                     a[1], a[2]), b)
    with pytest.raises(tfp8.TFP8Error, match="TFP8_E_ARG"):  # the output over an input
        codes = torch.zeros(512 * 512, dtype=torch.uint8, device=DEV).view(512, 512)
        s = torch.ones(512, 4, device=DEV)
        tfp8.matmul((codes, s, s), b, out=codes.view(-1).view(torch.bfloat16)[:512 * 9].view(512, 9))
