"""Cases that time the products of compressed tensors and the transposed compress.

Four operators, in the framework's own format (E4M3 codes with a float32 pair alpha, scale for each
block of `block` elements along the contraction):

  matmul            A[M, K] B[N, K]^T of two compressed operands
  compress_t        compress of x^T: blocks along the rows of x, ragged by group where it has groups
  matmul_grouped    rows sorted by expert, each expert's rows times that expert's weights
  matmul_grouped_t  the experts' weight gradients: the contraction runs over each expert's own rows

With `own` False, `run` computes them from elementary torch operations in float32; with `own` True
it calls the package.
"""
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a decoded sequence through a square projection: bound by latency
        {"name": "matmul_one_token", "op": "matmul", "m": 1, "n": 4096, "k": 4096, "block": 128,
         "dtype": "bf16"},
        # a small batch of decoded tokens through an up projection: the weights' bytes
        {"name": "matmul_24_tokens", "op": "matmul", "m": 24, "n": 10240, "k": 5120, "block": 128,
         "dtype": "bf16"},
        # a ragged batch and an odd number of outputs (a head with a vocabulary that is no
        # multiple of anything), float32 logits
        {"name": "matmul_odd_f32", "op": "matmul", "m": 1003, "n": 2571, "k": 2560, "block": 128,
         "dtype": "f32"},
        # the forward product of a training step on [4, 2048, 4096] activations, block 256
        {"name": "matmul_train", "op": "matmul", "m": 8192, "n": 16384, "k": 4096, "block": 256,
         "dtype": "bf16"},
        # a small float32 gradient whose rows are no multiple of the block
        {"name": "compress_t_small_f32", "op": "compress_t", "m": 517, "n": 640, "groups": 1,
         "block": 128, "dtype": "f32"},
        # a [4, 4096, 5120] bf16 gradient, for the weight gradient's product
        {"name": "compress_t_grad", "op": "compress_t", "m": 16384, "n": 5120, "groups": 1,
         "block": 128, "dtype": "bf16"},
        # the same for tokens routed to 16 experts
        {"name": "compress_t_ragged", "op": "compress_t", "m": 8192, "n": 3584, "groups": 16,
         "block": 128, "dtype": "bf16"},
        # decoding with experts: a few rows each, every expert's weights are read
        {"name": "grouped_decode", "op": "matmul_grouped", "m": 48, "groups": 16, "n": 2560,
         "k": 4096, "block": 128, "dtype": "bf16"},
        # many small experts, some of them empty, an odd width
        {"name": "grouped_odd_f32", "op": "matmul_grouped", "m": 3001, "groups": 24, "n": 1001,
         "k": 1280, "block": 128, "dtype": "f32"},
        # the experts' forward product of a training step
        {"name": "grouped_train", "op": "matmul_grouped", "m": 16384, "groups": 8, "n": 5120,
         "k": 4096, "block": 128, "dtype": "bf16"},
        # small experts' weight gradients
        {"name": "grouped_t_small", "op": "matmul_grouped_t", "m": 700, "groups": 16, "n": 512,
         "k": 640, "block": 128, "dtype": "bf16"},
        # the experts' weight gradients of a training step
        {"name": "grouped_t_train", "op": "matmul_grouped_t", "m": 16384, "groups": 8, "n": 4096,
         "k": 2560, "block": 128, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["matmul", "compress_t", "matmul_grouped", "matmul_grouped_t"])
    block = rng.choice([128, 128, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    while True:
        if op == "matmul":
            c = {"m": _log(rng, 1, 16384), "n": _log(rng, 64, 16384),
                 "k": block * _log(rng, 1, 5120 // block)}
            cost = 2 * c["m"] * c["n"] * c["k"]
        elif op == "compress_t":
            c = {"m": _log(rng, 64, 16384), "n": _log(rng, 64, 5120), "groups": rng.choice([1, 1, 4, 16])}
            cost = 0
        else:
            c = {"m": _log(rng, 16, 16384), "groups": _log(rng, 2, 32), "n": _log(rng, 64, 5120),
                 "k": _log(rng, 64, 5120)}
            if op == "matmul_grouped":
                c["k"] = block * max(1, c["k"] // block)
            cost = 2 * c["m"] * c["n"] * c["k"]
            if c["groups"] * c["n"] * c["k"] > 16 * 2560 * 4096:  # weights, or their gradients
                continue
        if 3072 in c.values() or cost > 2 * 8192 * 16384 * 4096:
            continue
        return {"op": op, **c, "block": block, "dtype": dtype}


def _padded_rows(m, groups, block):
    """Length of a compressed row of x^T: room for every group's rows rounded up to a block."""
    return (m + groups * (block - 1)) // block * block


def _shares(groups):
    """The share of the tokens each expert gets: uneven, as routers trained to balance still are."""
    w = [(1.0 + e) ** -0.3 for e in range(groups)]
    return [x / sum(w) for x in w]


def work(case):
    op, m, n, b = case["op"], case["m"], case["n"], case["block"]
    elt = 2 if case["dtype"] == "bf16" else 4
    code = 1 + 8 / b  # a code and its part of the two scales
    g = case.get("groups", 1)
    if op == "compress_t":
        kp = m if g == 1 else m + g * (b - 1) / 2  # rows, and the padding that groups need
        return {"bytes": m * n * elt + n * kp * code, "flops": n * m * (b.bit_length() + 6)}
    k = case["k"]
    if op == "matmul":
        return {"bytes": (m + n) * k * code + m * n * elt, "flops": 2 * m * n * k}
    if op == "matmul_grouped":
        hit = sum(1 - (1 - p) ** m for p in _shares(g))  # experts that have a row
        return {"bytes": m * k * code + hit * n * k * code + m * n * elt, "flops": 2 * m * n * k}
    return {"bytes": (n + k) * m * code + g * n * k * elt, "flops": 2 * m * n * k}


# ------------------------------------------------------------------------------------ the inputs

def _hadamard(b, dtype):
    i = torch.arange(b, device=DEV)
    bits = (i[:, None] & i[None, :])[..., None] >> torch.arange(9, device=DEV) & 1
    return (1 - 2 * (bits.sum(-1) & 1)).to(dtype)


def _compress_rows(x, h):
    """[R, C] float32 -> codes uint8 [R, C], alpha and scale float32 [R, C / b] (target 1); h is
    the [b, b] orthogonal Hadamard matrix."""
    v = x.reshape(x.shape[0], -1, h.shape[0])
    m2 = (v * v).mean(-1)
    alpha = torch.where(m2 > 0, m2.clamp_min(2.0 ** -126).rsqrt().clamp(2.0 ** -126, 2.0 ** 126),
                        torch.ones_like(m2))
    y = torch.matmul(v * alpha[..., None], h)
    s = y.abs().amax(-1) / 448
    q = (y / torch.where(s > 0, s, torch.ones_like(s))[..., None]).to(torch.float8_e4m3fn)
    return q.reshape(x.shape).view(torch.uint8), alpha, s


def _activations(r, c, gen):
    """Most values near zero, a few wide channels, some outliers, and padding rows of zeros."""
    x = torch.randn(r, c, device=DEV, generator=gen)
    x *= torch.exp(0.7 * torch.randn(c, device=DEV, generator=gen))
    x[torch.rand(r, c, device=DEV, generator=gen) < 2e-4] *= 30
    if r > 8:
        x[torch.rand(r, device=DEV, generator=gen) < 0.01] = 0
    return x


def _weights(r, c, gen):
    return 0.02 * torch.randn(r, c, device=DEV, generator=gen)


def _offsets(m, groups, gen):
    p = torch.tensor(_shares(groups), device=DEV)
    e = torch.multinomial(p, m, replacement=True, generator=gen)
    counts = torch.bincount(e, minlength=groups)
    return torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), counts.cumsum(0)])


def _source_rows(offsets, m, kp, b):
    """For each position of a padded row: the row of x it holds, and whether it holds one."""
    counts = offsets[1:] - offsets[:-1]
    end = ((counts + b - 1) // b * b).cumsum(0)
    start = end - (counts + b - 1) // b * b
    j = torch.arange(kp, device=DEV)
    e = torch.searchsorted(end, j, right=True)
    held = e < counts.numel()
    e = e.clamp_max(counts.numel() - 1)
    src = offsets[e] + j - start[e]
    return src.clamp(0, m - 1), held & (src < offsets[e + 1])


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, m, n, b = case["op"], case["m"], case["n"], case["block"]
    g = case.get("groups", 1)
    h = _hadamard(b, torch.float32) * b ** -0.5
    s = {"op": op, "block": b, "m": m, "groups": g,
         "dtype": torch.bfloat16 if case["dtype"] == "bf16" else torch.float32}
    if op == "compress_t":
        s["h"] = h
        s["x"] = _activations(m, n, gen).to(s["dtype"])
        s["offsets"] = _offsets(m, g, gen) if g > 1 else None
        return s
    k = case["k"]
    if op == "matmul":
        s["a"] = _compress_rows(_activations(m, k, gen), h)
        s["b"] = _compress_rows(_weights(n, k, gen), h)
        return s
    s["offsets"] = _offsets(m, g, gen)
    s["longest"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())  # the largest expert's rows
    if op == "matmul_grouped":
        s["a"] = _compress_rows(_activations(m, k, gen), h)
        codes, alpha, scale = _compress_rows(_weights(g * n, k, gen), h)
        s["b"] = (codes.view(g, n, k), alpha.view(g, n, -1), scale.view(g, n, -1))
        return s
    kp = _padded_rows(m, g, b)
    src, held = _source_rows(s["offsets"], m, kp, b)
    for name, c in (("a", n), ("b", k)):  # dY and X, compressed along the tokens
        x = _activations(m, c, gen)
        s[name] = _compress_rows((x[src] * held[:, None]).t().contiguous(), h)
    return s


# --------------------------------------------------------------------- the operators, plain form

def _values(t, b):
    """The values a compressed operand stands for, in the rotated basis, in float32: the rotation is
    orthogonal, so a product over whole blocks is the same there."""
    codes, alpha, scale = t
    v = codes.view(torch.float8_e4m3fn).to(torch.float32)
    v = v.view(*codes.shape[:-1], -1, b) * (scale / alpha)[..., None]
    return v.view(codes.shape)


def _plain_compress_t(s):
    x, b = s["x"], s["block"]
    kp = _padded_rows(s["m"], s["groups"], b)
    if s["offsets"] is None:
        xt = torch.zeros(x.shape[1], kp, device=DEV)
        xt[:, : x.shape[0]] = x.t()
    else:
        src, held = _source_rows(s["offsets"], s["m"], kp, b)
        xt = (x[src].to(torch.float32) * held[:, None]).t()
    codes, alpha, scale = _compress_rows(xt, s["h"])
    return {"codes": codes.view(torch.float8_e4m3fn), "alpha": alpha, "scale": scale}


def _plain_grouped(s):
    """Every expert's rows in a slab as long as the longest one's: one batched product, no loop."""
    a, w, off = _values(s["a"], s["block"]), _values(s["b"], s["block"]), s["offsets"]
    at = off[:-1, None] + torch.arange(s["longest"], device=DEV)
    slab = a[at.clamp_max(s["m"] - 1)] * (at < off[1:, None])[..., None]
    out = torch.bmm(slab, w.transpose(1, 2))
    row = torch.arange(s["m"], device=DEV)
    e = torch.searchsorted(off[1:].contiguous(), row, right=True)
    return out[e, row - off[e]].to(s["dtype"])


def _plain_grouped_t(s):
    b, off = s["block"], s["offsets"]
    counts = (off[1:] - off[:-1] + b - 1) // b * b
    end = counts.cumsum(0)
    at = (end - counts)[:, None] + torch.arange((s["longest"] + b - 1) // b * b, device=DEV)
    held = at < end[:, None]
    at = at.clamp_max(s["a"][0].shape[1] - 1)
    x = _values(s["a"], b)[:, at] * held
    y = _values(s["b"], b)[:, at] * held
    return torch.bmm(x.permute(1, 0, 2), y.permute(1, 2, 0)).to(s["dtype"])


def run(state):
    s, op, b = state, state["op"], state["block"]
    if own:
        import fp8_compression_tensor_amd as tfp8

        if op == "compress_t":
            codes, alpha, scale = tfp8.compress_t(s["x"], b, 1.0, offsets=s["offsets"])
            return {"codes": codes.view(torch.float8_e4m3fn), "alpha": alpha, "scale": scale}
        if op == "matmul":
            return tfp8.matmul(s["a"], s["b"], b, s["dtype"])
        if op == "matmul_grouped":
            return tfp8.matmul_grouped(s["a"], s["b"], s["offsets"], b, s["dtype"])
        return tfp8.matmul_grouped_t(s["a"], s["b"], s["offsets"], s["m"], b, s["dtype"])
    if op == "compress_t":
        return _plain_compress_t(s)
    if op == "matmul":
        return torch.matmul(_values(s["a"], b), _values(s["b"], b).t()).to(s["dtype"])
    return _plain_grouped(s) if op == "matmul_grouped" else _plain_grouped_t(s)


# -------------------------------------------------------------------------- the same, in 64 bits

def _e4m3_table():
    """The values of the OCP E4M3 codes, from its definition (127 and 255, its NaN, never occur)."""
    c = torch.arange(256, dtype=torch.float64, device=DEV)
    e, f = torch.floor(c / 8) % 16, c % 8
    v = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * 2.0 ** (e - 10))
    return torch.where(c < 128, v, -v)


def _reconstruct(t, b):
    """x^ = H (s dec q) / (sqrt(b) alpha), block by block."""
    codes, alpha, scale = t
    v = _e4m3_table()[codes.to(torch.int64)].view(*codes.shape[:-1], -1, b)
    v = torch.matmul(v * scale.double()[..., None], _hadamard(b, torch.float64)) / b ** 0.5
    return (v / alpha.double()[..., None]).view(codes.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op, b = s["op"], s["block"]
    if op == "matmul":
        return torch.matmul(_reconstruct(s["a"], b), _reconstruct(s["b"], b).t())
    off = [0, s["m"]] if s["offsets"] is None else s["offsets"].tolist()
    if op == "compress_t":
        x = s["x"].double()
        n, kp = x.shape[1], _padded_rows(s["m"], s["groups"], b)
        xt = torch.zeros(n, kp, dtype=torch.float64, device=DEV)
        at = 0
        for lo, hi in zip(off, off[1:]):
            xt[:, at:at + hi - lo] = x[lo:hi].t()
            at += (hi - lo + b - 1) // b * b
        v = xt.view(n, -1, b)
        empty = (v == 0).all(-1)
        alpha = torch.where(empty, 1.0, (v * v).mean(-1).rsqrt().clamp(2.0 ** -126, 2.0 ** 126))
        y = torch.matmul(v * alpha[..., None], _hadamard(b, torch.float64)) / b ** 0.5
        scale = y.abs().amax(-1) / 448
        q = y / torch.where(empty, 1.0, scale)[..., None]  # before it is rounded to a code
        return {"codes": q.view(n, kp), "alpha": alpha, "scale": scale}
    x, y = _reconstruct(s["a"], b), s["b"]
    out, at = [], 0
    for e, (lo, hi) in enumerate(zip(off, off[1:])):
        if op == "matmul_grouped":
            out.append(torch.matmul(x[lo:hi], _reconstruct(tuple(t[e] for t in y), b).t()))
        else:
            to = at + (hi - lo + b - 1) // b * b
            part = tuple(t[:, at // d:to // d].contiguous() for t, d in zip(y, (1, b, b)))
            out.append(torch.matmul(x[:, at:to], _reconstruct(part, b).t()))
            at = to
    return torch.cat(out) if op == "matmul_grouped" else torch.stack(out)
