"""The layer of experts where blocks of a row, or of the weights, are far apart in magnitude."""
import pytest
import torch

import fp8_compression_tensor_amd as tfp8
import moe_helpers as H
from test_gpu_moe import check, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def entered_by_block(x, b, rotate, exact):
    """moe_helpers.entered, where what float16 cuts off near zero hangs on the largest value of the block, not of
    the row."""
    r = H.rotated(x, b, rotate)
    blocks = lambda t: t.view(*t.shape[:-1], -1, b)
    rounded = 2.0 ** -22 if exact else 2.0 ** -12
    off = 11 * 2.0 ** -24 * blocks(r).norm(dim=-1, keepdim=True) \
        + 2.0 ** -33 * blocks(x).abs().amax(-1, keepdim=True)
    return r, rounded * r.abs() + off.expand(*off.shape[:-1], b).reshape(r.shape)


def far_weights(experts, k, f, b, gen, size, flags=0):
    """Weights of a layer whose first half of the places that are contracted over, 1 / size of the others; the
    last fourth of the experts have zeros there."""
    out = []
    for shape in ((experts, 2 * f, k), (experts, k, f)):
        w = torch.randn(*shape, device=DEV, generator=gen) * shape[-1] ** -0.5
        w[..., :max(shape[-1] // 2 // b, 1) * b] /= size
        w[-(-3 * experts // 4):, ..., :max(shape[-1] // 2 // b, 1) * b] = 0
        codes, alpha, scale = tfp8.compress(w, b, flags=flags)
        out.append((codes, alpha.view(*shape[:2], -1), scale.view(*shape[:2], -1)))
    return out


# one and two tokens of few and many experts (the choice and the rotation within the products, or not), half-height
# tiles, many tokens, several workgroups an expert
@pytest.mark.parametrize("tokens,experts,top_k,k,f,b", [
    (1, 8, 3, 512, 512, 128), (2, 70, 8, 512, 256, 128), (2, 8, 2, 4096, 512, 256), (1, 6, 2, 512, 16640, 128),
    (7, 9, 2, 1024, 1024, 512), (20, 5, 3, 384, 640, 128), (64, 40, 6, 512, 512, 256), (20, 5, 3, 256, 4096, 128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 50])
def test_large_blocks_beside_small_ones(tokens, experts, top_k, k, f, b, dtype, size, monkeypatch):
    """Where x is large the weights are small, or zero: the other blocks' part of the result is the larger one."""
    monkeypatch.setattr(H, "entered", entered_by_block)
    gen = torch.Generator(device=DEV).manual_seed(31)
    up, down = far_weights(experts, k, f, b, gen, size)
    x, router = inputs(tokens, experts, k, torch.float32, gen)
    x[:, :k // 2 // b * b] *= size
    router[:, :k // 2 // b * b] /= size
    got = tfp8.moe_layer(x, router, up, down, top_k, b, dtype=dtype)
    check(got, *H.layer(x, router, up, down, top_k, b, exact=dtype == torch.float32))


@pytest.mark.parametrize("flags", [0, tfp8.FLAG_NO_ROTATION])
def test_hidden_values_far_apart(flags, monkeypatch):
    """Rows of W3 2^40 apart, and columns of W2 that take it back."""
    monkeypatch.setattr(H, "entered", entered_by_block)
    gen = torch.Generator(device=DEV).manual_seed(32)
    experts, k, f, b = 6, 256, 512, 128
    w1 = torch.randn(experts, 2 * f, k, device=DEV, generator=gen) * k ** -0.5
    w2 = torch.randn(experts, k, f, device=DEV, generator=gen) * f ** -0.5
    w1[:, f + b:f + 2 * b] *= 2.0 ** 40
    w2[:, :, b:2 * b] *= 2.0 ** -40
    w2[:3, :, b:2 * b] = 0
    up, down = (tfp8.compress(w, b, flags=flags) for w in (w1, w2))
    for tokens in (1, 12):
        x, router = inputs(tokens, experts, k, torch.bfloat16, gen)
        got = tfp8.moe_layer(x, router, up, down, 2, b, dtype=torch.float32, flags=flags)
        check(got, *H.layer(x, router, up, down, 2, b, rotate=not flags))
