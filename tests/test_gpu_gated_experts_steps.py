"""GatedExperts' steps: which of them count."""
import pytest
import torch

from test_gpu_gated_experts import layer

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_step_that_is_left_out_does_not_count(bits, bad):
    """A layer whose first, and third, step was left out goes on as one that never saw them."""
    print("gated experts, steps left out", bits, bad, flush=True)
    (L, gen), (twin, _) = layer(bits=bits), layer(bits=bits)
    for i in range(4):
        grads = [0.1 * torch.randn(p.shape, device=DEV, generator=gen) for p in L.params]
        if i % 2 == 0:
            broken = [g.clone() for g in grads]
            broken[1][2, 3, 4] = bad
            assert not torch.isfinite(L.step(broken, 1e-2))
        L.step(grads, 1e-2)
        twin.step(grads, 1e-2)
        for a, b in zip(L.params, twin.params):
            assert torch.equal(a, b), i
        for a, b in zip([*L.state, *L.rows[0], *L.rows[1]], [*twin.state, *twin.rows[0], *twin.rows[1]]):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("top_k", [1, 3])
def test_no_tokens(top_k):
    """Outputs and gradients of no tokens at all."""
    print("gated experts, no tokens", top_k, flush=True)
    L, gen = layer(top_k=top_k)
    x = torch.randn(0, 256, device=DEV, generator=gen).to(torch.bfloat16).requires_grad_()
    y = L(x)
    assert y.shape == (0, 256) and y.dtype == x.dtype
    y.float().sum().backward()
    assert x.grad.shape == (0, 256)
    for p in L.params:
        assert p.grad is not None and not p.grad.any()
    with torch.no_grad():
        assert L.answer(x).shape == (0, 256)
