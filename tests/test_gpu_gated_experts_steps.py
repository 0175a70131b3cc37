"""GatedExperts' steps: which of them count, and what they do to the parameters."""
import pytest
import torch

import fp8_compression_tensor_amd as tfp8
from test_gpu_gated_experts import layer
from test_gpu_optimizer import check_step

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


@pytest.mark.parametrize("bits", [8, 32])
def test_steps_are_adamws(bits):
    """Parameters, states and codes after the steps of a layer that follows another one: AdamW's, in float64,
    from the gradients of two micro-batches, the experts' added up in codes, and clipped."""
    print("gated experts, steps against the formula", bits, flush=True)
    (L, gen), (teacher, _) = layer(bits=bits), layer(seed=1)
    clipped = 0
    for step in (1, 2, 3):
        main = None
        for _ in range(2):
            x = torch.randn(200, 256, device=DEV, generator=gen).to(torch.bfloat16)
            with torch.no_grad():
                want = teacher(x)
            (L(x) - want).float().square().mean().backward()
            grads = [p.grad for p in L.params]
            for p in L.params:
                p.grad = None
            if main is None:
                main = [grads[0], *(tfp8.compress(g) for g in grads[1:])]
            else:
                main[0] += grads[0]
                for m, g in zip(main[1:], grads[1:]):
                    tfp8.accumulate(*m, g, inplace=True)
        before = [p.detach().flatten().clone() for p in L.params]
        old = tuple(t.clone() for t in L.state)
        most = 0.05 if step < 3 else 1e3
        c = float(tfp8.grad_norm(main, most)[1])
        clipped += c < 1
        L.step(main, 2e-3, most, 0.1)
        flat = [main[0].flatten(), *main[1:]]
        codes = [None, *((c.flatten(), a.flatten(), s.flatten()) for c, a, s in L.rows)]
        check_step([p.detach().flatten() for p in L.params], before, flat, old, L.state, codes, 128, step,
                   c=c, lr=2e-3)
    assert clipped == 2 and int(L.steps) == 3
