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
