"""The layer of experts: arguments that are refused before anything runs (no GPU needed)."""
import pytest

from fp8_compression_tensor_amd import expert_layer


@pytest.mark.parametrize("steps,micro", [(0, 2), (-1, 1), (3, 0)])
def test_no_steps_are_refused(steps, micro):
    with pytest.raises(ValueError, match="at least one of each"):
        expert_layer.train(tokens=64, experts=2, width=128, steps=steps, micro=micro, rate=0.4)


@pytest.mark.parametrize("top_k", [0, -1, 4, 5])
def test_gated_experts_have_top_k_experts(top_k):
    import torch

    router, up, down = torch.zeros(3, 256), torch.zeros(3, 256, 256), torch.zeros(3, 256, 128)
    with pytest.raises(ValueError, match=r"top_k must be 1 to 3, got"):
        expert_layer.GatedExperts(router, up, down, top_k)
