"""Calls of the layer of experts beside a plain training step."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def layer():
    from fp8_compression_tensor_amd import expert_layer

    return expert_layer


def test_second_derivatives_are_refused():
    """A gradient penalty: its terms through the layer must not go missing beside those that do not."""
    L = layer()
    print("expert layer, second derivative", flush=True)
    x = torch.randn(200, 128, device="cuda", requires_grad=True)
    w = (torch.randn(2, 128, 128, device="cuda") * 0.1).requires_grad_()
    off = torch.tensor([0, 120, 200], device="cuda")
    y = L.expert_linear(x, w, L.CompressedWeights(w), off)
    (g,) = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (g.square().sum() + x.square().sum()).backward()


def test_the_time_of_a_step_is_of_steps_that_ran():
    print("expert layer, one step and two", flush=True)
    one = layer().train(tokens=256, experts=2, width=128, steps=1, micro=1, rate=0.4)
    assert one["ms_per_step"] is None and one["loss_first"] == one["loss_last"]
    two = layer().train(tokens=256, experts=2, width=128, steps=2, micro=1, rate=0.4)
    assert 0 < two["ms_per_step"] < 10e3  # of one step, not a clock's reading
