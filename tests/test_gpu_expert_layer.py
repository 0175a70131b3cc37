"""The layer of experts on compressed operands: its gradients and a few steps of training."""
import pytest
import torch

pytestmark = pytest.mark.gpu

# E4M3 rounds a value by 2.6% (root mean square), so a product of two rounded operands is off by
# sqrt(2) * 2.6% = 3.7% of its norm; bfloat16 outputs add 0.2%.  A gradient that comes from one rounded
# product (dx, dw) is held to 5%.
REL = 0.05


def layer():
    from fp8_compression_tensor_amd import expert_layer

    return expert_layer


@pytest.mark.parametrize("counts", [[100, 0, 300, 1], [0, 0, 77], [513]])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gradients_follow_the_uncompressed_layer(counts, dtype):
    L = layer()
    print("expert layer gradients", counts, dtype, flush=True)
    n, k, experts, rows = 256, 384, len(counts), sum(counts)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, k, device="cuda", generator=gen).to(dtype).requires_grad_()
    w = (torch.randn(experts, n, k, device="cuda", generator=gen) * 0.05).requires_grad_()
    off = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), device="cuda")
    y = L.expert_linear(x, w, L.CompressedWeights(w), off)
    dy = torch.randn(rows, n, device="cuda", generator=gen).to(dtype)
    y.backward(dy)
    want = torch.cat([x[lo:hi].detach().float() @ w[e].detach().t()
                      for e, (lo, hi) in enumerate(zip(off[:-1], off[1:]))])
    dx, dw = L.plain_gradients(x.detach(), w.detach(), dy, off)
    rel = lambda a, b: float((a.float() - b).norm() / b.norm())
    assert y.dtype == dtype and x.grad.dtype == dtype and w.grad.dtype == torch.float32
    assert rel(y.detach(), want) < REL and rel(x.grad, dx) < REL and rel(w.grad, dw) < REL
    for e, c in enumerate(counts):
        if c == 0:
            assert not w.grad[e].any()


def test_training_follows_the_teacher():
    print("expert layer training", flush=True)
    r = layer().train(tokens=512, experts=4, width=256, steps=8, micro=2, rate=0.4)
    assert r["loss_last"] < 0.2 * r["loss_first"], r
    assert r["dw_rel_l2"] < REL and r["dx_rel_l2"] < REL and r["logits"] == [1, 256], r


def test_sizes_that_are_no_whole_blocks_are_refused():
    L = layer()
    with pytest.raises(ValueError, match="block size"):
        L.CompressedWeights(torch.zeros(2, 128, 200, device="cuda"))
