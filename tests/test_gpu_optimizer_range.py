"""The AdamW step where second moments, or their squares, leave float32's normal range."""
import pytest
import torch

import fp8_compression_tensor_amd as tfp8
import optimizer_helpers as H

pytestmark = pytest.mark.gpu
DEV = "cuda"
BETAS, B = (0.9, 0.99), 128


def formula(g, m, v, eps, step, dv_least, dg):
    """(u, m', v') of a step of lr 1 from p = 0, p' = -u, in float64, and how far float32's may be from each.

    m' takes 6 roundings of its terms, v' 10, and no less than dv_least where it is subnormal; a gradient
    that is off by dg times itself adds to both.  The root's is half of v's relative one, or its root, and a
    step (2 roundings); its factor, eps' sum and 6 roundings of the quotient follow."""
    b1, b2 = BETAS
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    dm = 6 * H.EPS * (abs(b1 * m) + abs((1 - b1) * g)) + dg * (1 - b1) * abs(g) + 2.0 ** -148
    dv = 10 * H.EPS * v1 + 2.1 * dg * (1 - b2) * g * g + dv_least
    root = v1.sqrt()
    droot = torch.where(root > 0, torch.minimum(dv.sqrt(), dv / root.clamp_min(1e-300)), dv.sqrt())
    droot = droot + 2 * H.EPS * root + 2.0 ** -148
    den = root / (1 - b2 ** step) ** 0.5 + eps
    low = (den - droot / (1 - b2 ** step) ** 0.5 - 3 * H.EPS * den).clamp_min(eps * (1 - 2 * H.EPS))
    rate = 1 / (1 - b1 ** step)
    u = rate * m1 / den
    du = rate * (dm / low + abs(m1) * (1 / low - 1 / den)) + 8 * H.EPS * abs(u)
    return (u, m1, root, v1), (du, dm, droot, dv)


def gradients(size, kind, gen, n=8 * B):
    g = size * (0.5 + torch.rand(n, device=DEV, generator=gen))
    g = torch.where(torch.rand(n, device=DEV, generator=gen) < 0.5, g, -g)
    g[torch.rand(n, device=DEV, generator=gen) < 0.1] = 0
    return tfp8.compress(g, B) if kind == "codes" else g


@pytest.mark.parametrize("kind", ["f32", "codes"])
@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -63, 2.0 ** -66, 2.0 ** -70])
def test_subnormal_second_moments(size, kind):
    """In 32 bits: v' below 2^-126 keeps the bits that float32 has there, and the step takes them."""
    gen = torch.Generator(device=DEV).manual_seed(21)
    p = torch.zeros(8 * B, device=DEV)
    state = tfp8.adamw_state([p], 32, B)
    eps = 2.0 ** -72
    for step in (1, 2, 3):
        g = gradients(size, kind, gen)
        m, v = H.state_values(state, B)
        p.zero_()
        tfp8.adamw([p], [g], state, 1.0, BETAS, eps, 0.0, step, block=B)
        g, dg = (H.reconstruct(g, B), 5 * H.EPS) if kind == "codes" else (g.double().cpu(), 0.0)
        # two roundings of half a unit, 2^-150, each
        (u, m1, _, v1), (du, dm, _, dv) = formula(g, m, v, eps, step, 2.0 ** -149, dg)
        assert (abs(state[0].double().cpu() - m1) <= dm).all()
        assert (abs(state[1].double().cpu() - v1) <= dv).all()
        assert (abs(p.double().cpu() + u) <= du).all(), float((abs(p.double().cpu() + u) / du).max())


@pytest.mark.parametrize("size,kind", [
    (2.0 ** -118, "f32"), (2.0 ** -90, "f32"), (2.0 ** -90, "codes"), (2.0 ** -70, "f32"),
    (2.0 ** -62, "codes"), (2.0 ** -50, "f32"), (1.0, "codes"), (2.0 ** 62, "f32"), (2.0 ** 66, "f32"),
    (2.0 ** 70, "codes"), (2.0 ** 98, "codes"), (2.0 ** 118, "f32")])
def test_roots_far_from_one(size, kind):
    """In 8 bits the state is the root, whose square may lie outside of float32's range: the root does not."""
    gen = torch.Generator(device=DEV).manual_seed(22)
    p = torch.zeros(8 * B, device=DEV)
    state = tfp8.adamw_state([p], 8, B)
    eps = max(2.0 ** -126, size * 2.0 ** -12)
    for step in (1, 2, 3):
        g = gradients(size, kind, gen)
        m, v = H.state_values(state, B)
        p.zero_()
        tfp8.adamw([p], [g], state, 1.0, BETAS, eps, 0.0, step, block=B, seed=5)
        g, dg = (H.reconstruct(g, B), 5 * H.EPS) if kind == "codes" else (g.double().cpu(), 0.0)
        (u, m1, root, _), (du, dm, droot, _) = formula(g, m, v, eps, step, 0.0, dg)
        assert (abs(p.double().cpu() + u) <= du).all(), float((abs(p.double().cpu() + u) / du).max())
        if size < 2.0 ** -98:  # moments below 2^-100 are stored as zeros
            assert not any(t.any() for t in H.state_values(state, B))  # (0x80 is a zero, too)
            continue
        r = H.random_bits(5, step, 0, len(g))
        half = lambda bits: (bits.double() + 0.5) / 65536
        H.check_codes(state[0], state[1].cpu(), m1, dm, half(r & 0xFFFF), B, False)
        H.check_codes(state[2], state[3].cpu(), root, droot, half(r >> 16), B, True)


@pytest.mark.parametrize("size", [2.0 ** 66, 2.0 ** 110])
def test_a_huge_gradient_leaves_its_neighbours(size):
    """A finite gradient whose square is past float32: states of its block stay finite, and the next step is
    the formula's from what they hold."""
    gen = torch.Generator(device=DEV).manual_seed(23)
    p = torch.zeros(8 * B, device=DEV)
    state = tfp8.adamw_state([p], 8, B)
    for step in (1, 2, 3):
        g = gradients(1.0, "f32", gen)
        if step == 1:
            g[3 * B + 5] = size
        m, v = H.state_values(state, B)
        assert torch.isfinite(m).all() and torch.isfinite(v).all()
        p.zero_()
        tfp8.adamw([p], [g], state, 1.0, BETAS, 1e-8, 0.0, step, block=B)
        (u, *_), (du, *_) = formula(g.double().cpu(), m, v, 1e-8, step, 0.0, 0.0)
        assert (abs(p.double().cpu() + u) <= du).all(), float((abs(p.double().cpu() + u) / du).max())
    assert all(torch.isfinite(t).all() for t in (state[1], state[3]))
