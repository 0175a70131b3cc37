"""Refusals of the layer of experts' C call: before any HIP call, so they run without a GPU."""
import pytest

import fp8_compression_tensor_amd as tfp8

F = 0x7F0000000000  # an aligned address that is never dereferenced here
G = 1 << 34


def call(x=F, xd=0, ldx=256, router=F + G, rd=0, up=(F + 2 * G, F + 3 * G, F + 4 * G),
         down=(F + 5 * G, F + 6 * G, F + 7 * G), tokens=5, experts=8, top_k=2, k=256, f=512, block=128,
         flags=0, ws=F + 8 * G, nbytes=1 << 30, out=F + 9 * G, od=0, ldo=256):
    return tfp8.moe_layer_raw((x, xd, ldx), (router, rd), up, down, tokens, experts, top_k, k, f, block,
                              flags, ws, nbytes, (out, od, ldo))


def test_sizes():
    for block in (0, 64, 96, 1024):
        assert call(block=block) == -3
    for bad in (dict(tokens=-1), dict(tokens=65), dict(experts=0), dict(experts=513), dict(top_k=0),
                dict(top_k=9), dict(k=0), dict(k=200), dict(f=0), dict(f=500), dict(block=512),
                dict(k=(1 << 20) + 128, ldx=1 << 21, ldo=1 << 21), dict(f=(1 << 20) + 128),
                dict(tokens=64, experts=512, top_k=512, f=1 << 15), dict(ldx=1 << 35), dict(ldo=1 << 35)):
        assert call(**bad) == -2, bad
    assert call(ldx=255) == -6 and call(ldo=255) == -6
    assert call(tokens=0, x=None, out=None, ws=None) == 0


def test_types_flags_and_pointers():
    assert call(xd=2) == -4 and call(rd=-1) == -4 and call(od=3) == -4
    assert call(flags=1) == -6 and call(flags=8) == -6
    for name in ("x", "router", "ws", "out"):
        assert call(**{name: None}) == -1
    for name, at in (("up", F + 2 * G), ("down", F + 5 * G)):
        for i in range(3):
            three = [at, at + G, at + 2 * G]
            three[i] = None
            assert call(**{name: tuple(three)}) == -1
            three[i] = at + i * G + (8 if i == 0 else 2)
            assert call(**{name: tuple(three)}) == -5
    assert call(x=F + 1) == -5 and call(x=F + 2, xd=1) == -5 and call(out=F + 9 * G + 1) == -5
    assert call(ws=F + 8 * G + 8) == -5 and call(router=F + G + 1) == -5


def test_workspace_and_overlaps():
    need = tfp8.lib().tfp8_moe_workspace(5, 8, 2, 256, 512)
    assert need > 0 and call(nbytes=need - 1) == -2
    assert tfp8.lib().tfp8_moe_workspace(65, 8, 2, 256, 512) == 0
    for at in (F, F + G, F + 2 * G, F + 3 * G, F + 5 * G, F + 7 * G):
        assert call(out=at) == -6 and call(ws=at) == -6
    assert call(out=F + 8 * G + need - 16) == -6  # over the workspace


def test_most_hidden_values():
    """2^29 of them would take a launch of 2^32 threads."""
    assert call(tokens=64, experts=512, top_k=512, f=1 << 14, nbytes=1 << 40) == -2
    assert tfp8.lib().tfp8_moe_workspace(64, 512, 512, 256, 1 << 14) == 0
    assert tfp8.lib().tfp8_moe_workspace(64, 512, 512, 256, (1 << 14) - 128) > 0


def test_flags_of_the_wrapper():
    """Only FLAG_NO_ROTATION: the C call's bit for the softmax of all is renormalize's."""
    import torch

    x = torch.zeros(1, 128)
    for flags in (4, 4 | tfp8.FLAG_NO_ROTATION, tfp8.FLAG_INT8, 8, -1):
        with pytest.raises(tfp8.TFP8Error, match="TFP8_E_ARG"):
            tfp8.moe_layer(x, x, (), (), 1, flags=flags)
    with pytest.raises(ValueError, match="GPU"):
        tfp8.moe_layer(x, x, (), (), 1, flags=tfp8.FLAG_NO_ROTATION)
