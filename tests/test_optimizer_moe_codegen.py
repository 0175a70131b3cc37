"""The generated gfx950 code of the optimizer's step and of the layer of experts (hipcc, no GPU needed): no packed
float32 arithmetic, no scratch memory, the wait states that the inline asm needs, and registers that
let in the wavefronts which the launches count on."""
import os
import re
import shutil
import subprocess

import pytest

from test_codegen_hazards import _parse, _regs, _states
from test_products_codegen import CSRC, flags
from test_products_codegen_bodies import bodies_of

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not available")


@pytest.fixture(scope="module", params=["tfp8_optimizer.hip", "tfp8_moe.hip"])
def kernels(request, tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "k.s")
    r = subprocess.run(["hipcc", *flags(), "--cuda-device-only", "-S", "-o", out,
                        os.path.join(CSRC, request.param)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(out).read()
    return request.param, bodies_of(text), text


def test_every_kernel_was_found(kernels):
    name, bodies, text = kernels
    want = (["k_norm", "k_norm_finish", "k_adamw", "k_adamw_factors"] if "optimizer" in name else
            ["k_moe_scores", "k_moe_plan", "k_moe_up", "k_moe_rotate", "k_moe_down", "k_moe_join"])
    assert all(any(w in b for b in bodies) for w in want)
    assert len(bodies) == len(re.findall(r"^\s*\.amdhsa_kernel ", text, re.M))


def test_no_packed_float32_and_no_scratch_memory(kernels):
    name, bodies, text = kernels
    for kernel, code in bodies.items():
        assert not [l for l in code if re.match(r"v_pk_(add|mul|fma)_f32", l)], kernel
    sizes = re.findall(r"\.amdhsa_private_segment_fixed_size (\d+)", text)
    assert len(sizes) == len(bodies) and not any(map(int, sizes))


def test_dpp_sources_are_not_written_in_the_two_states_before(kernels):
    bad, checked = [], 0
    for name, body in kernels[1].items():
        parsed = [_parse(i) for i in body if not i.endswith(":")]
        for i, (op, ops) in enumerate(parsed):
            if "_dpp" not in op or len(ops) < 2:
                continue
            checked += 1
            src, waited = _regs(ops[1]), 0
            for pop, pops in reversed(parsed[max(0, i - 4):i]):
                if pop.startswith("v_") and pops and _regs(pops[0]) & src:
                    if waited < 2:
                        bad.append((name, " ".join([pop] + pops), op))
                    break
                waited += _states(pop, pops)
                if waited >= 2:
                    break
    assert checked > 100 and not bad, bad[:5]


def test_the_products_read_codes_through_wide_loads(kernels):
    name, bodies, text = kernels
    if "moe" not in name:
        return
    for kernel, code in bodies.items():
        if "k_moe_up" in kernel or "k_moe_down" in kernel:
            assert sum(l.startswith("v_mfma_f32_16x16x32_f16") for l in code) >= 16, kernel
            # the ring of units is filled and refilled by them: 2 of a set of rows, 3 units at least
            assert sum(l.startswith("buffer_load_dwordx4") for l in code) >= 12, kernel
            # two wavefronts a SIMD at least: 256 registers each
            found = re.search(rf"\.amdhsa_kernel {kernel}\b.*?\.amdhsa_next_free_vgpr (\d+)", text, re.S)
            assert int(found.group(1)) <= 256


def test_the_choice_in_the_products_holds_what_its_tokens_need(kernels):
    """k_moe_up's own choice, for two tokens at most: logits, ranks of four wavefronts, places and experts of 64
    experts each, beside the sums of four wavefronts."""
    name, bodies, text = kernels
    if "moe" not in name:
        return
    sums = 4 * 2 * 4 * 64 * 4
    choice = 2 * 64 * 8 + 4 * 64 * 4 + 2 * 64 * 4 + 2 * 64 * 4
    seen = set()
    for kernel in bodies:
        if "k_moe_up" in kernel:
            found = re.search(rf"\.amdhsa_kernel {kernel}\b.*?\.amdhsa_group_segment_fixed_size (\d+)", text, re.S)
            chooses = "Lb1EEEv" in kernel  # the last template argument
            seen.add(chooses)
            assert int(found.group(1)) == sums + (choice if chooses else 0), kernel
    assert seen == {True, False}
