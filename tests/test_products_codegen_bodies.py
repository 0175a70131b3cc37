"""The generated gfx950 code of the products and of the transposed compress over whole kernels, from the
label to the function's end: a kernel returns early where it has no tile, and its loads, matrix
instructions and loops lie past the first s_endpgm.  (hipcc, no GPU needed.)

The loads to LDS are written as asm, so three things that the compiler would look after hang on the
source: m0 holds the address of the load that follows, and nothing else; a load has arrived
before the same place is filled again; and before others read it past a barrier."""
import os
import re
import shutil
import subprocess

import pytest

from test_products_codegen import CSRC, flags

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="hipcc not available")


def bodies_of(text):
    """Name and instructions (labels included) of every kernel."""
    out = {}
    for m in re.finditer(r"^(_ZN4tfp8\w*k_\w+):(.*?)^\.Lfunc_end", text, re.S | re.M):
        code = [l.split(";")[0].strip() for l in m.group(2).split("\n")]
        out[m.group(1)] = [l for l in code if l and (l.endswith(":") or not l.startswith("."))]
    return out


def is_lds_load(line):
    return line.startswith("buffer_load") and line.endswith(" lds")


def m0_mistakes(code):
    bad = []
    code = [l for l in code if not l.endswith(":")]
    for i, l in enumerate(code):
        if re.search(r"\bm0\b", l):
            if not (re.match(r"s_mov_b32 m0, s\d+$", l) and code[i + 1] == "s_nop 0"
                    and re.match(r"buffer_load_dwordx4 v\d+, s\[\d+:\d+\], s\d+ offen lds$",
                                 code[i + 2])):
                bad.append(l)
        if is_lds_load(l) and not code[i - 2].startswith("s_mov_b32 m0"):
            bad.append(l)
    return bad


def successors(code):
    at = {l[:-1]: i for i, l in enumerate(code) if l.endswith(":")}
    out = []
    for i, l in enumerate(code):
        to = [i + 1] if i + 1 < len(code) else []
        if l.startswith("s_endpgm"):
            to = []
        elif l.startswith("s_branch"):
            to = [at[l.split()[1]]]
        elif l.startswith("s_cbranch"):
            to = to + [at[l.split()[1]]]
        out.append(to)
    return out


def wait_mistakes(code, barriers):
    """Loads to LDS that can come round again, or (barriers) pass two barriers, with no
    s_waitcnt vmcnt(0) on the way.  (Tiles are read past one barrier after the wait; where scales are
    refilled, another one lies between a load and its wait.)"""
    to = successors(code)
    bad = []
    for start, l in enumerate(code):
        if not is_lds_load(l):
            continue
        seen, front = set(), [(n, 0) for n in to[start]]
        while front:
            n, passed = front.pop()
            if (n, passed) in seen:
                continue
            seen.add((n, passed))
            if re.match(r"s_waitcnt.*vmcnt\(0\)", code[n]):
                continue
            passed += code[n] == "s_barrier"
            if n == start or (barriers and passed == 2):
                bad.append((start, l))
                break
            front += [(x, passed) for x in to[n]]
    return bad


@pytest.fixture(scope="module", params=["tfp8_matmul.hip", "tfp8_compress_t.hip"])
def kernels(request, tmp_path_factory):
    out = str(tmp_path_factory.mktemp("asm") / "k.s")
    r = subprocess.run(["hipcc", *flags(), "--cuda-device-only", "-S", "-o", out,
                        os.path.join(CSRC, request.param)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    text = open(out).read()
    return request.param, bodies_of(text), text


def test_the_bodies_are_whole(kernels):
    name, bodies, text = kernels
    assert len(bodies) == len(re.findall(r"^\s*\.amdhsa_kernel ", text, re.M))
    for kernel, code in bodies.items():
        if "k_matmul" in kernel:
            assert any(is_lds_load(l) for l in code) and any(l.startswith("v_mfma") for l in code), kernel
        else:
            assert any(l.startswith("global_store") for l in code), kernel


def test_no_packed_float32(kernels):
    for kernel, code in kernels[1].items():
        assert not [l for l in code if re.match(r"v_pk_(add|mul|fma)_f32", l)], kernel


def test_no_scratch_memory(kernels):
    sizes = re.findall(r"\.amdhsa_private_segment_fixed_size (\d+)", kernels[2])
    assert len(sizes) == len(kernels[1]) and not any(map(int, sizes)), sizes


def test_m0_holds_the_address_of_the_load_that_follows(kernels):
    for kernel, code in kernels[1].items():
        assert not m0_mistakes(code), kernel


def test_loads_to_lds_are_waited_for(kernels):
    for kernel, code in kernels[1].items():
        assert not wait_mistakes(code, "k_matmul_tile" in kernel), kernel


def test_planted_mistakes_are_found(kernels):
    name, bodies, _ = kernels
    for kernel, code in bodies.items():
        if "k_matmul" not in kernel:
            continue
        last = max(i for i, l in enumerate(code) if l.startswith("v_mfma"))
        assert m0_mistakes(code[:last] + ["s_mov_b32 m0, 0"] + code[last:]), kernel
        loads = [i for i, l in enumerate(code) if is_lds_load(l)]
        assert m0_mistakes(code[:loads[-1] - 1] + code[loads[-1]:]), kernel  # no s_nop
        dry = [l for l in code if not re.match(r"s_waitcnt.*vmcnt\(0\)", l)]
        assert wait_mistakes(dry, "k_matmul_tile" in kernel), kernel


def test_workgroups_a_compute_unit(kernels):
    """kPace's slots are what registers (512 a lane of a SIMD, in eights) and LDS (160 KB) let in, save
    for the three kernels that its comment names."""
    name, bodies, text = kernels
    if "matmul" not in name:
        return
    source = open(os.path.join(CSRC, name)).read()
    table = re.search(r"kPace\[2\]\[kKinds\] = (.*?);", source, re.S).group(1)
    rows = [tuple(map(int, r.split(","))) if r else None
            for r in re.findall(r"\{([\d, ]*)\}", re.sub(r"\s+", " ", table))]
    assert len(rows) == 14
    slots = {(i // 7, *r[:3]): r[3] for i, r in enumerate(rows) if r}
    fewer = {(1, 64, 64, 256): 3, (1, 64, 64, 512): 1, (1, 16, 16, 512): 3}
    found = set()
    for m in re.finditer(r"\.amdhsa_kernel (\S+)(.*?)\.end_amdhsa_kernel", text, re.S):
        tile = re.search(r"k_matmul_tileILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi\d+ELi\dELb(\d)",
                         m.group(1))
        if tile:
            bm, bn, wm, wn, teams, f32 = map(int, tile.groups())
            waves = wm * wn * teams
        else:
            mt, tn, f32 = map(int, re.search(r"k_matmul_splitILi(\d)ELi(\d)ELi\dELb(\d)",
                                             m.group(1)).groups())
            bm, bn, waves = 16 * mt, 16 * tn, 8
        of = lambda k: int(re.search(rf"\.amdhsa_{k} (\d+)", m.group(2)).group(1))
        registers = (of("next_free_vgpr") + 7) // 8 * 8
        fits = min(min(512 // registers, 8) * 4 // waves,
                   160 * 1024 // of("group_segment_fixed_size"))
        key = (f32, bm, bn, 64 * waves)
        found.add(key)
        assert fits == fewer.get(key, slots[key]), (key, fits)
    assert found == set(slots)
