"""Refusals of the optimizer's calls (before any HIP call, so they run without a GPU), and the random bits."""
import ctypes
import math

import numpy as np
import pytest
import torch

import fp8_compression_tensor_amd as tfp8
import optimizer_helpers as H
from fp8_compression_tensor_amd.optimizer import AdamWOptions

F = 0x7F0000000000  # an aligned address that is never dereferenced here
G = 1 << 30
STATE = (F + 8 * G, F + 9 * G, F + 10 * G, F + 11 * G)
DATA, ALPHA, SCALE, N, DTYPE, PARAM, COPY, CALPHA, CSCALE, START, PDTYPE, CDTYPE = range(12)
DENSE = (F, 0, 0, 1000, 1, F + G, 0, 0, 0, 0, 1, -1)
CODES = (F, F + 2 * G, F + 3 * G, 1024, 2, F + G, F + 4 * G, F + 5 * G, F + 6 * G, 0, 1, 2)


def put(row, **changes):
    names = "DATA ALPHA SCALE N DTYPE PARAM COPY CALPHA CSCALE START PDTYPE CDTYPE".split()
    row = list(row)
    for k, v in changes.items():
        row[names.index(k)] = v
    return tuple(row)


def options(**changes):
    o = AdamWOptions(1e-3, 0.9, 0.999, 1e-8, 0.01, 1, 0)
    for k, v in changes.items():
        setattr(o, k, v)
    return o


def step(rows, block=128, bits=8, state=STATE, out=None, n=2048, o=None, count=None):
    t = np.array(rows, dtype=np.int64)
    o = options() if o is None else o
    return tfp8.adamw_raw(t.ctypes.data, len(rows) if count is None else count, block, bits, state,
                          state if out is None else out, n, ctypes.byref(o))


def norm(rows, block=128, max_norm=1.0, ws=F + 20 * G, nbytes=1 << 20, norm=F + 21 * G,
         scale=F + 22 * G, count=None):
    t = np.array([r[:5] for r in rows], dtype=np.int64)
    return tfp8.grad_norm_raw(t.ctypes.data, len(rows) if count is None else count, block, max_norm, ws,
                              nbytes, norm, scale)


@pytest.mark.parametrize("call", [step, norm])
@pytest.mark.parametrize("row", [DENSE, CODES])
def test_gradients_are_refused(call, row):
    for block in (0, 96, 1024, -64):
        assert call([row], block=block) == -3
    assert call([row], count=-1) == -2 and call([row], count=(1 << 24) + 1) == -2
    assert call([put(row, N=-1)]) == -2 and call([put(row, N=(1 << 40) + 128)]) == -2
    assert call([put(row, DTYPE=3)]) == -4 and call([put(row, DTYPE=-1)]) == -4
    assert call([put(row, DATA=0)]) == -1 and call([put(row, DATA=F + 8)]) == -5
    assert call([put(CODES, N=1000)]) == -2
    assert call([put(CODES, ALPHA=0)]) == -1 and call([put(CODES, SCALE=0)]) == -1
    assert call([put(CODES, ALPHA=F + 2 * G + 2)]) == -5


def test_norm_arguments():
    for bad in (0.0, -1.0, math.nan):
        assert norm([DENSE], max_norm=bad) == -6
    assert norm([DENSE], ws=0) == -1 and norm([DENSE], norm=0) == -1 and norm([DENSE], scale=0) == -1
    assert norm([DENSE], ws=F + 20 * G + 4) == -5 and norm([DENSE], norm=F + 21 * G + 2) == -5
    need = tfp8.lib().tfp8_grad_norm_workspace(1)
    assert norm([DENSE], nbytes=need - 1) == -2
    assert tfp8.lib().tfp8_grad_norm_workspace(-1) == 0
    for at in (DENSE[0], DENSE[0] + 3996, F + 21 * G):
        assert norm([DENSE], scale=at) == -6 and norm([DENSE], norm=at, scale=at) == -6


def test_step_arguments():
    assert step([DENSE], bits=16) == -6
    for bad in (dict(beta1=1.0), dict(beta2=-0.1), dict(beta1=math.nan), dict(eps=0.0), dict(eps=1e-39),
                dict(eps=math.inf), dict(lr=math.nan), dict(weight_decay=math.inf), dict(step=0)):
        assert step([DENSE], o=options(**bad)) == -6, bad
    assert step([DENSE], o=options(lr_dev=F + 30 * G)) == -1  # no workspace
    assert step([DENSE], o=options(step_dev=F + 30 * G + 4, workspace=F + 31 * G)) == -5
    assert step([DENSE], o=options(grad_scale=F + 2)) == -5
    assert step([put(DENSE, PDTYPE=2)]) == -4 and step([put(DENSE, CDTYPE=1)]) == -4
    assert step([put(DENSE, PARAM=0)]) == -1 and step([put(DENSE, PARAM=F + G + 4)]) == -5
    assert step([put(DENSE, CDTYPE=0)]) == -1
    assert step([put(CODES, CALPHA=0)]) == -1 and step([put(CODES, COPY=F + 4 * G + 8)]) == -5
    assert step([put(DENSE, COPY=F + 4 * G, CALPHA=F + 5 * G, CSCALE=F + 6 * G, CDTYPE=2)]) == -2
    assert step([put(DENSE, START=64)]) == -2 and step([put(DENSE, START=-128)]) == -2
    assert step([put(DENSE, START=1152)]) == -6  # past the states
    second = put(DENSE, DATA=F + 2 * G, PARAM=F + 3 * G)
    assert step([DENSE, put(second, START=896)]) == -6  # into the first one's last block
    assert step([put(DENSE, START=1024, N=512), put(second, N=512)]) == -6  # out of order
    for i in range(4):
        lost = tuple(None if k == i else a for k, a in enumerate(STATE))
        assert step([DENSE], state=lost, out=STATE) == -1 and step([DENSE], out=lost) == -1
        off = tuple(a + 2 if k == i else a for k, a in enumerate(STATE))
        assert step([DENSE], state=off, out=STATE) == -5
    assert step([put(DENSE, N=0, DATA=0, PARAM=0)], state=(None,) * 4) == 0
    assert step([DENSE], count=0) == 0


def test_overlaps_are_refused():
    assert step([put(DENSE, PARAM=F)]) == -6 and step([put(DENSE, PARAM=F + 3984)]) == -6
    second = put(DENSE, DATA=F + 2 * G, START=1024)
    assert step([DENSE, second]) == -6  # one parameter twice
    assert step([put(CODES, COPY=F + G)]) == -6 and step([put(CODES, CALPHA=F + 6 * G)]) == -6
    assert step([put(DENSE, PARAM=STATE[2])]) == -6
    moved = (STATE[0] + 16, *STATE[1:])
    assert step([DENSE], out=moved) == -6  # neither in place nor apart
    assert step([DENSE], o=options(grad_scale=F + G + 400)) == -6


def test_wrappers_refuse_what_is_not_on_a_gpu():
    p = torch.zeros(256)
    for call in (lambda: tfp8.grad_norm([p]), lambda: tfp8.adamw_state([p]),
                 lambda: tfp8.adamw([p], [p], (p, p), 1e-3)):
        with pytest.raises(ValueError, match="GPU"):
            call()
    for call in (lambda: tfp8.grad_norm([]), lambda: tfp8.grad_norm([p], block=96),
                 lambda: tfp8.grad_norm([p], 0.0), lambda: tfp8.adamw([], [], (), 1e-3),
                 lambda: tfp8.adamw([p], [], (), 1e-3), lambda: tfp8.adamw_state([p], 16)):
        with pytest.raises(ValueError):
            call()


def test_random_bits_are_even():
    """The mixing of seed, step and index: every bit of the halves that the rounding takes is set half of
    the time, whatever neighbouring indexes, steps and seeds are, and neighbours share nothing."""
    n = 1 << 16
    rows = [H.random_bits(seed, step, 0, n) for seed in (0, 1, 1 << 40) for step in (1, 2, 3, 1 << 33)]
    rows.append(H.random_bits(0, 1, (1 << 32) - n // 2, n))
    for r in rows:
        for k in range(32):
            assert abs(float((r >> k & 1).double().mean()) - 0.5) < 6 * 0.5 / n ** 0.5
        for half in (r & 0xFFFF, r >> 16):
            u = half.double() / 65536 - 0.5
            assert abs(float(u.mean())) < 6 * 12 ** -0.5 / n ** 0.5
            for lag in (1, 2, 4, 128, 1024):
                assert abs(float((u[lag:] * u[:-lag]).mean())) < 6 / 12 / (n - lag) ** 0.5
    for i, a in enumerate(rows):
        for c in rows[:i]:
            x, y = (t.double() / 2 ** 32 - 0.5 for t in (a, c))
            assert abs(float((x * y).mean())) < 6 / 12 / n ** 0.5


def test_rows_of_tensors():
    """What the module makes of a list: rows of what lies contiguous on the device, which is the CPU's
    number -1 here and so nothing but None; the others are left to the caller, whatever they are."""
    from fp8_compression_tensor_amd import optimizer

    x = torch.ones(3)
    items = [x, torch.nn.Parameter(torch.ones(4, 2)), None, (1, 2), torch.ones(2).double(), "x", (x, x, x)]
    table = np.full((7, 5), 7, dtype=np.int64)
    assert optimizer._fill(items, -1, table, 64, 7) == list(range(7)) and (table == 7).all()
    assert optimizer._fill(items, -1, table, 64, 15) == [0, 1, 3, 4, 5, 6]
    assert table[2].tolist() == [0, 0, 0, 0, -1]
    assert optimizer._fill([], 0, table, 64, 7) == ()
    for bad in ((), (items, 0), (tuple(items), 0, table, 5, 64, 7), (items, "0", table, 5, 64, 7),
                (items, 0, None, 5, 64, 7)):
        with pytest.raises(TypeError):
            optimizer._rows(*bad)
    for bad in ((6, 64, 7), (4, 64, 7), (0, 64, 7), (-5, 64, 7), (5, 0, 7)):  # past the table, no block
        with pytest.raises(ValueError):
            optimizer._rows(items, 0, table, *bad)
    with pytest.raises(BufferError):
        optimizer._rows(items, 0, bytes(280), 5, 64, 7)


def test_a_missing_module_raises(monkeypatch):
    import sys
    from fp8_compression_tensor_amd import optimizer

    monkeypatch.setattr(optimizer, "_rows", None)
    monkeypatch.setitem(sys.modules, "fp8_compression_tensor_amd._rows", None)
    with pytest.raises(RuntimeError, match="not built"):
        optimizer._fill([], 0, None, 64, 7)


def test_an_empty_gradient_is_refused():
    for g in ((), [], ((),)):
        with pytest.raises(ValueError):
            tfp8.grad_norm([g])


def test_submodules_take_no_name_of_the_package():
    """Importing a submodule binds its name in the package, over a function of that name."""
    import subprocess
    import sys

    code = """if 1:
        import importlib, os, pkgutil
        import fp8_compression_tensor_amd as tfp8
        before = dict(vars(tfp8))
        names = [m.name for m in pkgutil.iter_modules(tfp8.__path__)]
        assert "_rows" in names and "optimizer" in names, names
        for name in names:
            if name in ("_rows", "optimizer", "expert_layer", "ablation", "build"):
                importlib.import_module("fp8_compression_tensor_amd." + name)
        changed = [k for k, v in before.items() if vars(tfp8)[k] is not v]
        assert not changed, changed
    """
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_step_rows_arguments():
    from fp8_compression_tensor_amd import optimizer

    optimizer._load()
    x, table = torch.ones(3), np.zeros((2, 12), dtype=np.int64)
    assert optimizer._step_rows([], [], None, 0, table, 64) == (0, table.ctypes.data)
    assert optimizer._step_rows([x], [x], None, -1, table, 64) is None  # not on a GPU: the caller's
    for bad in ((), ((x,), [x], None, 0, table, 64), ([x], [x], (None,), 0, table, 64),
                ([x], [x], None, "0", table, 64), ([x], [x], None, 0, None, 64)):
        with pytest.raises(TypeError):
            optimizer._step_rows(*bad)
    for bad in (([x] * 3, [x] * 3, None, 0, table, 64), ([x], [], None, 0, table, 64),
                ([x], [x], [], 0, table, 64), ([x], [x], None, 0, table, 0)):
        with pytest.raises(ValueError):
            optimizer._step_rows(*bad)
    with pytest.raises(BufferError):
        optimizer._step_rows([x], [x], None, 0, bytes(192), 64)
    assert optimizer._address(table) == table.ctypes.data
    for bad in (bytes(8), None):
        with pytest.raises((BufferError, TypeError)):
            optimizer._address(bad)


@pytest.mark.parametrize("bits", [8, 32])
def test_states_hold_whole_blocks(bits):
    """A tensor's part of the states is rounded up to whole blocks, of which states of 8 bits have a scale each:
    with 1000 elements in states of 1000, the scale of the eighth block would lie past the seven."""
    odd = (STATE[0] + 2, *STATE[1:])  # refused after the tensors: no call here gets past the checks
    for n in (1000, 1023):
        assert step([DENSE], bits=bits, state=odd, n=n) == -6
        assert step([put(DENSE, START=1024)], bits=bits, state=odd, n=1024 + n) == -6
    assert step([put(DENSE, N=1)], block=512, bits=bits, state=odd, n=511) == -6
    assert step([DENSE], bits=bits, state=odd, n=1024) == -5
    assert step([put(DENSE, N=896)], bits=bits, state=odd, n=1000) == -5


def test_scales_of_whole_blocks():
    """States of 1000 have seven scales: the two lists of them may not share the seventh."""
    shared = (STATE[0], STATE[1], STATE[2], STATE[1] + 24)
    assert step([put(DENSE, N=896)], state=shared, n=1000) == -6


def test_the_package_without_numpy():
    """Only grad_norm and adamw lay their tables out with numpy: without it they say so, and the rest is there."""
    import subprocess
    import sys

    code = """if 1:
        import sys, warnings
        warnings.simplefilter("ignore")
        sys.modules["numpy"] = None
        import fp8_compression_tensor_amd as tfp8
        from fp8_compression_tensor_amd import expert_layer, optimizer
        assert tfp8.lib().tfp8_version() > 0
        for columns in (5, 12):
            try:
                optimizer._table(3, columns)
            except RuntimeError as e:
                assert "numpy" in str(e)
            else:
                raise AssertionError
    """
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
