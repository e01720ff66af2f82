"""Positions of several axes without a GPU: the axes of pairs, their tables,
the argument struct, and refusals."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import moe_lora_expert_gb300 as m
from moe_lora_expert_gb300 import attention as A
from oracle import attention_oracle as ao
from test_attention_devices import CALLS, Stream, Stand, fake, ints  # noqa: F401
from test_attention_host import FAKE, append_args, lib, rope_args  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_axes_of_pairs():
    assert m.rope_axes([2, 1, 3]) == bytes([0, 0, 1, 2, 2, 2])
    assert m.rope_axes([3, 1, 2], turns=True) == bytes([0, 1, 2, 0, 2, 0])
    assert m.rope_axes([2, 0, 1], turns=True) == bytes([0, 2, 0])
    assert m.rope_axes([5]) == m.rope_axes([5], turns=True) == bytes(5)
    for bad in ([], [1, 2, 3, 4, 5], [3, -1], [0, 0]):
        with pytest.raises(ValueError):
            m.rope_axes(bad)


def test_tables_of_axes():
    """An axis of its own table has the columns of a table of its own size."""
    axes = m.rope_axes([3, 5], turns=True)
    t = m.rope_table(50, 16, axes=axes)
    for a, n in ((0, 3), (1, 5)):
        own = m.rope_table(50, 2 * n)
        at = [i for i, x in enumerate(axes) if x == a]
        assert torch.equal(t[:, at], own[:, :n]) and torch.equal(t[:, [8 + i for i in at]], own[:, n:])
    assert torch.equal(m.rope_table(50, 16, axes=bytes(8)), m.rope_table(50, 16))
    with pytest.raises(ValueError):
        m.rope_table(50, 16, axes=bytes(7))


def test_oracle_of_axes():
    """One position on all axes is the plain rotation; a column turns by its own axis alone."""
    rng = np.random.default_rng(0)
    f, _ = m.rope_frequencies(16)
    x = rng.standard_normal((2, 20))
    axes = m.rope_axes([3, 2, 3], turns=True)
    for inter in (False, True):
        np.testing.assert_array_equal(ao.rotate_axes(x, [9, 9, 9], axes, f, interleaved=inter), ao.rotate(x, 9, f, interleaved=inter))
        y = ao.rotate_axes(x, [9, 0, 40], axes, f, interleaved=inter)
        for i, a in enumerate(axes):
            for col in ((2 * i, 2 * i + 1) if inter else (i, i + 8)):
                np.testing.assert_array_equal(y[:, col], ao.rotate(x, [9, 0, 40][a], f, interleaved=inter)[:, col])
        np.testing.assert_array_equal(y[:, 16:], x[:, 16:])


def test_the_struct_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = [n for n, _ in m.RopeAxes._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_lora.h"\nint main(void) {\nprintf("%zu", sizeof(moe_rope_axes_t));\n'
                   + "\n".join(f'printf(" %zu", offsetof(moe_rope_axes_t, {n}));' for n in fields) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(m.RopeAxes)] + [getattr(m.RopeAxes, n).offset for n in fields]
    packed = m.RopeAxes.from_buffer_copy(A._AXES.pack(528, 3, 77, bytes([2, 1])))
    assert (packed.struct_size, packed.num_axes, packed.positions_stride, list(packed.axis_of_pair[:3])) == (ctypes.sizeof(packed), 3, 77, [2, 1, 0])


def axes_args(**over):
    x = m.RopeAxes(struct_size=ctypes.sizeof(m.RopeAxes), num_axes=3, positions_stride=4)
    for i in range(64):
        x.axis_of_pair[i] = i % 3
    for k, v in over.items():
        if k == "pair":
            x.axis_of_pair[v[0]] = v[1]
        else:
            setattr(x, k, v)
    return x


AXES_REFUSALS = [({"struct_size": 8}, m.MOE_ERR_UNSUPPORTED), ({"num_axes": 0}, m.MOE_ERR_SHAPE), ({"num_axes": 5}, m.MOE_ERR_UNSUPPORTED),
                 ({"num_axes": 2}, m.MOE_ERR_SHAPE), ({"positions_stride": -1}, m.MOE_ERR_SHAPE), ({"pair": (63, 3)}, m.MOE_ERR_SHAPE)]


@pytest.mark.parametrize("over,status", AXES_REFUSALS)
def test_axes_refusals(lib, over, status):  # noqa: F811
    x = bytes(axes_args(**over))
    assert lib.moe_rope_axes(bytes(rope_args()), x, None) == status
    a = append_args(cos_sin=FAKE, rotary_dim=128, positions=FAKE, num_positions=100)
    assert lib.moe_kv_append_axes(bytes(a), x, None) == status


def test_axes_beyond_the_pairs_are_not_read(lib):  # noqa: F811
    x = bytes(axes_args(pair=(64, 200)))
    assert lib.moe_rope_axes(bytes(rope_args(N=0)), x, None) == m.MOE_OK
    a = append_args(cos_sin=FAKE, rotary_dim=128, positions=FAKE, num_positions=100, N=0, B=0)
    assert lib.moe_kv_append_axes(bytes(a), x, None) == m.MOE_OK


def test_other_refusals(lib):  # noqa: F811
    x = bytes(axes_args())
    for over, status in (({"positions": None}, m.MOE_ERR_NULL), ({"rotary_dim": 130}, m.MOE_ERR_SHAPE), ({"dtype": 3}, m.MOE_ERR_UNSUPPORTED)):
        assert lib.moe_rope_axes(bytes(rope_args(**over)), x, None) == status
    good = dict(cos_sin=FAKE, rotary_dim=128, positions=FAKE, num_positions=100)
    for over, status in (({"positions": None}, m.MOE_ERR_NULL), ({"cos_sin": None, "rotary_dim": 0}, m.MOE_ERR_SHAPE), ({"k": None}, m.MOE_ERR_NULL)):
        assert lib.moe_kv_append_axes(bytes(append_args(**{**good, **over})), x, None) == status
    for fn, args in ((lib.moe_rope_axes, rope_args()), (lib.moe_kv_append_axes, append_args(**good))):
        assert fn(None, x, None) == m.MOE_ERR_NULL and fn(bytes(args), None, None) == m.MOE_ERR_NULL


# ----------------------------------------------------------- the binding's part

AXES_CALLS = {"_rope_axes_fn": "_rope_fn", "_append_axes_fn": "_append_fn"}


@pytest.fixture
def calls(fake, monkeypatch):  # noqa: F811
    """Stand-ins for the two entry points as well: what they were given."""
    seen, current = [], fake[1]
    for name in AXES_CALLS:
        monkeypatch.setattr(A, name, lambda args, axes, handle, name=name: seen.append((name, current[0], handle, axes)) or 0)
    return seen, current


def run(name, **over):
    call, args = CALLS[AXES_CALLS[name]]
    args = {k: t.moved(1) for k, t in args.items()}
    return call(**{**args, "positions": ints(3, 4), "axes": m.rope_axes([10, 11, 11]), **over})


@pytest.mark.parametrize("name", AXES_CALLS)
def test_axes_calls_run_on_their_tensors_device(calls, name):
    seen, current = calls
    run(name)
    run(name, stream=Stream(7, 1))
    run(name, axes=list(m.rope_axes([10, 11, 11])))
    assert [s[:3] for s in seen] == [(name, 1, 100), (name, 1, 7), (name, 1, 100)] and current[0] == 0
    x = m.RopeAxes.from_buffer_copy(seen[0][3])
    assert (x.num_axes, x.positions_stride, bytes(x.axis_of_pair[:32])) == (3, 4, m.rope_axes([10, 11, 11]))
    assert seen[2][3] == seen[0][3]


@pytest.mark.parametrize("name", AXES_CALLS)
@pytest.mark.parametrize("over,word", [
    ({"positions": ints(4)}, "positions"), ({"positions": ints(3, 5)}, "positions"), ({"positions": Stand((3, 4), torch.int64)}, "positions"),
    ({"positions": Stand((3, 4), torch.int32, 0)}, "positions"), ({"positions": None}, "positions"), ({"positions": ints(2, 4)}, "axes"),
    ({"positions": ints(5, 4)}, "axes"), ({"axes": bytes(31)}, "axes"), ({"axes": bytes(33)}, "axes"), ({"axes": b""}, "axes")])
def test_axes_calls_refuse(calls, name, over, word):
    with pytest.raises(ValueError, match=word):
        run(name, **over)
    assert not calls[0]
