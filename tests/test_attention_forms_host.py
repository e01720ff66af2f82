"""Sinks and shared prefixes without a GPU: argument structs, refusals, what the
binding hands on, and the oracle's own pins."""
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
from test_attention_devices import CALLS, Stand, Stream, fake, ints  # noqa: F401
from test_attention_host import FAKE, attend_args, lib  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_struct_matches_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    fields = [n for n, _ in m.SharedPrefix._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_lora.h"\nint main(void) {\nprintf("%zu", sizeof(moe_shared_prefix_t));\n'
                   + "\n".join(f'printf(" %zu", offsetof(moe_shared_prefix_t, {n}));' for n in fields) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(m.SharedPrefix)] + [getattr(m.SharedPrefix, n).offset for n in fields]
    x = m.SharedPrefix.from_buffer_copy(A._SHARED.pack(48, 3, 77, 1, 2, 4, 5))
    assert (x.struct_size, x.groups, x.max_tokens, x.seqs, x.lens, x.partial, x.partial_bytes) == (ctypes.sizeof(x), 3, 77, 1, 2, 4, 5)


@pytest.mark.parametrize("sinks,over,status", [
    (-1, {}, m.MOE_ERR_SHAPE), (4, {"window": -1}, m.MOE_ERR_SHAPE), (4, {"q": None}, m.MOE_ERR_NULL), (4, {"struct_size": 8}, m.MOE_ERR_UNSUPPORTED),
    (4, {"workspace": None}, m.MOE_ERR_WORKSPACE), (4, {"N": 0, "B": 0}, m.MOE_OK), (-4, {"N": 0, "B": 0}, m.MOE_ERR_SHAPE),
    (4, {"max_q_len": 0}, m.MOE_OK)])
def test_sinks_refusals(lib, sinks, over, status):  # noqa: F811
    assert lib.moe_paged_attention_sinks(bytes(attend_args(lib, **{"window": 64, **over})), sinks, None) == status


def shared(lib, **over):  # noqa: F811
    x = m.SharedPrefix(struct_size=ctypes.sizeof(m.SharedPrefix), groups=2, max_tokens=4, seqs=FAKE, lens=FAKE, partial=FAKE,
                       partial_bytes=lib.moe_shared_prefix_partial_size(4, 32, 128, 2))
    for k, v in over.items():
        setattr(x, k, v)
    return bytes(x)


@pytest.mark.parametrize("over,more,status", [
    ({}, {"struct_size": 8}, m.MOE_ERR_UNSUPPORTED), ({"window": 5}, {}, m.MOE_ERR_UNSUPPORTED), ({}, {"groups": -1}, m.MOE_ERR_SHAPE),
    ({}, {"max_tokens": -1}, m.MOE_ERR_SHAPE), ({}, {"lens": None}, m.MOE_ERR_NULL), ({}, {"seqs": None}, m.MOE_ERR_NULL),
    ({}, {"partial": None}, m.MOE_ERR_WORKSPACE), ({}, {"partial": FAKE + 16}, m.MOE_ERR_WORKSPACE), ({}, {"partial_bytes": 64}, m.MOE_ERR_WORKSPACE),
    ({"q": None}, {}, m.MOE_ERR_NULL), ({"Hq": 30}, {}, m.MOE_ERR_SHAPE), ({"N": 0, "B": 0}, {}, m.MOE_OK), ({"max_q_len": 0}, {}, m.MOE_OK)])
def test_shared_refusals(lib, over, more, status):  # noqa: F811
    assert lib.moe_paged_attention_shared(bytes(attend_args(lib, **over)), shared(lib, **more), None) == status


def test_null_arguments(lib):  # noqa: F811
    assert lib.moe_paged_attention_sinks(None, 4, None) == m.MOE_ERR_NULL
    assert lib.moe_paged_attention_shared(None, shared(lib), None) == m.MOE_ERR_NULL
    assert lib.moe_paged_attention_shared(bytes(attend_args(lib)), None, None) == m.MOE_ERR_NULL


def test_partial_size(lib):  # noqa: F811
    """Some pieces of every row, with its reference and denominator; less for
    each where there are many rows."""
    size = lib.moe_shared_prefix_partial_size
    assert size(0, 32, 128, 1) == size(4, 0, 128, 1) == size(4, 32, 0, 1) == size(4, 32, 128, 0) == 0
    for N, Hq, D, G in ((1, 1, 16, 1), (64, 32, 128, 1), (128, 32, 128, 5), (100000, 64, 64, 3)):
        pieces, rest = divmod(size(N, Hq, D, G) - 4 * G, N * Hq * (4 * D + 8))
        assert rest == 0 and 3 <= pieces <= 33 and pieces % 2 == 1
    assert size(64, 32, 128, 1) > size(32, 32, 128, 1) / 2


# ----------------------------------------------------------- the binding's part

@pytest.fixture
def calls(fake, monkeypatch):  # noqa: F811
    seen, current = [], fake[1]
    for name in ("_attend_fn", "_sinks_fn", "_shared_fn"):
        monkeypatch.setattr(A, name, lambda args, *more, name=name: seen.append((name, current[0], more)) or 0)
    real = A._empty
    monkeypatch.setattr(A, "_empty", lambda shape, dtype, device, stream: Stand(shape, dtype, 1) if dtype is torch.uint8 else real(shape, dtype, device, stream))
    return seen, current


def run(**over):
    call, args = CALLS["_attend_fn"]
    return call(**{**{k: t.moved(1) for k, t in args.items()}, **over})


def test_calls_of_forms(calls):
    seen, current = calls
    lens, seqs = ints(2), ints(3)
    run()
    run(window=5, sinks=3)
    run(window=5, sinks=1 << 40)
    run(shared_lens=lens, shared_seqs=seqs)
    run(shared_lens=lens, shared_seqs=seqs, max_shared_q=2, stream=Stream(7, 1))
    run(shared_lens=ints(1))
    assert [s[:2] for s in seen] == [("_attend_fn", 1), ("_sinks_fn", 1), ("_sinks_fn", 1), ("_shared_fn", 1), ("_shared_fn", 1), ("_shared_fn", 1)]
    assert current[0] == 0 and seen[0][2] == (100,) and seen[1][2] == (3, 100) and seen[2][2] == (1 << 30, 100) and seen[4][2][1] == 7
    x = [m.SharedPrefix.from_buffer_copy(s[2][0]) for s in seen[3:]]
    assert [(a.groups, a.max_tokens, bool(a.seqs), bool(a.lens)) for a in x] == [(2, 4, True, True), (2, 2, True, True), (1, 4, False, True)]
    assert lens.used_on.cuda_stream == seqs.used_on.cuda_stream == 7


@pytest.mark.parametrize("over,word", [
    (dict(shared_lens=ints(2), window=5), "window"), (dict(shared_lens=ints(2), sinks=5), "window"), (dict(shared_lens=ints(2)), "shared_seqs"),
    (dict(shared_seqs=ints(3)), "shared_lens"), (dict(shared_lens=ints(2), shared_seqs=ints(2)), "shared_seqs"),
    (dict(shared_lens=Stand((1,), torch.int64)), "shared_lens"), (dict(shared_lens=Stand((1,), torch.int32, 0)), "shared_lens"),
    (dict(shared_lens=ints(1), shared_seqs=Stand((2,), torch.int32, -1)), "shared_seqs")])
def test_refusals_of_forms(calls, over, word):
    with pytest.raises(ValueError, match=word):
        run(**over)
    assert not calls[0]


# ------------------------------------------------------------ the oracle's pins

def test_oracle_of_sinks():
    """A row sees its window and the first tokens: the softmax over just those."""
    rng = np.random.default_rng(0)
    kc, vc = (ao.e4m3_encode(rng.standard_normal((4, 1, 8, 16))) for _ in range(2))
    one = np.ones((4, 1), np.float32)
    q = rng.standard_normal((2, 1, 16))
    table, n = [[2, 0, 3, 1]], 27
    out, lse, _, _ = ao.attend(q, kc, vc, one, one, table, [n], [0, 2], 0.25, window=6, sinks=3)
    k, v = (ao.E4M3_VALUES[c[table[0]]].reshape(-1, 16) for c in (kc, vc))
    for t in range(2):
        i = n - 2 + t
        see = [0, 1, 2] + list(range(i - 5, i + 1))
        s = torch.from_numpy(q[t] @ k[see].T * 0.25)
        np.testing.assert_allclose(out[t], torch.softmax(s, -1).numpy() @ v[see], rtol=1e-12)
        np.testing.assert_allclose(lse[t], torch.logsumexp(s, -1).numpy(), rtol=1e-12)
    same = ao.attend(q, kc, vc, one, one, table, [n], [0, 2], 0.25, window=6, sinks=22)
    full = ao.attend(q, kc, vc, one, one, table, [n], [0, 2], 0.25)
    np.testing.assert_allclose(same[0], full[0], rtol=1e-12)
    np.testing.assert_array_equal(ao.attend(q, kc, vc, one, one, table, [n], [0, 2], 0.25, window=6, sinks=0)[0],
                                  ao.attend(q, kc, vc, one, one, table, [n], [0, 2], 0.25, window=6)[0])
