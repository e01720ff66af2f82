"""The attention half without a GPU: argument structs, refusals, the angle
tables, and the oracle's own pins."""
import ctypes
import math
import os
import shutil
import subprocess

import numpy as np
import pytest

import moe_lora_expert_gb300 as m
from moe_lora_expert_gb300 import attention as A
from oracle import attention_oracle as ao

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(m.LIB_PATH):
        from moe_lora_expert_gb300 import _build
        _build.build()
    return m.lib()


def test_structs_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = [(m.RopeArgs, "moe_rope_args_t"), (m.KvCache, "moe_kv_cache_t"),
               (m.KvAppendArgs, "moe_kv_append_args_t"), (m.PagedAttentionArgs, "moe_paged_attention_args_t")]
    lines = []
    for struct, ctype in structs:
        lines.append(f'printf("{ctype} sizeof %zu\\n", sizeof({ctype}));')
        for f, _ in struct._fields_:
            lines.append(f'printf("{ctype} {f} %zu\\n", offsetof({ctype}, {f}));')
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moe_lora.h"\nint main(void) {\n'
                   + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run([cc, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = {tuple(ln.split()[:2]): int(ln.split()[2])
           for ln in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines()}
    for struct, ctype in structs:
        assert got[ctype, "sizeof"] == ctypes.sizeof(struct)
        for f, _ in struct._fields_:
            assert got[ctype, f] == getattr(struct, f).offset, (ctype, f)


def test_packed_bytes_are_the_structs():
    """The bytes that the binding packs land in the fields they are meant for."""
    r = m.RopeArgs.from_buffer_copy(A._ROPE.pack(A._ROPE.size, 1, *range(10, 14), *range(20, 28), 30, 31, 32,
                                                 *range(40, 48)))
    assert ctypes.sizeof(r) == A._ROPE.size == r.struct_size
    assert (r.q, r.k_out, r.q_stride_token, r.k_out_stride_head, r.positions, r.status, r.N, r.inverse) == (
        10, 13, 20, 27, 30, 32, 40, 47)
    cache = A._CACHE.pack(1, 2, 3, 4, *range(5, 11), 12, 13, 14, 15)
    raw = A._HEAD.pack(7, 0) + cache + A._APPEND.pack(1, 2, *range(3, 7), 8, 9, *range(10, 14), *range(20, 26),
                                                      *range(30, 38))
    k = m.KvAppendArgs.from_buffer_copy(raw)
    assert len(raw) == ctypes.sizeof(k)
    assert (k.cache.v_scale, k.cache.v_stride_token, k.cache.head_dim, k.v, k.q_out, k.status, k.N, k.interleaved) == (
        4, 10, 15, 2, 9, 25, 30, 37)
    raw = A._HEAD.pack(7, 0) + cache + A._ATTEND.pack(1, 2, 3, *range(4, 8), *range(10, 16), *range(20, 28), 0.5, 9)
    t = m.PagedAttentionArgs.from_buffer_copy(raw)
    assert len(raw) == ctypes.sizeof(t)
    assert (t.lse, t.block_table, t.workspace_bytes, t.wait_timeout_ms, t.scale, t.debug_flags) == (3, 10, 15, 27, .5, 9)


FAKE = 1 << 20   # never dereferenced: each call fails a check first


def rope_args(**over):
    a = m.RopeArgs()
    a.struct_size = ctypes.sizeof(a)
    a.q = a.q_out = a.positions = a.cos_sin = FAKE
    a.q_stride_token = a.q_out_stride_token = 256
    a.q_stride_head = a.q_out_stride_head = 128
    a.N, a.Hq, a.Hk, a.D, a.rotary_dim, a.num_positions = 4, 2, 0, 128, 128, 100
    for k, v in over.items():
        setattr(a, k, v)
    return a


def cache(**over):
    c = m.KvCache(FAKE, FAKE, FAKE, FAKE, 4 * 16 * 128, 16 * 128, 128, 4 * 16 * 128, 16 * 128, 128, 10, 4, 16, 128)
    for k, v in over.items():
        setattr(c, k, v)
    return c


def append_args(cache_over=None, **over):
    a = m.KvAppendArgs()
    a.struct_size = ctypes.sizeof(a)
    a.cache = cache(**(cache_over or {}))
    a.k = a.v = a.block_table = a.seq_lens = FAKE
    a.k_stride_token, a.k_stride_head, a.v_stride_token, a.v_stride_head = 512, 128, 512, 128
    a.N = a.B = 4
    a.table_width, a.max_q_len = 8, 1
    for k, v in over.items():
        setattr(a, k, v)
    return a


def attend_args(lib, cache_over=None, **over):
    a = m.PagedAttentionArgs()
    a.struct_size = ctypes.sizeof(a)
    a.cache = cache(**(cache_over or {}))
    a.q = a.out = a.block_table = a.seq_lens = a.workspace = FAKE
    a.q_stride_token = a.out_stride_token = 32 * 128
    a.q_stride_head = a.out_stride_head = 128
    a.workspace_bytes = lib.moe_paged_attention_workspace_size()
    a.N = a.B = 4
    a.Hq, a.table_width, a.max_q_len, a.max_seq_len, a.scale = 32, 8, 1, 128, 0.1
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("over,status", [
    ({"struct_size": 8}, m.MOE_ERR_UNSUPPORTED), ({"dtype": 3}, m.MOE_ERR_UNSUPPORTED),
    ({"N": -1}, m.MOE_ERR_SHAPE), ({"rotary_dim": 130}, m.MOE_ERR_SHAPE), ({"rotary_dim": 63}, m.MOE_ERR_SHAPE),
    ({"rotary_dim": 0}, m.MOE_ERR_SHAPE), ({"D": 127, "rotary_dim": 64}, m.MOE_ERR_SHAPE),
    ({"D": 2048}, m.MOE_ERR_UNSUPPORTED), ({"q": None}, m.MOE_ERR_NULL), ({"q_out": None}, m.MOE_ERR_NULL),
    ({"Hk": 1}, m.MOE_ERR_NULL), ({"positions": None}, m.MOE_ERR_NULL), ({"cos_sin": None}, m.MOE_ERR_NULL),
    ({"cos_sin": FAKE + 4}, m.MOE_ERR_ALIGN), ({"N": 0}, m.MOE_OK), ({"Hq": 0}, m.MOE_OK),
])
def test_rope_refusals(lib, over, status):
    assert lib.moe_rope(bytes(rope_args(**over)), None) == status


@pytest.mark.parametrize("cache_over,over,status", [
    ({}, {"struct_size": 8}, m.MOE_ERR_UNSUPPORTED), ({}, {"dtype": m.MOE_DTYPE_F32}, m.MOE_ERR_UNSUPPORTED),
    ({"head_dim": 136}, {}, m.MOE_ERR_UNSUPPORTED), ({"head_dim": 144}, {}, m.MOE_ERR_UNSUPPORTED),
    ({"page_size": 12}, {}, m.MOE_ERR_UNSUPPORTED), ({"page_size": 264}, {}, m.MOE_ERR_UNSUPPORTED),
    ({"page_size": 0}, {}, m.MOE_ERR_SHAPE), ({"kv_heads": 0}, {}, m.MOE_ERR_SHAPE), ({"k": None}, {}, m.MOE_ERR_NULL),
    ({"v_scale": None}, {}, m.MOE_ERR_NULL), ({"k": FAKE + 8}, {}, m.MOE_ERR_ALIGN),
    ({"v_stride_token": 136}, {}, m.MOE_ERR_ALIGN), ({"k_stride_page": -16}, {}, m.MOE_ERR_SHAPE),
    ({}, {"N": 5}, m.MOE_ERR_SHAPE), ({}, {"B": -1}, m.MOE_ERR_SHAPE), ({}, {"seq_lens": None}, m.MOE_ERR_NULL),
    ({}, {"block_table": None}, m.MOE_ERR_NULL), ({}, {"k": None}, m.MOE_ERR_NULL),
    ({}, {"rotary_dim": 64}, m.MOE_ERR_NULL), ({}, {"cos_sin": FAKE, "rotary_dim": 130}, m.MOE_ERR_SHAPE),
    ({}, {"cos_sin": FAKE + 4, "rotary_dim": 64}, m.MOE_ERR_ALIGN), ({}, {"Hq": 2}, m.MOE_ERR_NULL),
    ({}, {"N": 0, "B": 0}, m.MOE_OK),
])
def test_append_refusals(lib, cache_over, over, status):
    assert lib.moe_kv_append(bytes(append_args(cache_over, **over)), None) == status


@pytest.mark.parametrize("cache_over,over,status", [
    ({}, {"struct_size": 8}, m.MOE_ERR_UNSUPPORTED), ({}, {"dtype": m.MOE_DTYPE_F32}, m.MOE_ERR_UNSUPPORTED),
    ({"head_dim": 136}, {}, m.MOE_ERR_UNSUPPORTED), ({"page_size": 12}, {}, m.MOE_ERR_UNSUPPORTED),
    ({}, {"Hq": 30}, m.MOE_ERR_SHAPE), ({}, {"Hq": 0}, m.MOE_ERR_SHAPE), ({}, {"window": -1}, m.MOE_ERR_SHAPE),
    ({}, {"max_seq_len": -1}, m.MOE_ERR_SHAPE), ({}, {"N": 3}, m.MOE_ERR_SHAPE), ({}, {"q": None}, m.MOE_ERR_NULL),
    ({}, {"out": None}, m.MOE_ERR_NULL), ({}, {"q": FAKE + 8}, m.MOE_ERR_ALIGN),
    ({}, {"q_stride_head": 132}, m.MOE_ERR_ALIGN), ({}, {"workspace": None}, m.MOE_ERR_WORKSPACE),
    ({}, {"workspace": FAKE + 64}, m.MOE_ERR_WORKSPACE), ({}, {"workspace_bytes": 16}, m.MOE_ERR_WORKSPACE),
    ({}, {"debug_flags": 8}, m.MOE_ERR_UNSUPPORTED),
    ({}, {"Hq": 4 * 257}, m.MOE_ERR_UNSUPPORTED), ({}, {"N": 0, "B": 0}, m.MOE_OK),
])
def test_attention_refusals(lib, cache_over, over, status):
    assert lib.moe_paged_attention(bytes(attend_args(lib, cache_over, **over)), None) == status


def test_null_arguments(lib):
    for fn in (lib.moe_rope, lib.moe_kv_append, lib.moe_paged_attention):
        assert fn(None, None) == m.MOE_ERR_NULL


def test_new_status_strings():
    for code in (m.MOE_ERR_BAD_PAGE, m.MOE_ERR_BAD_POSITION):
        assert m.status_string(code).startswith("MOE_ERR_BAD")


# ----------------------------------------------------------------- the angles

def test_frequencies():
    f, g = m.rope_frequencies(8, base=10000.0)
    assert g == 1.0 and f == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-14)
    f4, _ = m.rope_frequencies(8, scaling={"kind": "linear", "factor": 4})
    assert f4 == pytest.approx([x / 4 for x in f], rel=1e-14)
    # ntk: the fastest pair keeps its angle, the slowest gets the factor's share
    fn, _ = m.rope_frequencies(64, scaling={"kind": "ntk", "factor": 8})
    f1, _ = m.rope_frequencies(64)
    assert fn[0] == f1[0] and fn[-1] == pytest.approx(f1[-1] / 8, rel=1e-12)


def test_yarn_and_llama3_ends():
    R, s = 128, 8.0
    f, _ = m.rope_frequencies(R)
    y, g = m.rope_frequencies(R, scaling={"kind": "yarn", "factor": s, "original": 4096})
    assert g == pytest.approx(0.1 * math.log(s) + 1)
    assert m.rope_frequencies(R, scaling={"kind": "yarn", "factor": s, "original": 4096, "mscale": 1})[1] == 1.0
    l3, _ = m.rope_frequencies(R, scaling={"kind": "llama3", "factor": s, "original": 4096})
    for x, a, b in zip(f, y, l3):
        turns = 4096 * x / (2 * math.pi)
        assert x / s * (1 - 1e-12) <= a <= x * (1 + 1e-12)      # between divided and kept
        if turns > 40:
            assert a == x
        if turns < 0.8:
            assert a == pytest.approx(x / s)
        if turns >= 4:
            assert b == x
        elif turns <= 1:
            assert b == pytest.approx(x / s)
        else:
            assert b == pytest.approx(x / s + (x - x / s) * (turns - 1) / 3)
    assert sorted(y, reverse=True) == y


@pytest.mark.parametrize("bad", [dict(rotary_dim=7), dict(rotary_dim=0),
                                 dict(rotary_dim=8, scaling={"kind": "warp"}),
                                 dict(rotary_dim=8, scaling={"kind": "linear", "factor": 0}),
                                 dict(rotary_dim=8, scaling={"kind": "linear", "factr": 2})])
def test_frequency_refusals(bad):
    with pytest.raises(ValueError):
        m.rope_frequencies(**bad)


def test_table_far_positions():
    """The last of a million positions is as exact as the first."""
    t = m.rope_table(1 << 20, 4)
    p = (1 << 20) - 1
    want = [math.cos(p), math.cos(p * 0.01), math.sin(p), math.sin(p * 0.01)]
    np.testing.assert_allclose(t[p].numpy(), want, atol=2.0 ** -24, rtol=0)


# ------------------------------------------------------------ the oracle's pins

def test_oracle_e4m3_against_torch():
    import torch
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(ao.E4M3_VALUES, v)
    rng = np.random.default_rng(0)
    fine = ao.E4M3_VALUES[:0x7F]
    x = np.concatenate([rng.standard_normal(4096) * 10.0 ** rng.uniform(-4, 2.2, 4096), (fine[1:] + fine[:-1]) / 2, fine, -fine])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ao.e4m3_encode(x), want)
    assert ao.e4m3_encode([1e9, -np.inf, np.nan]).tolist() == [0x7E, 0xFE, 0x7F]


def test_oracle_page_scale():
    assert ao.page_scale(0.0) == 2.0 ** -42
    assert ao.page_scale(448.0) == 1.0 and ao.page_scale(np.nextafter(448.0, 1e9)) == 2.0
    assert ao.page_scale(447.0) == 1.0 and ao.page_scale(224.0) == 0.5


def test_oracle_rotation_keeps_products_of_equal_distance():
    """q at i and k at j: the product depends on i - j alone, and the inverse
    undoes the rotation."""
    rng = np.random.default_rng(1)
    f, _ = m.rope_frequencies(16)
    q, k = rng.standard_normal((2, 1, 24))
    for inter in (False, True):
        dots = [(ao.rotate(q, i, f, interleaved=inter) * ao.rotate(k, i - 5, f, interleaved=inter)).sum()
                for i in (5, 17, 900)]
        np.testing.assert_allclose(dots, dots[0], rtol=1e-12)
        back = ao.rotate(ao.rotate(q, 77, f, interleaved=inter), 77, f, interleaved=inter, inverse=True)
        np.testing.assert_allclose(back, q, rtol=1e-12)
        assert (ao.rotate(q, 3, f, interleaved=inter)[:, 16:] == q[:, 16:]).all()


def test_oracle_attention_special_cases():
    """Equal keys give the mean of the values; one key gives its value; no key
    gives zero; torch's own softmax agrees."""
    import torch
    rng = np.random.default_rng(2)
    kc = np.broadcast_to(ao.e4m3_encode(rng.standard_normal(16)), (3, 1, 8, 16)).copy()
    vc = ao.e4m3_encode(rng.standard_normal((3, 1, 8, 16)))
    one = np.ones((3, 1), np.float32)
    q = rng.standard_normal((3, 2, 16))
    table, lens, cu = [[2, 0], [1, -1], [-1, -1]], [11, 1, 0], [0, 1, 2, 3]
    out, lse, _, _ = ao.attend(q, kc, vc, one, one, table, lens, cu, 0.25)
    v = ao.E4M3_VALUES[vc]
    np.testing.assert_allclose(out[0], np.broadcast_to(np.concatenate([v[2, 0], v[0, 0, :3]]).mean(0), (2, 16)))
    np.testing.assert_allclose(out[1], np.broadcast_to(v[1, 0, 0], (2, 16)))
    assert (out[2] == 0).all() and (lse[2] == -np.inf).all()
    kc = ao.e4m3_encode(rng.standard_normal((3, 1, 8, 16)))
    ks = np.array([[0.5], [2.0], [1.0]], np.float32)
    out, lse, _, _ = ao.attend(q[:1], kc, vc, ks, one, [[1, 2]], [13], [0, 1], 0.25, window=9)
    k = np.concatenate([ao.E4M3_VALUES[kc[1, 0]] * 2.0, ao.E4M3_VALUES[kc[2, 0]]])[4:13]
    vv = np.concatenate([v[1, 0], v[2, 0]])[4:13]
    s = torch.from_numpy(q[0] @ k.T * 0.25)
    np.testing.assert_allclose(out[0], torch.softmax(s, -1).numpy() @ vv, rtol=1e-12)
    np.testing.assert_allclose(lse[0], torch.logsumexp(s, -1).numpy(), rtol=1e-12)
