"""Attention with a window and lasting first tokens, and of batches that share
prefixes, against the float64 oracle.

Bounds as in test_gpu_attention (weights round to float16, scores are float32
sums).  A joined row adds factors 2^(m - m') of the two parts, each off by 2^-22
relative, which the 2^-17 of the probabilities' errors holds many times.
"""
import importlib.util
import os

import numpy as np
import pytest

import moe_lora_expert_gb300 as m
from oracle import attention_oracle as ao
from test_gpu_attention import ATTENDS, HALF_STEP, Batch, f64, rounded, tensor, torch_mod

pytestmark = pytest.mark.gpu


def compare(got, lgot, batch, q, dtype, table=None, scale=None, **kw):
    scale = batch.D ** -0.5 if scale is None else scale
    ref, lref, spread, size = ao.attend(q, *batch.codes, *batch.scales, batch.table if table is None else table, batch.lens, batch.cu, scale, **kw)
    es = 128 * 2.0 ** -22 * size
    bound = (2.0 ** -11 + 4 * es[..., None] + 2.0 ** -17) * spread + 2.0 ** -22 * 448 * batch.scales[1].max() + 1.01 * HALF_STEP[dtype] * np.abs(ref)
    got, lgot = f64(got), f64(lgot)
    empty = np.isneginf(lref)
    assert (got[empty] == 0).all() and np.isneginf(lgot[empty]).all()
    err = np.abs(got - ref)
    assert (err <= bound).all(), (float((err - bound).max()), np.unravel_index((err - bound).argmax(), err.shape))
    lerr = np.abs(lgot[~empty] - lref[~empty])
    assert (lerr <= es[~empty] + 2.0 ** -20 * (1 + np.abs(lref[~empty]))).all(), float(lerr.max())


# ----------------------------------------------------------------------- sinks

WINDOWS = [(1, 1), (5, 3), (16, 16), (40, 64), (70, 200), (128, 1), (33, 1000), (300, 130)]


def unseen_pages(batch, window, sinks):
    """The block table with entries that no row looks at out of the cache."""
    table = batch.table.copy()
    for b, (n, e) in enumerate(zip(batch.new, batch.lens)):
        first = max(0, e - n - window + 1)
        for page in range(table.shape[1]):
            if page * batch.P >= sinks and (page + 1) * batch.P <= first:
                table[b, page] = 1 << 30
    return table


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("new,lens,Hkv,Hq,P,D", ATTENDS)
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_sinks(dtype, new, lens, Hkv, Hq, P, D, window, sinks):
    rng = np.random.default_rng(P * D + sum(lens) + window + sinks)
    batch = Batch(rng, new, lens, Hkv, P, D, tokens_first=sinks % 2 == 0, std=0.5)
    q = rounded(rng, (sum(new), Hq, D), dtype)
    table = unseen_pages(batch, window, sinks)
    decode = all(n == 1 for n in new)
    out, lse = batch.cache.attend(tensor(q, dtype, (1, 8)), tensor(table, "int32"), batch.dev["seq_lens"], cu_q=None if decode else batch.cu_dev,
                                  max_q_len=max(new), window=window, sinks=sinks, return_lse=True)
    compare(out, lse, batch, q, dtype, window=window, sinks=sinks)
    assert batch.cache.device_status() == m.MOE_OK


@pytest.mark.parametrize("new,lens,window,sinks", [([1], [60000], 9001, 700), ([3, 1], [40000, 70], 300, 17), ([150], [20000], 4000, 260),
                                                   ([40, 200], [9000, 201], 129, 127), ([1, 1], [30000, 4000], 1 << 20, 5)])
@pytest.mark.parametrize("Hkv,Hq,D", [(1, 4, 64), (2, 16, 128)])
def test_sinks_on_long_contexts(new, lens, window, sinks, Hkv, Hq, D):
    """Rows whose keys several CTAs have, far from their sinks."""
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(51)
    P, B, N = 32, len(new), sum(new)
    width = -(-max(lens) // P)
    shape = (B * width, Hkv, P, D)
    k, v = ((torch.randn(shape, generator=gen, device="cuda") * 40).to(torch.float8_e4m3fn) for _ in range(2))
    cache = m.PagedKVCache(k.view(torch.uint8), v.view(torch.uint8), *[torch.full(shape[:2], 2.0 ** -6, device="cuda") for _ in range(2)])
    table = torch.randperm(B * width, generator=gen, device="cuda").to(torch.int32).view(B, width)
    q = torch.randn((N, Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
    cu = np.cumsum([0] + new)
    out, lse = cache.attend(q, table, tensor(np.array(lens, np.int32), "int32"), cu_q=tensor(cu.astype(np.int32), "int32"), max_q_len=max(new),
                            window=window, sinks=sinks, return_lse=True)
    for b, (n, e) in enumerate(zip(new, lens)):
        pages = table[b, :-(-e // P)].long()
        kk, vv = (x[pages].double().transpose(0, 1).flatten(1, 2)[:, :e] * 2.0 ** -6 for x in (k, v))
        at, key = torch.arange(e - n, e, device="cuda")[:, None], torch.arange(e, device="cuda")[None]
        hidden = (key > at) | ((key <= at - window) & (key >= sinks))
        for h in range(Hq):
            row = q[cu[b]:cu[b + 1], h].double()
            s = (row @ kk[h * Hkv // Hq].T * D ** -0.5).masked_fill(hidden, -np.inf)
            p = torch.softmax(s, -1)
            ref, spread = p @ vv[h * Hkv // Hq], p @ vv[h * Hkv // Hq].abs()
            es = 128 * 2.0 ** -22 * D ** -0.5 * (row.abs() @ kk[h * Hkv // Hq].abs().T).amax(-1, keepdim=True)
            bound = (2.0 ** -11 + 4 * es + 2.0 ** -17) * spread + 2.0 ** -22 * 7 + 1.01 * 2.0 ** -8 * ref.abs()
            assert ((out[cu[b]:cu[b + 1], h].double() - ref).abs() <= bound).all()
            want = torch.logsumexp(s, -1)
            assert ((lse[cu[b]:cu[b + 1], h].double() - want).abs() <= es[:, 0] + 2.0 ** -20 * (1 + want.abs())).all()
    assert cache.device_status() == m.MOE_OK


@pytest.mark.parametrize("new,lens", [([1, 1], [300, 40]), ([90, 5], [300, 40])])
def test_sinks_that_change_nothing(new, lens):
    """No sinks, no window, and sinks that the window has anyway: the same bits."""
    torch = torch_mod()
    rng = np.random.default_rng(52)
    batch = Batch(rng, new, lens, 2, 16, 64, std=0.5)
    q = tensor(rounded(rng, (sum(new), 8, 64), "bfloat16"), "bfloat16")
    kw = dict(**batch.dev, cu_q=batch.cu_dev, max_q_len=max(new), return_lse=True)
    for window, sinks in ((0, 7), (50, 0), (400, 7), (400, 10 ** 12)):
        for a, b in zip(batch.cache.attend(q, window=window, sinks=sinks, **kw), batch.cache.attend(q, window=window, **kw)):
            assert torch.equal(a, b)
    for a, b in zip(batch.cache.attend(q, window=3, sinks=300, **kw), batch.cache.attend(q, **kw)):     # all of them
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -6 * b.abs().max()
    with pytest.raises(m.MoeError):
        batch.cache.attend(q, window=3, sinks=-1, **kw)


@pytest.mark.parametrize("new,lens,Hkv,Hq,D", [([1, 1, 1], [400, 90, 17], 2, 8, 64), ([200, 30], [500, 31], 1, 2, 128), ([7, 3], [300, 260], 2, 4, 80)])
def test_nan_in_sinks(new, lens, Hkv, Hq, D):
    """NaN values among the sinks, between them and the window, and in the
    window's hidden parts: only what a row sees touches it."""
    torch = torch_mod()
    rng = np.random.default_rng(53)
    batch = Batch(rng, new, lens, Hkv, 16, D, std=0.5)
    q = rounded(rng, (sum(new), Hq, D), "bfloat16")
    window, sinks = 60, 21
    for j, col in ((3, 1), (20, 2), (21, 3), (25, 4), (130, 5), (270, 6)):
        for b, e in enumerate(lens):
            if j < e:
                batch.codes[1][batch.table[b, j // 16], :, j % 16, col] = 0x7F
    batch.cache.v.copy_(tensor(batch.codes[1], torch.uint8))
    out, lse = batch.cache.attend(tensor(q, "bfloat16"), **batch.dev, cu_q=batch.cu_dev, max_q_len=max(new), window=window, sinks=sinks, return_lse=True)
    ref, lref = ao.attend(q, *batch.codes, *batch.scales, batch.table, batch.lens, batch.cu, D ** -0.5, window, sinks)[:2]
    np.testing.assert_array_equal(np.isnan(f64(out)), np.isnan(ref))
    assert np.isnan(ref).any() and np.abs(f64(lse) - lref).max() < 1e-2
    good = ~np.isnan(ref)
    assert np.abs(f64(out) - ref)[good].max() < 0.05 * np.abs(ref[good]).max()


def test_nan_in_many_sinks():
    """More hidden tiles with NaN than a unit notes, on both sides of the gap."""
    torch = torch_mod()
    rng = np.random.default_rng(54)
    batch = Batch(rng, [200], [4000], 1, 16, 64, std=0.5)
    q = rounded(rng, (200, 2, 64), "float16")
    table = batch.dev["block_table"]
    table[0, 1:240:13] = -1                            # a page of most of the tiles: hidden from all
    kw = dict(**batch.dev, cu_q=batch.cu_dev, return_lse=True, window=700, sinks=2500)
    clean, lse = batch.cache.attend(tensor(q, "float16"), **kw)
    host = table[0].cpu().numpy()
    want = f64(clean)
    at = np.arange(200) + 3800
    for j in range(5, 4000, 128):
        if host[j // 16] >= 0:
            batch.cache.v[int(host[j // 16]), 0, j % 16, (j // 128) % 64] = 0x7F
            want[(at >= j) & ((j > at - 700) | (j < 2500)), :, (j // 128) % 64] = np.nan
    out, lse_nan = batch.cache.attend(tensor(q, "float16"), **kw)
    np.testing.assert_array_equal(f64(out), want)
    assert torch.equal(lse, lse_nan) and batch.cache.device_status() == m.MOE_ERR_BAD_PAGE


# ------------------------------------------------------------- shared prefixes

LONG = 1 << 20   # a bound on the lengths that makes sharing worth while, whatever the lengths


class Shared(Batch):
    """Sequences whose first tokens are those of their group's first one:
    ``held`` own tokens before the new ones, after the group's lens (a sequence
    that ``strays`` is shorter than what its group shares)."""

    def __init__(self, rng, new, held, seqs, shared, Hkv, P, D, strays=(), **kw):
        torch = torch_mod()
        of = [next((g for g in range(len(shared)) if seqs[g] <= b < seqs[g + 1]), None) for b in range(len(new))]
        lens = [n + h + (0 if of[b] is None or b in strays else max(0, shared[of[b]])) for b, (n, h) in enumerate(zip(new, held))]
        super().__init__(rng, new, lens, Hkv, P, D, **kw)
        for b, g in enumerate(of):
            if g is None or b == seqs[g]:
                continue
            k, lead = min(max(0, shared[g]), lens[b]), seqs[g]
            self.table[b, :k // P] = self.table[lead, :k // P]
            if k % P:                                  # the page in which it ends is the sequence's own
                mine, first = self.table[b, k // P], self.table[lead, k // P]
                for codes, scales in zip(self.codes, self.scales):
                    codes[mine, :, :k % P], scales[mine] = codes[first, :, :k % P], scales[first]
        for t, c in zip((self.cache.k, self.cache.v), self.codes):
            t.copy_(tensor(c, torch.uint8))
        for t, s in zip((self.cache.k_scale, self.cache.v_scale), self.scales):
            t.copy_(tensor(s, "float32"))
        # whoever takes part does not look at its own entries for what is shared
        self.blind = self.table.copy()
        for b, g in enumerate(of):
            if g is not None and b != seqs[g] and b not in strays:
                self.blind[b, :max(0, shared[g]) // P] = 1 << 30
        self.dev["block_table"] = tensor(self.blind, "int32")
        self.groups = dict(shared_lens=tensor(np.array(shared, np.int32), "int32"), shared_seqs=tensor(np.array(seqs, np.int32), "int32"))


SHARED = [
    # new, held, seqs, shared, strays, Hkv, Hq, P, D
    ([1] * 8, [0, 5, 17, 40, 0, 1, 2, 3], [0, 8], [100], (), 4, 32, 16, 128),
    ([1] * 2, [0, 300], [0, 2], [64], (), 1, 4, 64, 64),
    ([1] * 9, [3, 0, 17, 200, 64, 1, 0, 9, 30], [0, 3, 3, 7, 9], [64, 50, 33, 1], (), 2, 10, 8, 80),
    ([1] * 7, [3, 4, 17, 20, 64, 1, 5], [1, 4, 6], [200, 90], (), 2, 4, 24, 96),          # the first and the last in no group
    ([4, 1, 3, 2, 4, 4], [9, 0, 70, 1, 0, 130], [0, 6], [333], (), 2, 8, 16, 64),
    ([4, 1, 0, 3, 2, 4], [9, 0, 5, 70, 1, 0], [0, 3, 6], [128, 129], (), 1, 20, 32, 128),
    ([1] * 40, list(range(0, 80, 2)), [0, 40], [270], (), 2, 8, 16, 64),                   # many rows: the other kernel
    ([1] * 40, list(range(40)), [0, 25, 40], [130, 500], (3, 30, 31), 3, 12, 40, 112),
    ([2] * 30, [7] * 30, [0, 30], [1000], (5,), 1, 16, 128, 48),
    ([1] * 6, [3, 0, 1, 40, 0, 9], [0, 2, 4, 6], [0, -5, 70], (), 2, 2, 16, 16),           # nothing shared in two of the groups
    ([8] * 5, [0, 1, 2, 3, 4], [0, 5], [77], (1,), 2, 32, 16, 128),                        # 128 rows a sequence and key head
    ([9] * 4, [0, 1, 2, 3], [0, 4], [77], (1,), 2, 32, 16, 128),                           # more: as without
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("new,held,seqs,shared,strays,Hkv,Hq,P,D", SHARED)
@pytest.mark.parametrize("bound", [False, True])
def test_shared(dtype, new, held, seqs, shared, strays, Hkv, Hq, P, D, bound):
    torch = torch_mod()
    rng = np.random.default_rng(P * D + sum(held))
    batch = Shared(rng, new, held, seqs, shared, Hkv, P, D, strays=strays, tokens_first=bound, std=0.5)
    N = sum(new)
    q = rounded(rng, (N, Hq, D), dtype)
    decode = all(n == 1 for n in new)
    most = max(sum(new[a:b]) for a, b in zip(seqs, seqs[1:])) if bound else N
    # sequences of many rows, and groups of few, are not worth the sharing: then each table row is looked at
    alone = max(new) * (Hq // Hkv) > 128 or most * (Hq // Hkv) < 32
    del_me = torch.full((N * Hq * (4 * D + 8) // 4,), float("nan"), device="cuda")       # what the partial sums' memory may hold
    del del_me
    out, lse = batch.cache.attend(tensor(q, dtype, (1, 8) if bound else None), tensor(batch.table, "int32") if alone else batch.dev["block_table"],
                                  batch.dev["seq_lens"], cu_q=None if decode else batch.cu_dev, max_q_len=max(new), return_lse=True,
                                  max_shared_q=most if bound else None, max_seq_len=LONG, **batch.groups)
    compare(out, lse, batch, q, dtype)
    assert batch.cache.device_status() == m.MOE_OK


def test_shared_by_all_and_by_none():
    """Without a list all sequences are one group; no group is plain attention;
    refusals."""
    torch = torch_mod()
    rng = np.random.default_rng(60)
    batch = Shared(rng, [1] * 6, [1, 0, 30, 4, 100, 2], [0, 6], [90], 2, 16, 64, std=0.5)
    q = rounded(rng, (6, 16, 64), "bfloat16")
    qt, lens = tensor(q, "bfloat16"), batch.groups["shared_lens"]
    out, lse = batch.cache.attend(qt, **batch.dev, shared_lens=lens, return_lse=True, max_seq_len=LONG)
    compare(out, lse, batch, q, "bfloat16")
    table = tensor(batch.table, "int32")
    none = dict(shared_lens=lens[:0], shared_seqs=batch.groups["shared_seqs"][:1])
    assert torch.equal(batch.cache.attend(qt, table, batch.dev["seq_lens"], **none), batch.cache.attend(qt, table, batch.dev["seq_lens"]))
    for bad in (dict(window=5), dict(window=5, sinks=2), dict(shared_lens=lens.expand(2).contiguous()), dict(shared_lens=lens.long()),
                dict(shared_seqs=torch.zeros(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            batch.cache.attend(qt, **batch.dev, **{"shared_lens": lens, **bad})
    with pytest.raises(ValueError):
        batch.cache.attend(qt, **batch.dev, shared_seqs=batch.groups["shared_seqs"])


def test_shared_empty_slots():
    """A decode batch of fixed size: slots without a sequence, the group's first
    among them, whose table row has the prefix's pages all the same."""
    rng = np.random.default_rng(61)
    batch = Shared(rng, [1] * 7, [1, 0, 30, 4, 100, 2, 5], [0, 4, 7], [90, 33], 2, 16, 64, std=0.5)
    for b in (0, 2, 6):
        batch.lens[b] = 0
    q = rounded(rng, (7, 16, 64), "bfloat16")
    out, lse = batch.cache.attend(tensor(q, "bfloat16"), batch.dev["block_table"], tensor(np.array(batch.lens, np.int32), "int32"), return_lse=True,
                                  max_seq_len=LONG, **batch.groups)
    compare(out, lse, batch, q, "bfloat16")
    assert (f64(out)[[0, 2, 6]] == 0).all() and batch.cache.device_status() == m.MOE_OK


@pytest.mark.parametrize("most", [0, 1, 5, 11, 12])
def test_shared_past_the_bound(most):
    """More tokens in a group than max_shared_q: those sequences read their
    keys themselves."""
    rng = np.random.default_rng(62)
    batch = Shared(rng, [3, 2, 4, 3], [1, 0, 30, 4], [0, 4], [90], 2, 16, 64, std=0.5)
    q = rounded(rng, (12, 16, 64), "bfloat16")
    out, lse = batch.cache.attend(tensor(q, "bfloat16"), tensor(batch.table, "int32"), batch.dev["seq_lens"], cu_q=batch.cu_dev, max_q_len=4,
                                  return_lse=True, max_shared_q=most, max_seq_len=LONG, **batch.groups)
    compare(out, lse, batch, q, "bfloat16")


def test_shared_bad_pages_and_groups():
    """A bad entry of the first row, a prefix past the table, lists that are out
    of order or out of range: reported or passed over, and nothing is touched
    that is not the call's."""
    torch = torch_mod()
    rng = np.random.default_rng(63)
    batch = Shared(rng, [1] * 6, [1, 0, 30, 4, 100, 2], [0, 6], [90], 2, 16, 64, std=0.5)
    q = rounded(rng, (6, 16, 64), "bfloat16")
    table = batch.blind.copy()
    table[0, 2] = batch.pages
    out, lse = batch.cache.attend(tensor(q, "bfloat16"), tensor(table, "int32"), batch.dev["seq_lens"], return_lse=True, max_seq_len=LONG,
                                  **batch.groups)
    assert batch.cache.device_status() == m.MOE_ERR_BAD_PAGE
    left = batch.table.copy()
    left[:, 2] = batch.pages                           # its keys are left out for all
    compare(out, lse, batch, q, "bfloat16", table=left)
    qt, table = tensor(q, "bfloat16"), tensor(batch.table, "int32")
    want = batch.cache.attend(qt, table, batch.dev["seq_lens"])
    for seqs, lens in (([0, -3], [90]), ([9, 12], [90]), ([0, 6], [1 << 30]), ([-5, -1, 0], [3, 3]), ([7, 0, 6], [3, 0])):
        got = batch.cache.attend(qt, table, batch.dev["seq_lens"], shared_seqs=tensor(np.array(seqs, np.int32), "int32"),
                                 shared_lens=tensor(np.array(lens, np.int32), "int32"), max_seq_len=LONG)
        assert (got.float() - want.float()).abs().max() <= 2.0 ** -6 * want.abs().max()
        batch.cache.device_status()


@pytest.mark.parametrize("B,Hkv,Hq,D,shared", [(40, 1, 8, 128, 20001), (8, 2, 8, 64, 30000), (17, 4, 32, 128, 5000)])
def test_shared_long_prefixes(B, Hkv, Hq, D, shared):
    """Prefixes that many CTAs have parts of, twice with the same bits, and
    against the same call without sharing."""
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(64)
    P, own = 64, 130
    pages, each = -(-shared // P), -(-own // P) + 1
    shape = (pages + B * each, Hkv, P, D)
    k, v = ((torch.randn(shape, generator=gen, device="cuda") * 40).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
    cache = m.PagedKVCache(k, v, *[torch.full(shape[:2], 2.0 ** -6, device="cuda") for _ in range(2)])
    order = torch.randperm(shape[0], generator=gen, device="cuda").to(torch.int32)
    whole = shared // P
    table = torch.cat([order[:whole].expand(B, whole), order[whole:whole + B * each].view(B, each)], dim=1).contiguous()
    shared = whole * P
    lens = shared + 1 + torch.randint(0, own, (B,), generator=gen, device="cuda", dtype=torch.int32)
    q = torch.randn((B, Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
    want, want_lse = cache.attend(q, table, lens, return_lse=True)
    n = torch.tensor([shared], dtype=torch.int32, device="cuda")
    out, lse = cache.attend(q, table, lens, return_lse=True, shared_lens=n)
    # both are within the derived bound of the exact row; weights of thousands of keys: far under a percent
    assert (out.float() - want.float()).abs().max() <= 0.02 * want.abs().max() and (lse - want_lse).abs().max() < 1e-3
    again, lse2 = cache.attend(q, table, lens, return_lse=True, shared_lens=n)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    for h in range(0, Hq, 3):
        kv = h * Hkv // Hq
        for b in (0, B - 1):
            e = int(lens[b])
            pg = table[b, :-(-e // P)].long()
            kk, vv = (x[pg, kv].view(torch.float8_e4m3fn).double().flatten(0, 1)[:e] * 2.0 ** -6 for x in (k, v))
            s = kk @ q[b, h].double() * D ** -0.5
            p = torch.softmax(s, 0)
            es = 128 * 2.0 ** -22 * D ** -0.5 * (kk.abs() @ q[b, h].double().abs()).max()
            ref = p @ vv
            bound = (2.0 ** -11 + 4 * es + 2.0 ** -17) * (p @ vv.abs()) + 2.0 ** -22 * 7 + 1.01 * 2.0 ** -8 * ref.abs()
            assert ((out[b, h].double() - ref).abs() <= bound).all()
            assert abs(float(lse[b, h]) - float(torch.logsumexp(s, 0))) <= float(es) + 2.0 ** -20 * (1 + abs(float(lse[b, h])))
    assert cache.device_status() == m.MOE_OK


def test_shared_rows_one_part_dominates():
    """Nearly all of the mass in the prefix, or in the sequence's own keys, at
    scores far apart: the join keeps what is there."""
    torch = torch_mod()
    for big in (0, 1):
        rng = np.random.default_rng(65 + big)
        batch = Shared(rng, [1] * 5, [1, 0, 30, 4, 100], [0, 5], [90], 1, 16, 64, std=0.5)
        q = rounded(rng, (5, 8, 64), "bfloat16")
        batch.codes[0][...] = np.where(batch.codes[0] == 0x7F, 0x7F, ao.e4m3_encode(np.full(64, 0.25)))
        j = 40 if big == 0 else 90                     # a key of the prefix, or each sequence's first own one
        for b in range(5):
            batch.codes[0][batch.table[b, j // 16], :, j % 16] = ao.e4m3_encode(np.sign(q[b, 0]) * 448)
        batch.cache.k.copy_(tensor(batch.codes[0], torch.uint8))
        out, lse = batch.cache.attend(tensor(q, "bfloat16"), **batch.dev, scale=4.0, return_lse=True, max_seq_len=LONG, **batch.groups)
        compare(out, lse, batch, q, "bfloat16", scale=4.0)


def test_forms_in_graphs():
    """Captured once, replayed with other lengths, prefixes and groups, on two
    streams at once and beside eager calls."""
    torch = torch_mod()
    made = []
    for seed, B in ((70, 6), (71, 40)):
        rng = np.random.default_rng(seed)
        half = B // 2
        a = Shared(rng, [1] * B, [5 + b % 7 for b in range(B)], [0, half, B], [90, 200], 2, 16, 64, std=0.5)
        q = tensor(rounded(rng, (B, 16, 64), "bfloat16"), "bfloat16")
        table, lens = tensor(a.table, "int32"), a.dev["seq_lens"]
        n, seqs = a.groups["shared_lens"], a.groups["shared_seqs"]

        def call(a=a, q=q, table=table, lens=lens, n=n, seqs=seqs):
            return [*a.cache.attend(q, table, lens, return_lse=True, shared_lens=n, shared_seqs=seqs, max_seq_len=LONG),
                    *a.cache.attend(q, table, lens, return_lse=True, window=20, sinks=9)]
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = call()
        made.append((graph, outs, call, lens, n))
    streams = [torch.cuda.Stream() for _ in made]
    for change in (0, 3, 40):
        for _, _, _, lens, n in made:
            lens.sub_(change).clamp_(min=0)            # some become shorter than what is shared
            n.sub_(change // 2)
        wants = [call() for _, _, call, _, _ in made]
        torch.cuda.synchronize()
        for _ in range(5):
            for (graph, *_), s in zip(made, streams):
                with torch.cuda.stream(s):
                    graph.replay()
            eager = [call() for _, _, call, _, _ in made]
            torch.cuda.synchronize()
            for (_, outs, *_), want, e in zip(made, wants, eager):
                assert all(torch.equal(o, w) for o, w in zip(outs, want)) and all(torch.equal(o, w) for o, w in zip(e, want))


def test_forms_on_a_given_stream():
    """Operands and scratch of a call on another stream are its own until it is done."""
    torch = torch_mod()
    rng = np.random.default_rng(72)
    batch = Shared(rng, [1] * 12, [5] * 12, [0, 12], [400], 2, 16, 64, std=0.5)
    q = torch.randn((12, 8, 64), device="cuda").to(torch.bfloat16)
    batch.groups["max_seq_len"] = LONG
    want = batch.cache.attend(q, **batch.dev, **batch.groups)
    want_sinks = batch.cache.attend(q, tensor(batch.table, "int32"), batch.dev["seq_lens"], window=30, sinks=4)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    batch.cache.attend(q, **batch.dev, **batch.groups, stream=side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    table, lens = tensor(batch.table, "int32"), batch.groups["shared_lens"].clone()
    out = batch.cache.attend(q, table, batch.dev["seq_lens"], shared_lens=lens, stream=side, max_seq_len=LONG)
    sinks = batch.cache.attend(q, table, batch.dev["seq_lens"], window=30, sinks=4, stream=side)
    held = (table.data_ptr(), lens.data_ptr())
    del table, lens
    taken = [torch.zeros(12 * 27, dtype=torch.int32, device="cuda") for _ in range(64)] + [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(64)]
    assert all(t.data_ptr() not in held for t in taken)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(sinks, want_sinks)


@pytest.mark.parametrize("form", ["sinks", "shared", "shared many"])
def test_forms_whose_wait_runs_out(form):
    """No key tile comes: the status says so, and the next call is right."""
    rng = np.random.default_rng(73)
    B = 40 if form == "shared many" else 8
    batch = Shared(rng, [1] * B, [5] * B, [0, B], [400], 2, 16, 64, std=0.5)
    q = rounded(rng, (B, 8, 64), "bfloat16")
    kw = dict(window=30, sinks=4) if form == "sinks" else {**batch.groups, "max_seq_len": LONG}
    args = dict(block_table=tensor(batch.table, "int32"), seq_lens=batch.dev["seq_lens"], **kw)
    batch.cache.attend(tensor(q, "bfloat16"), **args, wait_timeout_ms=20, debug_flags=m.MOE_DEBUG_STALL_ATTENTION)
    assert batch.cache.device_status() == m.MOE_ERR_DEVICE_TIMEOUT
    out, lse = batch.cache.attend(tensor(q, "bfloat16"), **args, return_lse=True)
    assert batch.cache.device_status() == m.MOE_OK
    compare(out, lse, batch, q, "bfloat16", **(kw if form == "sinks" else {}))


@pytest.mark.parametrize("where", ["key", "value", "own key", "own value", "query"])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 64), (40, 1, 128)])
def test_shared_nan(where, Hq, Hkv, D):
    """NaN codes in the prefix's last, partly filled tile and in a sequence's
    own keys, and a NaN query: what sees them has NaN, in the columns it should."""
    torch = torch_mod()
    rng = np.random.default_rng(75)
    batch = Shared(rng, [1] * 6, [1, 0, 30, 4, 100, 2], [0, 6], [150], Hkv, 16, D, std=0.5)
    q = rounded(rng, (6, Hq, D), "bfloat16")
    codes = batch.codes[0 if "key" in where else 1]
    if where == "query":
        q[3, 1, 5] = np.nan
    elif "own" in where:
        codes[batch.table[4, 170 // 16], 0, 170 % 16, 7] = 0x7F      # one of sequence 4's own
    else:
        for b in range(6):                                          # one that all share, in its page's copies too
            codes[batch.table[b, 145 // 16], 0, 145 % 16, 7] = 0xFF
    for t, c in zip((batch.cache.k, batch.cache.v), batch.codes):
        t.copy_(tensor(c, torch.uint8))
    out, lse = batch.cache.attend(tensor(q, "bfloat16"), **batch.dev, return_lse=True, max_seq_len=LONG, **batch.groups)
    with np.errstate(invalid="ignore"):
        ref, lref = ao.attend(q, *batch.codes, *batch.scales, batch.table, batch.lens, batch.cu, D ** -0.5)[:2]
    assert np.isnan(ref).any()
    np.testing.assert_array_equal(np.isnan(f64(out)), np.isnan(ref))
    np.testing.assert_array_equal(np.isnan(f64(lse)), np.isnan(lref))
    good = ~np.isnan(ref)
    assert (np.abs(f64(out) - ref)[good] < 0.05 * np.nanmax(np.abs(ref), initial=0.0)).all()


def test_forms_of_nothing():
    """No tokens, no sequences."""
    torch = torch_mod()
    rng = np.random.default_rng(76)
    batch = Batch(rng, [1], [20], 2, 16, 64)
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    none = torch.empty((0,), dtype=torch.int32, device="cuda")
    table = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    n = torch.ones((1,), dtype=torch.int32, device="cuda")
    for kw in (dict(window=5, sinks=3), dict(shared_lens=n), dict(shared_lens=n, shared_seqs=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        out, lse = batch.cache.attend(q, table, none, return_lse=True, **kw)
        assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert batch.cache.device_status() == m.MOE_OK


def test_shared_of_many_sequences_and_groups():
    """More sequences than one launch of the own pass takes, in many groups."""
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(77)
    B, P, Hkv, Hq, D, each = 600, 16, 1, 8, 64, 8
    groups = B // each
    shared, own, width = 96, 40, 9
    shape = (groups * shared // P + B * 3, Hkv, P, D)
    k, v = ((torch.randn(shape, generator=gen, device="cuda") * 40).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
    cache = m.PagedKVCache(k, v, *[torch.full(shape[:2], 2.0 ** -6, device="cuda") for _ in range(2)])
    order = torch.randperm(shape[0], generator=gen, device="cuda").to(torch.int32)
    first = order[:groups * 6].view(groups, 1, 6).expand(groups, each, 6).reshape(B, 6)
    table = torch.cat([first, order[groups * 6:].view(B, 3)], dim=1).contiguous()
    assert table.shape[1] == width
    lens = shared + 1 + torch.randint(0, own, (B,), generator=gen, device="cuda", dtype=torch.int32)
    q = torch.randn((B, Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
    want, want_lse = cache.attend(q, table, lens, return_lse=True)
    seqs = torch.arange(0, B + 1, each, dtype=torch.int32, device="cuda")
    n = torch.full((groups,), shared, dtype=torch.int32, device="cuda")
    got = [cache.attend(q, table, lens, return_lse=True, shared_lens=n, shared_seqs=seqs, max_seq_len=LONG, max_shared_q=most) for most in (None, each)]
    for out, lse in got:
        assert (out.float() - want.float()).abs().max() <= 0.02 * want.abs().max() and (lse - want_lse).abs().max() < 1e-3
    assert cache.device_status() == m.MOE_OK


def test_answers_to_one_prompt():
    """Positions of several axes, a shared prompt, a window with lasting first
    tokens and the routed MoE together, as the example serves them."""
    torch = torch_mod()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layer.py")
    spec = importlib.util.spec_from_file_location("decoder_layer_answers", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    worst, out, status = example.answers()
    # two orders of summing the same keys, rounded to bf16 between layers' parts
    assert worst < 2e-2 and status == [m.MOE_OK, m.MOE_OK] and torch.isfinite(out).all()


def test_a_decode_step_in_a_graph():
    """append with axes, attend with a shared prefix and attend with sinks in one
    captured step, replayed as lengths and positions move on."""
    torch = torch_mod()
    rng = np.random.default_rng(80)
    B, Hkv, Hq, P, D = 8, 2, 16, 16, 64
    batch = Shared(rng, [1] * B, [20 + b for b in range(B)], [0, B], [96], Hkv, P, D, std=0.5)
    table, lens, axes = tensor(batch.table, "int32"), batch.dev["seq_lens"], m.rope_axes([12, 10, 10], turns=True)
    cos_sin, n = m.rope_table(400, D, device="cuda"), batch.groups["shared_lens"]
    k, v = (tensor(rounded(rng, (B, Hkv, D), "bfloat16"), "bfloat16") for _ in range(2))
    q = tensor(rounded(rng, (B, Hq, D), "bfloat16"), "bfloat16")
    pos = tensor(np.stack([np.array(batch.lens) - 1] * 3).astype(np.int32), "int32")

    def step():
        turned = batch.cache.append(k, v, table, lens, q=q, cos_sin=cos_sin, positions=pos, axes=axes)
        return (turned, batch.cache.attend(turned, table, lens, shared_lens=n, max_seq_len=LONG), batch.cache.attend(turned, table, lens, window=30, sinks=5),
                batch.cache.attend(turned, table, lens))
    parts = (batch.cache.k, batch.cache.v, batch.cache.k_scale, batch.cache.v_scale)
    saved = [x.clone() for x in parts]
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for i in range(3):
        want = None
        for _ in range(2):                             # once eagerly, once replayed, from the same cache
            for x, s in zip(parts, saved):
                x.copy_(s)
            if want is None:
                want = [o.clone() for o in step()]
            else:
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))
        assert (want[1].float() - want[3].float()).abs().max() <= 2.0 ** -6 * want[3].abs().max()
        saved = [x.clone() for x in parts]
        lens.add_(1)
        pos.add_(torch.tensor([[1], [2], [0]], dtype=torch.int32, device="cuda"))
    assert batch.cache.device_status() == m.MOE_OK


@pytest.mark.parametrize("dtype,scale", [("bfloat16", -0.2), ("float16", -0.2), ("float16", 0.2)])
@pytest.mark.parametrize("form", ["few", "many", "sinks few", "sinks many"])
def test_forms_with_queries_of_any_strides(dtype, scale, form):
    """Negative scales; queries that are one for all heads or tokens give the
    bits of a copy of them, and the copy's are right."""
    torch = torch_mod()
    rng = np.random.default_rng(81)
    B, Hq, Hkv = (40 if "many" in form else 8), 16, 2
    new = [1] * B if "sinks" not in form or "few" in form else [5] * B
    batch = Shared(rng, new, [b % 7 for b in range(B)], [0, B], [140], Hkv, 16, 80, std=0.5)
    N = sum(new)
    kw = dict(block_table=tensor(batch.table, "int32"), seq_lens=batch.dev["seq_lens"], cu_q=batch.cu_dev, max_q_len=max(new), scale=scale, return_lse=True)
    seen = dict(window=20, sinks=9) if "sinks" in form else {}
    kw.update(seen or {**batch.groups, "max_seq_len": LONG})
    one_head = tensor(rounded(rng, (N, 1, 80), dtype), dtype).expand(N, Hq, 80)
    one_token = tensor(rounded(rng, (1, Hq, 80), dtype), dtype).expand(N, Hq, 80)
    for q in (one_head, one_token):
        out, lse = batch.cache.attend(q, **kw)
        want, want_lse = batch.cache.attend(q.contiguous(), **kw)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        compare_signed(out, lse, batch, f64(q), dtype, scale, **seen)


def compare_signed(out, lse, batch, q, dtype, scale, **seen):
    """The oracle's error terms take a positive scale: the sign goes into q."""
    compare(out, lse, batch, q * np.sign(scale), dtype, scale=abs(scale), **seen)


@pytest.mark.parametrize("B", [8, 40])
def test_shared_leaves_other_rows(B):
    """Rows behind the last sequence and past max_q_len are left as they were."""
    torch = torch_mod()
    rng = np.random.default_rng(82)
    new = [3 if b == 1 else 2 for b in range(B)]
    batch = Shared(rng, new, [b % 5 for b in range(B)], [0, B], [140], 2, 16, 64, std=0.5)
    N = sum(new) + 4
    q = rounded(rng, (N, 16, 64), "bfloat16")
    out, lse = torch.full((N, 16, 64), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((N, 16), 7.0, device="cuda")
    batch.cache.attend(tensor(q, "bfloat16"), **batch.dev, cu_q=batch.cu_dev, max_q_len=2, out=out, lse=lse, max_seq_len=LONG, **batch.groups)
    left = np.ones(N, bool)
    for a, n in zip(batch.cu, new):
        left[a:a + min(n, 2)] = False
    assert (f64(out)[left] == 7).all() and (f64(lse)[left] == 7).all() and not (f64(lse)[~left] == 7).any()
    full, full_lse = batch.cache.attend(tensor(q[:N - 4], "bfloat16"), **batch.dev, cu_q=batch.cu_dev, max_q_len=3, return_lse=True, max_seq_len=LONG,
                                        **batch.groups)
    compare(full, full_lse, batch, q[:N - 4], "bfloat16")
    assert np.abs(f64(lse)[~left] - f64(full_lse)[~left[:N - 4]]).max() < 1e-3


def test_shared_scales_of_any_size():
    """Pages whose key and value scales differ by many powers of two, and value
    scales of zero: each part's reference follows its own."""
    torch = torch_mod()
    rng = np.random.default_rng(83)
    batch = Shared(rng, [1] * 8, [30 + b for b in range(8)], [0, 8], [300], 2, 16, 64, std=0.5)
    for part in batch.scales:
        part *= np.exp2(rng.integers(-6, 7, part.shape)).astype(np.float32)
        part[batch.table[1:, 300 // 16]] = part[batch.table[0, 300 // 16]]     # the copies of the page in which the prefix ends
    batch.scales[1][batch.table[0, 3]] = 0.0           # one of the shared pages
    for t, s in zip((batch.cache.k_scale, batch.cache.v_scale), batch.scales):
        t.copy_(tensor(s, "float32"))
    q = rounded(rng, (8, 16, 64), "bfloat16")
    out, lse = batch.cache.attend(tensor(q, "bfloat16"), **batch.dev, scale=0.02, return_lse=True, max_seq_len=LONG, **batch.groups)
    compare(out, lse, batch, q, "bfloat16", scale=0.02)
