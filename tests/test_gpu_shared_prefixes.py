"""Shared prefixes where the passes take their less common ways, against plain
sums in float64 on the GPU.

Bounds as in test_gpu_attention: weights round to float16 (2^-11 of what they
sum), scores are float32 sums of 128 products (es), outputs round once.
"""
import numpy as np
import pytest

import moe_lora_expert_gb300 as m
from test_gpu_attention import torch_mod

pytestmark = pytest.mark.gpu

LONG = 1 << 20   # a bound on the lengths that makes sharing worth while, whatever the lengths
HALF_STEP = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
SCALE = 2.0 ** -6


class Prefixes:
    """Groups of sequences, each with a prefix of ``shared[g]`` tokens whose whole
    pages the group's table rows have in common and whose last page, where the
    prefix ends inside one, each has as a copy; ``own[b]`` tokens follow, the
    last ``new[b]`` of them new."""

    def __init__(self, seed, sizes, shared, own, new, Hkv, Hq, D, P=64, dtype="bfloat16", std=40.0):
        torch = torch_mod()
        gen = torch.Generator(device="cuda").manual_seed(seed)
        B, rng = sum(sizes), np.random.default_rng(seed)
        self.new, self.Hkv, self.Hq, self.D, self.P, self.dtype = new, Hkv, Hq, D, P, dtype
        of = np.repeat(np.arange(len(sizes)), sizes)
        self.seqs = np.cumsum([0] + list(sizes)).astype(np.int32)
        self.lens = np.array([shared[of[b]] + own[b] for b in range(B)], np.int32)
        table, pages, copies = np.full((B, int(-(-self.lens.max() // P)) + 1), 1 << 30, np.int64), 0, []
        for b in range(B):
            g = of[b]
            lead, need, same = self.seqs[g], -(-int(self.lens[b]) // P), 0
            if b != lead:
                same = shared[g] // P
                table[b, :same] = table[lead, :same]
                if shared[g] % P:
                    copies.append((lead, b, same))
            table[b, same:need] = np.arange(pages, pages + need - same)
            pages += need - same
        order = rng.permutation(pages)
        real = table < pages
        table[real] = order[table[real]]
        shape = (pages, Hkv, P, D)
        self.k, self.v = ((torch.randn(shape, generator=gen, device="cuda") * std).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
        for lead, b, at in copies:
            for x in (self.k, self.v):
                x[table[b, at]] = x[table[lead, at]]
        self.cache = m.PagedKVCache(self.k, self.v, *[torch.full(shape[:2], SCALE, device="cuda") for _ in range(2)])
        self.table = torch.from_numpy(table.astype(np.int32)).cuda()
        self.cu = np.cumsum([0] + list(new)).astype(np.int32)
        self.q = torch.randn((int(self.cu[-1]), Hq, D), generator=gen, device="cuda").to(getattr(torch, dtype))
        self.args = dict(q=self.q, block_table=self.table, seq_lens=torch.from_numpy(self.lens).cuda(),
                         cu_q=None if max(new) == min(new) == 1 else torch.from_numpy(self.cu).cuda(), max_q_len=max(new), return_lse=True)
        self.groups = dict(shared_lens=torch.tensor(list(shared), dtype=torch.int32, device="cuda"), shared_seqs=torch.from_numpy(self.seqs).cuda(),
                           max_shared_q=int(max(sum(new[a:b]) for a, b in zip(self.seqs, self.seqs[1:]))))

    def attend(self, **over):
        return self.cache.attend(**{**self.args, **self.groups, "max_seq_len": LONG, **over})

    def check(self, out, lse, sequences=None):
        torch = torch_mod()
        G = self.Hq // self.Hkv
        for b in range(len(self.new)) if sequences is None else sequences:
            e, n = int(self.lens[b]), self.new[b]
            pg = self.table[b, :-(-e // self.P)].long()
            kk, vv = (x[pg].view(torch.float8_e4m3fn).double().transpose(0, 1).flatten(1, 2)[:, :e] * SCALE for x in (self.k, self.v))
            row = slice(int(self.cu[b]), int(self.cu[b]) + n)
            q = self.q[row].double().view(n, self.Hkv, G, self.D).permute(1, 2, 0, 3)                 # [Hkv, G, n, D]
            hidden = torch.arange(e, device="cuda")[None] > torch.arange(e - n, e, device="cuda")[:, None]
            s = (torch.einsum("hgnd,hkd->hgnk", q, kk) * self.D ** -0.5).masked_fill(hidden, -np.inf)
            es = 128 * 2.0 ** -22 * self.D ** -0.5 * torch.einsum("hgnd,hkd->hgnk", q.abs(), kk.abs()).amax(-1, keepdim=True)
            p = torch.softmax(s, -1)
            ref, spread = torch.einsum("hgnk,hkd->hgnd", p, vv), torch.einsum("hgnk,hkd->hgnd", p, vv.abs())
            bound = (2.0 ** -11 + 4 * es + 2.0 ** -17) * spread + 2.0 ** -22 * 448 * SCALE + 1.01 * HALF_STEP[self.dtype] * ref.abs()
            got = out[row].double().view(n, self.Hkv, G, self.D).permute(1, 2, 0, 3)
            assert ((got - ref).abs() <= bound).all(), (b, float(((got - ref).abs() - bound).max()))
            want, got = torch.logsumexp(s, -1), lse[row].double().view(n, self.Hkv, G).permute(1, 2, 0)
            assert ((got - want).abs() <= es[..., 0] + 2.0 ** -20 * (1 + want.abs())).all(), b


@pytest.mark.parametrize("shared", [[100] * 40, [1 + 7 * g for g in range(40)]])
def test_more_units_than_ctas(shared):
    """Pieces of one key tile or a few, several to a CTA, and more row tiles of
    the own pass than CTAs in one launch."""
    torch = torch_mod()
    sizes = [8] * 40
    batch = Prefixes(1, sizes, shared, [1 + (37 * b) % 90 for b in range(320)], [1] * 320, 4, 32, 64, P=16)
    out, lse = batch.attend()
    batch.check(out, lse)
    again = batch.attend()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]) and batch.cache.device_status() == m.MOE_OK


@pytest.mark.parametrize("chunk", [1, 3])
def test_prefixes_that_nobody_has_yet(chunk):
    """Sequences that are still in their first chunks: the rest of the prefix has
    no pages yet, which is no error, and a group that has it is served as ever."""
    torch = torch_mod()
    batch = Prefixes(2, [6, 6], [300, 300], [20] * 12, [chunk] * 12, 2, 32, 64, P=16)
    lens = batch.lens.copy()
    lens[:6] = [40, 16, 17, 3, 299, 60]
    batch.lens = lens
    table = batch.table.cpu().numpy()
    for b in range(6):
        table[b, -(-int(lens[b]) // 16):] = 1 << 30
    batch.table = torch.from_numpy(table).cuda()
    out, lse = batch.attend(block_table=batch.table, seq_lens=torch.from_numpy(lens).cuda())
    batch.check(out, lse)
    assert batch.cache.device_status() == m.MOE_OK


def test_a_table_too_wide_for_the_own_pass():
    """A call whose own keys the kernel for few rows cannot count in one line, and
    the plain call can: it does as that one."""
    torch = torch_mod()
    batch = Prefixes(3, [128], [250], [64] * 128, [64] * 128, 64, 64, 16, P=256)
    wide = torch.full((128, 16384), 1 << 30, dtype=torch.int32, device="cuda")
    wide[:, :batch.table.shape[1]] = batch.table
    batch.table = wide
    out, lse = batch.attend(block_table=wide)
    want, want_lse = batch.cache.attend(**{**batch.args, "block_table": wide})
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    batch.check(out, lse, [0, 77, 127])
    assert batch.cache.device_status() == m.MOE_OK


def test_scratch_is_taken_where_it_is_used(monkeypatch):
    """A call that is the plain one allocates what that one does; one that shares
    gives the same with the scratch that holds for whatever bounds."""
    torch = torch_mod()
    from moe_lora_expert_gb300 import attention as A
    many = Prefixes(4, [2], [64], [1024] * 2, [1024] * 2, 4, 32, 128)
    out, lse = torch.empty_like(many.q), torch.empty((2048, 32), device="cuda")

    def growth(**over):
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        many.cache.attend(**{**many.args, "return_lse": False, "out": out, "lse": lse, **over})
        return torch.cuda.max_memory_allocated() - before
    growth()                                            # the stream's workspace
    assert growth(**many.groups) == growth() == 0
    few = Prefixes(5, [8], [5000], [20] * 8, [1] * 8, 4, 32, 128)
    want = few.attend()
    monkeypatch.setattr(A, "_partial_size", lambda args, x: m.lib().moe_shared_prefix_partial_size(8, 32, 128, 1))
    assert all(torch.equal(a, b) for a, b in zip(few.attend(), want))


@pytest.mark.parametrize("shared", [20001, 29951, 29952, 29953])
@pytest.mark.parametrize("B,Hkv,Hq,D", [(8, 1, 8, 64), (5, 1, 16, 128), (20, 2, 16, 128)])
def test_long_prefixes_that_end_anywhere(B, Hkv, Hq, D, shared):
    """Prefixes in over 32 pieces that end inside a page, and one short of and one
    past a key tile; the join takes several rounds."""
    torch = torch_mod()
    batch = Prefixes(B + shared, [B], [shared], [1 + 11 * b for b in range(B)], [1] * B, Hkv, Hq, D)
    out, lse = batch.attend()
    batch.check(out, lse)
    again = batch.attend()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]) and batch.cache.device_status() == m.MOE_OK


@pytest.mark.parametrize("N", [1, 64])
def test_a_padded_batch_without_new_tokens(N):
    """Rows of no sequence alone: they are left as they were."""
    torch = torch_mod()
    batch = Prefixes(6, [8], [300], [20] * 8, [8] * 8, 2, 64, 64, P=16)
    q, cu = batch.q[:N], torch.zeros(9, dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((N, 64), 7.0, device="cuda")
    batch.attend(q=q, cu_q=cu, max_q_len=4, max_shared_q=N, out=out, lse=lse)
    assert bool((out == 7).all()) and bool((lse == 7).all()) and batch.cache.device_status() == m.MOE_OK
    out, lse = batch.attend()
    batch.check(out, lse)


@pytest.mark.parametrize("B,new,Hq", [(128, 1, 32), (80, 2, 32), (128, 1, 64)])
@pytest.mark.parametrize("shared", [129, 4000])
def test_more_row_tiles_than_ctas(B, new, Hq, shared):
    """One launch of the own pass with more (row tile, key head) pairs than CTAs,
    which then take the SMs that the prefix pass leaves: row tiles of 8 and of 16 rows."""
    batch = Prefixes(B + shared, [B], [shared], [new + (53 * b) % 700 for b in range(B)], [new] * B, 4, Hq, 64)
    out, lse = batch.attend()
    batch.check(out, lse)
    assert batch.cache.device_status() == m.MOE_OK


@pytest.mark.parametrize("Hkv,Hq,D,new", [(1, 8, 64, 1), (2, 16, 128, 1), (1, 8, 128, 2), (2, 32, 64, 4)])
@pytest.mark.parametrize("own", [[6001] + [30] * 7, [5, 2500, 40, 9, 64, 700, 1900, 4], [3000] * 2 + [5] * 6])
def test_own_keys_of_uneven_lengths(Hkv, Hq, D, new, own):
    """Sequences with far more keys of their own than the others: their row tiles
    are cut, in up to 47 pieces, and leave one piece for the join."""
    torch = torch_mod()
    batch = Prefixes(sum(own) + D, [8], [700], own, [new if n >= new else 1 for n in own], Hkv, Hq, D)
    out, lse = batch.attend()
    batch.check(out, lse)
    again = batch.attend()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1]) and batch.cache.device_status() == m.MOE_OK


def test_more_groups_than_threads():
    """Over 448 units, of which a thread of the prefix pass plans several."""
    groups = 460
    batch = Prefixes(7, [4] * groups, [1 + (29 * g) % 300 for g in range(groups)], [1 + b % 9 for b in range(4 * groups)], [1] * (4 * groups), 1, 16, 16, P=16)
    out, lse = batch.attend()
    batch.check(out, lse, range(0, 4 * groups, 7))
    assert batch.cache.device_status() == m.MOE_OK


def test_decode_with_float16_and_wide_pages():
    batch = Prefixes(8, [20, 12], [3001, 255], [1 + 13 * b for b in range(32)], [1] * 32, 2, 24, 112, P=256, dtype="float16")
    out, lse = batch.attend()
    batch.check(out, lse)
    assert batch.cache.device_status() == m.MOE_OK
