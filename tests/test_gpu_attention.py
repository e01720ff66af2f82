"""moe_rope, moe_kv_append and moe_paged_attention against the float64 oracle.

Bounds, with u = 2^-24 and half an output step h = 2^-8 (bf16, 8 significant
bits) or 2^-11 (f16, 11 bits) of the value (float32: u):
  rotation: two products and a sum in float32 on table values that are off by
    u: |error| <= 4 u (|x_a| + |x_b|) m, then the output's rounding.
  codes: the code of some value within that error of the float64 one.
  attention: the probabilities may be rounded to float16 (2^-11 of each, and
    2^-25 where they are subnormal) and the scores' error e_s = 128 * 2^-22 *
    max_j sum_d |q_d k_jd| scale changes each by a factor exp(2 e_s); values
    are exact.  So |error| <= (2^-11 + 4 e_s + 2^-17) sum_j p_j |v_j| + 2^-22
    max |v| + h |out|.
  lse: e_s + 2^-20 (1 + |lse|).
"""
import numpy as np
import pytest

import moe_lora_expert_gb300 as m
from oracle import attention_oracle as ao

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF_STEP = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11, "float32": U}


def torch_mod():
    import torch
    return torch


def tensor(a, dtype, pad=None):
    """``a`` on the GPU; ``pad``: as a view into a larger tensor (other strides)."""
    torch = torch_mod()
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda", getattr(torch, dtype) if isinstance(dtype, str) else dtype)
    if pad is None:
        return t
    N, H, D = t.shape
    big = torch.full((N, H + pad[0], D + pad[1]), float("nan"), dtype=t.dtype, device="cuda")
    big[:, :H, :D] = t
    return big[:, :H, :D]


def rounded(rng, shape, dtype, std=1.0):
    torch = torch_mod()
    x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * np.float32(std))
    return x.to(getattr(torch, dtype)).to(torch.float64).numpy()


def f64(t):
    return t.to(torch_mod().float64).cpu().numpy()


# ---------------------------------------------------------------------- rope

def rope_reference(x, pos, f, mscale, inter, inverse):
    return np.stack([ao.rotate(x[t], int(pos[t]), f, mscale, inter, inverse) for t in range(len(pos))])


def rope_bound(x, R, mscale, inter, ref, dtype):
    pair = np.zeros_like(x)
    a, b = (np.arange(0, R, 2), np.arange(1, R, 2)) if inter else (np.arange(R // 2), np.arange(R // 2, R))
    s = np.abs(x[..., a]) + np.abs(x[..., b])
    pair[..., a] = pair[..., b] = s
    return 4 * U * mscale * pair + HALF_STEP[dtype] * np.abs(ref) * 1.01 + 2.0 ** -25


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("N,Hq,Hk,D,R", [(1, 1, 0, 2, 2), (3, 4, 1, 128, 128), (5, 32, 4, 128, 64), (7, 3, 3, 80, 32),
                                         (2, 2, 1, 80, 40), (4, 5, 2, 96, 20), (3, 2, 2, 66, 6), (1, 70, 70, 256, 256)])
@pytest.mark.parametrize("inter,inverse,pad", [(False, False, None), (True, False, (1, 8)), (False, True, (0, 2)),
                                               (True, True, None)])
def test_rope(dtype, N, Hq, Hk, D, R, inter, inverse, pad):
    torch = torch_mod()
    rng = np.random.default_rng(N * 1000 + D + R)
    scaling = {"kind": "yarn", "factor": 4.0, "original": 1024}
    f, ms = m.rope_frequencies(R, scaling=scaling)
    table = m.rope_table(5000, R, scaling=scaling, device="cuda")
    q, k = rounded(rng, (N, Hq, D), dtype), rounded(rng, (N, Hk, D), dtype)
    pos = rng.integers(0, 5000, N).astype(np.int32)
    qt, kt = tensor(q, dtype, pad), tensor(k, dtype, pad) if Hk else None
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = m.moe_rope(qt, tensor(pos, "int32"), table, k=kt, interleaved=inter, inverse=inverse, status=status)
    got = got if Hk else (got,)
    for x, y in zip((q, k), got):
        ref = rope_reference(x, pos, f, ms, inter, inverse)
        assert (np.abs(f64(y) - ref) <= rope_bound(x, R, ms, inter, ref, dtype)).all()
        assert (f64(y)[..., R:] == x[..., R:]).all()
    assert status[0].item() == m.MOE_OK
    # in place gives the same bits
    same = m.moe_rope(qt, tensor(pos, "int32"), table, interleaved=inter, inverse=inverse, q_out=qt)
    assert same is qt and torch.equal(same, got[0])


def test_rope_gradient_against_differences():
    """d/dx of sum(w * rope(x)) by central differences is the inverse rotation
    of w; the map is linear, so float32 differences are exact but for rounding."""
    rng = np.random.default_rng(5)
    N, H, D, R = 3, 2, 24, 16
    table = m.rope_table(100, R, scaling={"kind": "yarn", "factor": 2.0, "original": 64}, device="cuda")
    pos = tensor(np.array([0, 7, 99], dtype=np.int32), "int32")
    x, w = rng.standard_normal((2, N, H, D)).astype(np.float32)
    for inter in (False, True):
        grad = f64(m.moe_rope(tensor(w, "float32"), pos, table, interleaved=inter, inverse=True))
        for at in [(0, 0, 3), (1, 1, 0), (2, 0, 15), (2, 1, 9), (1, 0, 20)]:
            d = np.zeros_like(x)
            d[at] = 0.5
            up, down = (f64(m.moe_rope(tensor(x + s * d, "float32"), pos, table, interleaved=inter)) for s in (1, -1))
            # each of the two affected outputs is off by 4 u (|x_a| + |x_b| + 1) at most
            assert abs(((up - down) * w).sum() - grad[at]) <= 64 * U * (1 + np.abs(x).max()) * np.abs(w).max()


def test_rope_bad_positions():
    torch = torch_mod()
    rng = np.random.default_rng(3)
    q = rounded(rng, (4, 2, 64), "bfloat16")
    table = m.rope_table(10, 64, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = f64(m.moe_rope(tensor(q, "bfloat16"), tensor(np.array([3, -1, 10, 9], np.int32), "int32"), table, status=status))
    assert status[0].item() == m.MOE_ERR_BAD_POSITION
    assert (got[1] == q[1]).all() and (got[2] == q[2]).all()
    assert (got[0] != q[0]).any() and (got[3] != q[3]).any()


# -------------------------------------------------------------------- append

class Batch:
    """Sequences of ``new`` tokens ending at ``lens``, on pages in any order."""

    def __init__(self, rng, new, lens, Hkv, P, D, spare=3, tokens_first=False, std=1.0):
        torch = torch_mod()
        self.new, self.lens, self.Hkv, self.P, self.D = new, lens, Hkv, P, D
        need = [-(-n // P) for n in lens]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        width = max(need + [1]) + 1
        self.table = np.full((len(lens), width), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cu = np.cumsum([0] + list(new)).astype(np.int32)
        shape = (self.pages, Hkv, P, D)
        codes = [ao.e4m3_encode(rng.standard_normal(shape) * std * 100) for _ in range(2)]
        self.scales = [np.exp2(rng.integers(-9, -5, shape[:2])).astype(np.float32) for _ in range(2)]
        # what no row may look at: NaN codes past each sequence's end and on the spare pages
        for c in codes:
            used = np.zeros((self.pages, P), bool)
            for b, n in enumerate(lens):
                for j in range(n):
                    used[self.table[b, j // P], j % P] = True
            c.transpose(0, 2, 1, 3)[~used] = 0x7F
        self.codes = codes
        dev = [tensor(c.transpose(0, 2, 1, 3), torch.uint8).transpose(1, 2) if tokens_first else tensor(c, torch.uint8)
               for c in codes]
        self.cache = m.PagedKVCache(*dev, *[tensor(s, "float32") for s in self.scales])
        self.dev = dict(block_table=tensor(self.table, "int32"), seq_lens=tensor(np.array(lens, np.int32), "int32"))
        self.cu_dev = tensor(self.cu, "int32")


def append_reference(batch, x, err, which):
    """Checks the cache's codes and scales of ``which`` (0: k, 1: v) against
    the definition, given each element's value x [N, Hkv, D] and its error."""
    got_c = (batch.cache.k, batch.cache.v)[which].cpu().numpy()
    got_s = (batch.cache.k_scale, batch.cache.v_scale)[which].cpu().numpy()
    codes, scales = batch.codes[which], batch.scales[which]
    want_c, want_s = codes.copy(), scales.copy()
    P = batch.P
    for b, (n, e) in enumerate(zip(batch.new, batch.lens)):
        p = e - n
        while p < e:
            page, off = batch.table[b, p // P], p % P
            k = min(P - off, e - p)
            t = batch.cu[b] + p - (e - n)
            for h in range(batch.Hkv):
                y, ey = x[t:t + k, h], err[t:t + k, h]
                lo, hi = (ao.page_scale(np.abs(y).max() * (1 + g) + g2) for g, g2 in ((0, -ey.max()), (0, ey.max())))
                s_old = scales[page, h] if off else 0.0
                s = got_s[page, h]
                assert max(lo, s_old) <= s <= max(hi, s_old)
                want_s[page, h] = s
                a, z = ao.E4M3_VALUES[ao.e4m3_encode((y - ey) / s)], ao.E4M3_VALUES[ao.e4m3_encode((y + ey) / s)]
                v = ao.E4M3_VALUES[got_c[page, h, off:off + k]]
                assert ((a <= v) & (v <= z)).all()
                want_c[page, h, off:off + k] = got_c[page, h, off:off + k]
                if off and s != s_old:
                    want_c[page, h, :off] = ao.e4m3_encode(ao.E4M3_VALUES[codes[page, h, :off]] * (s_old / s))
            p += k
    np.testing.assert_array_equal(got_s, want_s)       # nothing else has changed
    assert ((got_c == want_c) | ((got_c | 0x80) == 0x80) & ((want_c | 0x80) == 0x80)).all()


APPENDS = [
    # new, lens, Hkv, Hq, P, D, R, interleaved
    ([1, 1, 1, 1], [1, 16, 17, 40], 4, 32, 16, 128, 128, False),
    ([1, 1], [250, 300], 1, 0, 128, 64, 64, True),
    ([5, 40, 1, 0, 33], [5, 77, 30, 9, 33], 2, 6, 16, 128, 64, False),
    ([100, 3], [107, 3], 3, 3, 24, 80, 48, True),
    ([70], [200], 2, 4, 48, 96, 40, False),
    ([19, 64], [19, 64], 5, 5, 8, 16, 6, False),
    ([300], [301], 1, 2, 256, 128, 128, False),
    ([9, 2], [30, 12], 2, 2, 64, 112, 0, False),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("new,lens,Hkv,Hq,P,D,R,inter", APPENDS)
@pytest.mark.parametrize("tokens_first,pad", [(False, None), (True, (1, 8)), (False, (0, 1))])
def test_append(dtype, new, lens, Hkv, Hq, P, D, R, inter, tokens_first, pad):
    rng = np.random.default_rng(P * D + sum(lens))
    batch = Batch(rng, new, lens, Hkv, P, D, tokens_first=tokens_first)
    N = sum(new)
    k, v, q = (rounded(rng, (N, h, D), dtype, s) for h, s in ((Hkv, 3.0), (Hkv, 0.7), (Hq, 1.0)))
    k[N // 2] *= 4.0                                    # a token that raises its page's scale
    f, ms = m.rope_frequencies(R, scaling={"kind": "yarn", "factor": 2.0, "original": 128}) if R else ([], 1.0)
    table = m.rope_table(400, R, scaling={"kind": "yarn", "factor": 2.0, "original": 128}, device="cuda") if R else None
    pos = np.concatenate([np.arange(e - n, e) for n, e in zip(new, lens)]).astype(int)
    decode = all(n == 1 for n in new)
    got = batch.cache.append(tensor(k, dtype, pad), tensor(v, dtype, pad), **batch.dev,
                             cu_q=None if decode else batch.cu_dev, max_q_len=max(new),
                             q=tensor(q, dtype, pad) if Hq else None, cos_sin=table, interleaved=inter)
    kr = rope_reference(k, pos, f, ms, inter, False)
    err = rope_bound(k, R, ms, inter, np.zeros_like(kr), dtype) if R else np.zeros_like(kr)
    append_reference(batch, kr, err, 0)
    append_reference(batch, v, np.zeros_like(v), 1)
    if Hq:
        qr = rope_reference(q, pos, f, ms, inter, False)
        assert (np.abs(f64(got) - qr) <= (rope_bound(q, R, ms, inter, qr, dtype) if R else 0)).all()
    assert batch.cache.device_status() == m.MOE_OK


def test_append_given_positions_and_token_by_token():
    """Positions of the caller's choice; and a chunk appended at once leaves
    the values that the same tokens one by one leave, to the codes' step."""
    rng = np.random.default_rng(8)
    new, lens = [37], [37]
    table = m.rope_table(4000, 64, device="cuda")
    f, _ = m.rope_frequencies(64)
    k, v = (rounded(rng, (37, 2, 64), "bfloat16") for _ in range(2))
    k *= np.linspace(0.1, 3.0, 37)[:, None, None]       # scales grow along the page
    k = rounded_like(k)
    pos = rng.integers(0, 4000, 37)
    once = Batch(np.random.default_rng(1), new, lens, 2, 16, 64)
    once.cache.append(tensor(k, "bfloat16"), tensor(v, "bfloat16"), **once.dev, cu_q=once.cu_dev, cos_sin=table,
                      positions=tensor(pos.astype(np.int32), "int32"))
    kr = rope_reference(k, pos, f, 1.0, False, False)
    append_reference(once, kr, rope_bound(k, 64, 1.0, False, np.zeros_like(kr), "bfloat16"), 0)
    step = Batch(np.random.default_rng(1), new, lens, 2, 16, 64)
    for t in range(37):
        step.cache.append(tensor(k[t:t + 1], "bfloat16"), tensor(v[t:t + 1], "bfloat16"), step.dev["block_table"],
                          tensor(np.array([t + 1], np.int32), "int32"), cos_sin=table,
                          positions=tensor(pos[t:t + 1].astype(np.int32), "int32"))
    for a, b, sa, sb in ((once.cache.k, step.cache.k, once.cache.k_scale, step.cache.k_scale),
                         (once.cache.v, step.cache.v, once.cache.v_scale, step.cache.v_scale)):
        np.testing.assert_array_equal(f64(sa), f64(sb))
        a, b = a.cpu().numpy(), b.cpu().numpy()
        va, vb = ao.E4M3_VALUES[a], ao.E4M3_VALUES[b]
        small = np.abs(va) < 2.0 ** -6                   # only what became subnormal was rounded twice
        both = ~np.isnan(va)
        assert (va == vb)[both & ~small].all()
        assert (np.abs(va - vb)[both] <= 2.0 ** -9).all()


@pytest.mark.parametrize("D,R,inter", [(128, 128, False), (80, 48, True), (64, 64, True), (48, 8, False)])
def test_append_codes_of_unfused_products(D, R, inter):
    """Keys get the codes that float32 with every product rounded gives, ties included."""
    torch = torch_mod()
    N, H, P = 4096, 4, 64
    gen = torch.Generator(device="cuda").manual_seed(20)
    k, v = (torch.randn((N, H, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    table = m.rope_table(N, R, device="cuda")
    cache = m.PagedKVCache.create(N // P, H, P, D)
    pages = torch.randperm(N // P, generator=gen, device="cuda").to(torch.int32)
    cache.append(k, v, pages[None], tensor(np.array([N], np.int32), "int32"), cu_q=tensor(np.array([0, N], np.int32), "int32"),
                 max_q_len=N, cos_sin=table, interleaved=inter)
    cos, sin = table[:, None, :].split(R // 2, dim=-1)
    x = k.float()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if inter else (x[..., :R // 2], x[..., R // 2:R])
    u, w = a * cos - b * sin, b * cos + a * sin
    x[..., :R] = torch.stack([u, w], dim=-1).flatten(-2) if inter else torch.cat([u, w], dim=-1)
    for got, scale, want in ((cache.k, cache.k_scale, x), (cache.v, cache.v_scale, v.float())):
        want = want.view(N // P, P, H, D).transpose(1, 2) / scale[pages.long()][:, :, None, None]
        assert torch.equal(got[pages.long()], want.to(torch.float8_e4m3fn).view(torch.uint8))


def rounded_like(x):
    torch = torch_mod()
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).to(torch.float64).numpy()


def test_append_special_values():
    """NaN, infinities and zeros: each in its own element."""
    batch = Batch(np.random.default_rng(0), [2], [2], 1, 8, 16)
    x = np.zeros((2, 1, 16), np.float32)
    x[0, 0, :4] = [np.nan, 1.0, -2.0, 448.0]
    zero = np.zeros_like(x)
    batch.cache.append(tensor(x, "bfloat16"), tensor(zero, "bfloat16"), **batch.dev, cu_q=batch.cu_dev)
    pg = batch.table[0, 0]
    k = ao.E4M3_VALUES[batch.cache.k.cpu().numpy()[pg, 0, 0]] * batch.cache.k_scale[pg, 0].item()
    assert np.isnan(k[0]) and k[1:4].tolist() == [1.0, -2.0, 448.0] and (k[4:] == 0).all()
    assert (batch.cache.v.cpu().numpy()[pg, 0, :2] == 0).all() and batch.cache.v_scale[pg, 0].item() == 2.0 ** -42
    x[1, 0, 0] = -np.inf
    batch.cache.append(tensor(x, "bfloat16"), tensor(zero, "bfloat16"), **batch.dev, cu_q=batch.cu_dev)
    assert batch.cache.k_scale[pg, 0].item() == 2.0 ** 120 and batch.cache.k[pg, 0, 1, 0].item() == 0xFE


def test_append_drops_what_has_no_place():
    torch = torch_mod()
    rng = np.random.default_rng(4)
    batch = Batch(rng, [4, 4], [10, 10], 2, 8, 32)
    k = tensor(rounded(rng, (8, 2, 32), "bfloat16"), "bfloat16")
    table = batch.dev["block_table"].clone()
    table[0, 1] = batch.pages                          # past the cache
    before = batch.cache.k.clone()
    batch.cache.append(k, k, table, batch.dev["seq_lens"], cu_q=batch.cu_dev)
    assert batch.cache.device_status() == m.MOE_ERR_BAD_PAGE
    assert batch.cache.device_status() == m.MOE_OK     # reading clears it
    pg0, pg1 = batch.table[0, 0], batch.table[1, 1]
    assert not torch.equal(batch.cache.k[pg0, :, 6:], before[pg0, :, 6:])
    assert not torch.equal(batch.cache.k[pg1, :, :2], before[pg1, :, :2])
    # more new tokens than the sequence is long: the last ones are kept
    lens = tensor(np.array([3, 10], np.int32), "int32")
    batch.cache.append(k, k, batch.dev["block_table"], lens, cu_q=batch.cu_dev)
    assert batch.cache.device_status() == m.MOE_ERR_BAD_POSITION
    got = ao.E4M3_VALUES[batch.cache.k[pg0, :, :3].cpu().numpy()] * f64(batch.cache.k_scale[pg0])[:, None, None]
    want = f64(k[1:4]).transpose(1, 0, 2)
    assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -4 + 2.0 ** -10 * f64(batch.cache.k_scale[pg0])[:, None, None]).all()


# ----------------------------------------------------------------- attention

def check_attention(batch, q, dtype, window=0, scale=None, decode=False, tables=None, pad=None, **kw):
    scale = batch.D ** -0.5 if scale is None else scale
    out, lse = batch.cache.attend(tensor(q, dtype, pad), **batch.dev, cu_q=None if decode else batch.cu_dev,
                                  max_q_len=max(batch.new), scale=scale, window=window, return_lse=True, **kw)
    ref, lref, spread, size = ao.attend(q, *batch.codes, *batch.scales, batch.table if tables is None else tables,
                                        batch.lens, batch.cu, scale, window)
    vmax = 448 * batch.scales[1].max()
    es = 128 * 2.0 ** -22 * size
    bound = (2.0 ** -11 + 4 * es[..., None] + 2.0 ** -17) * spread + 2.0 ** -22 * vmax + 1.01 * HALF_STEP[dtype] * np.abs(ref)
    got, lgot = f64(out), f64(lse)
    empty = np.isneginf(lref)
    assert (got[empty] == 0).all() and np.isneginf(lgot[empty]).all()
    err = np.abs(got - ref)
    assert (err <= bound).all(), (float((err - bound).max()), np.unravel_index((err - bound).argmax(), err.shape))
    lerr = np.abs(lgot[~empty] - lref[~empty])
    assert (lerr <= es[~empty] + 2.0 ** -20 * (1 + np.abs(lref[~empty]))).all(), float(lerr.max())
    return out, lse


ATTENDS = [
    # new, lens, Hkv, Hq, P, D
    ([1], [1], 1, 1, 16, 128),
    ([1, 1, 1, 1], [1, 0, 17, 200], 4, 32, 16, 128),
    ([1] * 9, [64, 63, 65, 128, 127, 129, 5, 0, 700], 2, 10, 64, 64),
    ([1, 1], [333, 1000], 1, 16, 128, 128),
    ([1, 1, 1], [41, 90, 260], 2, 40, 24, 80),          # 20 query heads to a key head
    ([4, 1, 0, 7], [100, 1, 9, 7], 2, 8, 16, 128),
    ([3, 3], [50, 3], 3, 3, 48, 96),
    ([33, 20], [33, 150], 2, 8, 32, 128),
    ([130], [130], 1, 4, 64, 64),
    ([90, 1, 61], [300, 77, 61], 1, 5, 40, 112),
    ([10], [10], 1, 8, 8, 16),
    ([65], [321], 2, 2, 256, 48),
    ([5], [3], 1, 2, 16, 32),                            # more rows than keys: the first two see nothing
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("new,lens,Hkv,Hq,P,D", ATTENDS)
@pytest.mark.parametrize("window,tokens_first,pad", [(0, False, None), (29, True, (1, 8)), (1, False, (2, 0))])
def test_attention(dtype, new, lens, Hkv, Hq, P, D, window, tokens_first, pad):
    rng = np.random.default_rng(sum(lens) + Hq * D)
    batch = Batch(rng, new, lens, Hkv, P, D, tokens_first=tokens_first, std=0.5)
    q = rounded(rng, (sum(new), Hq, D), dtype)
    decode = all(n == 1 for n in new)
    check_attention(batch, q, dtype, window=window, decode=decode, pad=pad)
    assert batch.cache.device_status() == m.MOE_OK


@pytest.mark.parametrize("new,lens", [([1, 1], [900, 40]), ([140, 3], [140, 50])])
def test_attention_extreme_scales(new, lens):
    """Large scores (one key takes all), tiny and huge value scales side by
    side, zero scales."""
    rng = np.random.default_rng(6)
    batch = Batch(rng, new, lens, 2, 16, 128, std=0.5)
    for i in range(batch.pages):
        batch.scales[1][i] = np.float32(2.0) ** rng.integers(-60, 40)
    batch.scales[1][batch.table[0, 1]] = 0.0
    batch.scales[0][batch.table[0, 0]] = 0.0
    batch.cache.k_scale.copy_(tensor(batch.scales[0], "float32"))
    batch.cache.v_scale.copy_(tensor(batch.scales[1], "float32"))
    q = rounded(rng, (sum(new), 4, 128), "bfloat16", 30.0)
    check_attention(batch, q, "bfloat16", decode=len(new) == sum(new))
    check_attention(batch, q * 0, "bfloat16", decode=len(new) == sum(new))


@pytest.mark.parametrize("new,lens,window", [([4], [40], 0), ([40, 5], [40, 64], 0), ([150], [150], 0), ([1], [100], 33),
                                             ([140], [300], 50)])
def test_attention_nan_reaches_only_the_rows_that_see_it(new, lens, window):
    """A NaN among the values, and one among the keys, of the middle new token
    touch its own and later rows inside the window, no earlier ones."""
    rng = np.random.default_rng(11)
    for which in (0, 1):
        batch = Batch(rng, new, lens, 1, 16, 128, std=0.5)
        j = lens[0] - new[0] + new[0] // 2
        where = (batch.table[0, j // 16], 0, j % 16, 77)
        q = rounded(rng, (sum(new), 4, 128), "bfloat16")
        clean, _ = batch.cache.attend(tensor(q, "bfloat16"), **batch.dev, cu_q=batch.cu_dev, max_q_len=max(new),
                                      window=window, return_lse=True)
        (batch.cache.k, batch.cache.v)[which][where] = 0xFF
        out, lse = batch.cache.attend(tensor(q, "bfloat16"), **batch.dev, cu_q=batch.cu_dev, max_q_len=max(new),
                                      window=window, return_lse=True)
        out, lse, clean = f64(out), f64(lse), f64(clean)
        seq0 = np.arange(sum(new)) < new[0]
        sees = seq0 & (np.arange(sum(new)) >= new[0] // 2)
        if window:
            sees &= np.arange(sum(new)) < new[0] // 2 + window
        assert np.array_equal(out[~sees], clean[~sees])
        if which == 1:
            assert np.isnan(out[sees][..., 77]).all()
            rest = np.delete(out[sees], 77, axis=-1)
            assert np.array_equal(rest, np.delete(clean[sees], 77, axis=-1))
            assert np.isfinite(lse).all()
        else:
            assert np.isnan(out[sees]).all() and np.isnan(lse[sees]).all() and np.isfinite(lse[~sees]).all()


def test_attention_bad_pages_are_left_out():
    rng = np.random.default_rng(12)
    for new, lens in (([1, 1], [100, 30]), ([40], [100]), ([200], [300])):
        batch = Batch(rng, new, lens, 2, 16, 64, std=0.5)
        q = rounded(rng, (sum(new), 4, 64), "float16")
        batch.table[0, 1] = batch.pages + 5
        batch.table[0, 2] = -1
        batch.dev["block_table"].copy_(tensor(batch.table, "int32"))
        check_attention(batch, q, "float16", decode=len(new) == sum(new))
        assert batch.cache.device_status() == m.MOE_ERR_BAD_PAGE


@pytest.mark.parametrize("new,P", [([1, 1], 16), ([3, 2], 8), ([40, 1], 16), ([150, 3], 64)])
def test_attention_pages_before_the_window_may_be_gone(new, P):
    """Entries of pages that no row sees any more are never looked up."""
    rng = np.random.default_rng(15)
    window, lens = 45, [400, 331]
    batch = Batch(rng, new, lens, 2, P, 64, std=0.5)
    q = rounded(rng, (sum(new), 4, 64), "bfloat16")
    whole = batch.table.copy()
    for b, (n, e) in enumerate(zip(new, lens)):
        batch.table[b, :(e - n + 1 - window) // P] = -1
    batch.dev["block_table"].copy_(tensor(batch.table, "int32"))
    check_attention(batch, q, "bfloat16", window=window, decode=max(new) == 1, tables=whole)
    assert batch.cache.device_status() == m.MOE_OK


@pytest.mark.parametrize("new", [[1, 1], [8, 5], [300, 233]])
def test_attention_timeout_is_reported(new):
    """With no key tile arriving the waits run out, the status says so, and
    the next call on the same workspace is right."""
    rng = np.random.default_rng(16)
    batch = Batch(rng, new, [300, 250], 2, 16, 128, std=0.5)
    q = rounded(rng, (sum(new), 4, 128), "bfloat16")
    decode = max(new) == 1
    batch.cache.attend(tensor(q, "bfloat16"), **batch.dev, cu_q=None if decode else batch.cu_dev, max_q_len=max(new),
                       wait_timeout_ms=5, debug_flags=m.MOE_DEBUG_STALL_ATTENTION)
    assert batch.cache.device_status() == m.MOE_ERR_DEVICE_TIMEOUT
    check_attention(batch, q, "bfloat16", decode=decode)
    assert batch.cache.device_status() == m.MOE_OK


def test_attention_many_sequences():
    """More sequences than one launch's list, empty and short ones among them."""
    rng = np.random.default_rng(17)
    lens = [int(x) for x in rng.integers(0, 40, 700)]
    batch = Batch(rng, [1] * 700, lens, 1, 8, 16, std=0.5)
    check_attention(batch, rounded(rng, (700, 2, 16), "bfloat16"), "bfloat16", decode=True)


def test_attention_repeats_bit_for_bit_and_on_streams():
    """Twice the same bits; on two streams at once, each its own workspace."""
    torch = torch_mod()
    rng = np.random.default_rng(13)
    batch = Batch(rng, [1, 1, 1], [3000, 17, 900], 2, 32, 128, std=0.5)
    q = tensor(rounded(rng, (3, 16, 128), "bfloat16"), "bfloat16")
    first = batch.cache.attend(q, **batch.dev)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        batch.cache.workspace(s.cuda_stream)
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        outs += [batch.cache.attend(q, **batch.dev, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, first) for o in outs)


@pytest.mark.parametrize("new,lens,Hq,Hkv,P,D,window", [([70], [6001], 2, 1, 16, 64, 0), ([40, 3], [3000, 2500], 8, 2, 64, 128, 0),
                                                        ([129], [4100], 4, 2, 24, 128, 1500), ([1], [20000], 2, 1, 32, 128, 0),
                                                        ([3], [9000], 6, 1, 128, 96, 0)])
def test_attention_long_contexts_are_joined(new, lens, Hq, Hkv, P, D, window):
    """Rows whose keys lie in the stretches of many CTAs; and the same bits every time."""
    torch = torch_mod()
    rng = np.random.default_rng(18)
    batch = Batch(rng, new, lens, Hkv, P, D, std=0.5)
    q = rounded(rng, (sum(new), Hq, D), "bfloat16")
    out, lse = check_attention(batch, q, "bfloat16", window=window, decode=new == [1])
    for _ in range(3):
        again = batch.cache.attend(tensor(q, "bfloat16"), **batch.dev, cu_q=None if new == [1] else batch.cu_dev, max_q_len=max(new),
                                   window=window, return_lse=True)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("new,lens,Hq,Hkv,P,D,window", [
    ([700, 1, 333, 0, 64], [700, 90, 333, 5, 400], 64, 8, 64, 64, 0),   # more units than CTAs, whole: some CTAs get two, some one
    ([1500, 40], [1500, 40], 32, 2, 32, 128, 0),                        # twice as many units as CTAs, of 1 to 12 tiles
    ([300, 300], [300, 3500], 64, 8, 48, 64, 0),                        # long and short units, cut from the line
    ([100] * 40, [100 + 7 * i for i in range(40)], 8, 2, 16, 128, 96),  # units of one size in a window
    ([2] * 449 + [40], [9] * 449 + [41], 2, 1, 16, 64, 0),              # more entries than threads
])
def test_attention_many_units(new, lens, Hq, Hkv, P, D, window):
    """More rows than the CTAs take at once, dealt out whole or cut; the same bits every time."""
    torch = torch_mod()
    rng = np.random.default_rng(19)
    batch = Batch(rng, new, lens, Hkv, P, D, std=0.5)
    q = rounded(rng, (sum(new), Hq, D), "bfloat16")
    out, lse = check_attention(batch, q, "bfloat16", window=window)
    again = batch.cache.attend(tensor(q, "bfloat16"), **batch.dev, cu_q=batch.cu_dev, max_q_len=max(new), window=window, return_lse=True)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_attention_and_append_past_32_bits():
    """Pages more than 2^32 bytes into the cache: the bits are those of a small
    cache with the same codes."""
    torch = torch_mod()
    Hkv, P, D, pages = 8, 128, 128, 33000
    assert Hkv * P * D * (pages - 5) > 2 ** 32
    big = [torch.empty((pages, Hkv, P, D), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.ones((pages, Hkv), device="cuda") for _ in range(2)]
    rng = np.random.default_rng(19)
    for new, lens in (([1, 1], [300, 150]), ([90, 5], [300, 150])):
        small = Batch(rng, new, lens, Hkv, P, D, std=0.5)
        cache = m.PagedKVCache(*big, *scales)
        shift = pages - small.pages
        for b, c in zip(big, (small.cache.k, small.cache.v)):
            b[shift:] = c
        for s, c in zip(scales, (small.cache.k_scale, small.cache.v_scale)):
            s[shift:] = c
        table = torch.where(small.dev["block_table"] >= 0, small.dev["block_table"] + shift, small.dev["block_table"])
        N = sum(new)
        q, k, v = (tensor(rounded(rng, (N, h, D), "bfloat16"), "bfloat16") for h in (16, Hkv, Hkv))
        for c, t in ((small.cache, small.dev["block_table"]), (cache, table)):
            c.append(k, v, t, small.dev["seq_lens"], cu_q=small.cu_dev, max_q_len=max(new))
        got = cache.attend(q, table, small.dev["seq_lens"], cu_q=small.cu_dev, max_q_len=max(new))
        want = small.cache.attend(q, small.dev["block_table"], small.dev["seq_lens"], cu_q=small.cu_dev, max_q_len=max(new))
        assert torch.equal(got, want) and torch.isfinite(got.float()).all()
        assert torch.equal(big[0][shift:], small.cache.k) and torch.equal(scales[1][shift:], small.cache.v_scale)
        assert cache.device_status() == m.MOE_OK


@pytest.mark.parametrize("Hq,Hkv,new,lens", [(150, 1, [2], [100]), (256, 1, [1, 3], [40, 33]), (200, 1, [30], [64])])
def test_attention_many_heads_on_one_key_head(Hq, Hkv, new, lens):
    rng = np.random.default_rng(20)
    batch = Batch(rng, new, lens, Hkv, 16, 32, std=0.5)
    check_attention(batch, rounded(rng, (sum(new), Hq, 32), "float16"), "float16")


def test_append_and_attention_in_a_graph():
    """A captured decode step replays with new lengths and tokens."""
    torch = torch_mod()
    rng = np.random.default_rng(14)
    batch = Batch(rng, [1, 1], [60, 33], 2, 16, 64, std=0.5)
    table = m.rope_table(200, 64, device="cuda")
    q, k, v = (tensor(rounded(rng, (2, h, 64), "bfloat16"), "bfloat16") for h in (8, 2, 2))
    lens = tensor(np.array([50, 20], np.int32), "int32")
    bt = batch.dev["block_table"]

    def step():
        turned = batch.cache.append(k, v, bt, lens, q=q, cos_sin=table)
        return batch.cache.attend(turned, bt, lens)

    step()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    batch.cache.workspace(side.cuda_stream)
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for _ in range(3):
        lens += 1
        k.copy_(tensor(rounded(rng, (2, 2, 64), "bfloat16"), "bfloat16"))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step())                # the same step, launched: the same bits


def test_refusals_of_the_binding():
    torch = torch_mod()
    batch = Batch(np.random.default_rng(0), [1], [5], 2, 16, 64)
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    bt, sl = batch.dev["block_table"], batch.dev["seq_lens"]
    for bad in (dict(q=q.double()), dict(q=q[..., :32]), dict(q=q.cpu()), dict(block_table=bt.long()), dict(seq_lens=sl.cpu()),
                dict(block_table=bt[0]), dict(cu_q=torch.zeros(5, dtype=torch.int32, device="cuda")),
                dict(q=torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            batch.cache.attend(**{**dict(q=q, block_table=bt, seq_lens=sl), **bad})
    with pytest.raises(m.MoeError):
        batch.cache.attend(q[:, :3], bt, sl)           # 3 query heads on 2 key heads
    with pytest.raises(ValueError):
        batch.cache.append(q, q, bt, sl)               # 4 heads into a cache of 2
    with pytest.raises(ValueError):
        m.PagedKVCache(batch.cache.k, batch.cache.v[:1], batch.cache.k_scale, batch.cache.v_scale)
    with pytest.raises(ValueError):
        m.moe_rope(q, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros((4, 64), device="cuda").half())
    with pytest.raises(ValueError):
        m.moe_rope(q.double(), torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros((4, 64), device="cuda"))


def test_decoder_layer_example():
    """Prefill and decode steps of the example's layer agree with one prefill.
    Both see the same tokens; what differs is the rounding of codes on pages
    whose scale rose later (subnormals), of bf16 intermediates and the order
    of sums: a few 2^-8 of a layer whose output is mostly its input."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layer.py")
    spec = importlib.util.spec_from_file_location("decoder_layer_example", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    worst, status = example.main()
    assert status == [m.MOE_OK, m.MOE_OK]
    assert worst < 2e-2
