"""moe_rope and the cache's append with an axis for each pair, against the
float64 oracle.  Bounds as in test_gpu_attention: the rotation of a pair is the
same, only the table's row is another one for each axis."""
import numpy as np
import pytest

import moe_lora_expert_gb300 as m
from oracle import attention_oracle as ao
from test_gpu_attention import U, Batch, append_reference, f64, rope_bound, rounded, tensor, torch_mod

pytestmark = pytest.mark.gpu

SHAPES = [  # N, Hq, Hk, D, R, sections, turns
    (1, 1, 0, 2, 2, [1], False),
    (3, 4, 1, 128, 128, [16, 24, 24], False),
    (5, 32, 4, 128, 128, [24, 20, 20], True),
    (7, 3, 3, 80, 32, [7, 9], False),
    (2, 2, 1, 80, 40, [5, 5, 5, 5], True),
    (4, 5, 2, 96, 20, [0, 10], False),
    (3, 2, 2, 66, 6, [1, 1, 1], True),
    (2, 7, 2, 256, 256, [61, 3, 64], True),
    (2, 1, 1, 1024, 1024, [100, 200, 211, 1], True),
]


def reference(x, pos, axes, f, inter, inverse=False, mscale=1.0):
    return np.stack([ao.rotate_axes(x[t], pos[:, t], axes, f, mscale, inter, inverse) for t in range(pos.shape[1])])


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("N,Hq,Hk,D,R,sections,turns", SHAPES)
@pytest.mark.parametrize("inter,inverse,pad", [(False, False, None), (True, False, (1, 8)), (False, True, (0, 2)), (True, True, None)])
def test_rope_axes(dtype, N, Hq, Hk, D, R, sections, turns, inter, inverse, pad):
    torch = torch_mod()
    rng = np.random.default_rng(N * 1000 + D + R)
    scaling = {"kind": "yarn", "factor": 4.0, "original": 1024}
    f, ms = m.rope_frequencies(R, scaling=scaling)
    table = m.rope_table(5000, R, scaling=scaling, device="cuda")
    axes = m.rope_axes(sections, turns)
    q, k = rounded(rng, (N, Hq, D), dtype), rounded(rng, (N, Hk, D), dtype)
    pos = rng.integers(0, 5000, (len(sections), N)).astype(np.int32)
    qt, kt = tensor(q, dtype, pad), tensor(k, dtype, pad) if Hk else None
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    wide = torch.full((len(sections), N + 3), -9, dtype=torch.int32, device="cuda")     # positions as part of a wider array
    wide[:, :N] = tensor(pos, "int32")
    got = m.moe_rope(qt, wide[:, :N], table, k=kt, interleaved=inter, inverse=inverse, status=status, axes=axes)
    got = got if Hk else (got,)
    for x, y in zip((q, k), got):
        ref = reference(x, pos, axes, f, inter, inverse, ms)
        assert (np.abs(f64(y) - ref) <= rope_bound(x, R, ms, inter, ref, dtype)).all()
        assert (f64(y)[..., R:] == x[..., R:]).all()
    assert status[0].item() == m.MOE_OK
    same = m.moe_rope(qt, tensor(pos, "int32"), table, interleaved=inter, inverse=inverse, q_out=qt, axes=axes)     # in place: the same bits
    assert same is qt and torch.equal(same, got[0])


@pytest.mark.parametrize("sections,turns", [([16, 24, 24], False), ([24, 20, 20], True)])
def test_text_has_the_bits_of_one_axis(sections, turns):
    """Where a token's positions are alike, the axes change nothing; also with
    one row of positions for all axes."""
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, k = (torch.randn((50, h, 128), generator=gen, device="cuda").to(torch.bfloat16) for h in (32, 4))
    pos = torch.randint(0, 900, (50,), generator=gen, device="cuda", dtype=torch.int32)
    table, axes = m.rope_table(900, 128, device="cuda"), m.rope_axes(sections, turns)
    want = m.moe_rope(q, pos, table, k=k)
    for p in (pos.expand(3, 50), pos.expand(3, 50).contiguous()):
        got = m.moe_rope(q, p, table, k=k, axes=axes)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_tokens():
    torch = torch_mod()
    q = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    pos = torch.empty((3, 0), dtype=torch.int32, device="cuda")
    assert m.moe_rope(q, pos, m.rope_table(9, 64, device="cuda"), axes=m.rope_axes([12, 10, 10])).shape == (0, 4, 64)


def test_gradient_against_differences():
    """The map is linear: central differences of sum(w rope(x)) are exact but
    for rounding, and the inverse rotation of w is the gradient."""
    rng = np.random.default_rng(5)
    N, H, D, R = 3, 2, 24, 16
    table = m.rope_table(100, R, scaling={"kind": "yarn", "factor": 2.0, "original": 64}, device="cuda")
    axes, pos = m.rope_axes([3, 3, 2], True), tensor(np.array([[0, 7, 99], [5, 5, 1], [80, 0, 2]], dtype=np.int32), "int32")
    x, w = rng.standard_normal((2, N, H, D)).astype(np.float32)
    for inter in (False, True):
        grad = f64(m.moe_rope(tensor(w, "float32"), pos, table, interleaved=inter, inverse=True, axes=axes))
        for at in [(0, 0, 3), (1, 1, 0), (2, 0, 15), (2, 1, 9), (1, 0, 20)]:
            d = np.zeros_like(x)
            d[at] = 0.5
            up, down = (f64(m.moe_rope(tensor(x + s * d, "float32"), pos, table, interleaved=inter, axes=axes)) for s in (1, -1))
            # each of the two affected outputs is off by 4 u (|x_a| + |x_b| + 1) at most
            assert abs(((up - down) * w).sum() - grad[at]) <= 64 * U * (1 + np.abs(x).max()) * np.abs(w).max()


def test_bad_positions():
    """One axis outside the table: the whole token stays unturned."""
    torch = torch_mod()
    rng = np.random.default_rng(3)
    q = rounded(rng, (5, 2, 64), "bfloat16")
    table, axes = m.rope_table(10, 64, device="cuda"), m.rope_axes([12, 10, 10])
    pos = np.array([[3, -1, 3, 3, 9], [3, 3, 10, 3, 1], [3, 3, 3, 2 ** 30, 9]], np.int32)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    got = f64(m.moe_rope(tensor(q, "bfloat16"), tensor(pos, "int32"), table, status=status, axes=axes))
    assert status[0].item() == m.MOE_ERR_BAD_POSITION
    assert (got[1:4] == q[1:4]).all() and (got[0] != q[0]).any() and (got[4] != q[4]).any()


APPENDS = [  # new, lens, Hkv, Hq, P, D, R, interleaved, sections, turns
    ([1, 1, 1, 1], [1, 16, 17, 40], 4, 32, 16, 128, 128, False, [16, 24, 24], False),
    ([1, 1], [250, 300], 1, 0, 128, 64, 64, True, [12, 10, 10], True),
    ([5, 40, 1, 0, 33], [5, 77, 30, 9, 33], 2, 6, 16, 128, 64, False, [16, 16], True),
    ([100, 3], [107, 3], 3, 3, 24, 80, 48, True, [4, 10, 10], False),
    ([19, 64], [19, 64], 5, 5, 8, 16, 6, False, [1, 1, 1], True),
    ([70], [200], 2, 4, 48, 96, 40, False, [3, 6, 5, 6], True),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("new,lens,Hkv,Hq,P,D,R,inter,sections,turns", APPENDS)
@pytest.mark.parametrize("tokens_first,pad", [(False, None), (True, (1, 8)), (False, (0, 1))])
def test_append_axes(dtype, new, lens, Hkv, Hq, P, D, R, inter, sections, turns, tokens_first, pad):
    rng = np.random.default_rng(P * D + sum(lens))
    batch = Batch(rng, new, lens, Hkv, P, D, tokens_first=tokens_first)
    N, axes = sum(new), m.rope_axes(sections, turns)
    k, v, q = (rounded(rng, (N, h, D), dtype, s) for h, s in ((Hkv, 3.0), (Hkv, 0.7), (Hq, 1.0)))
    k[N // 2] *= 4.0                                    # a token that raises its page's scale
    f, _ = m.rope_frequencies(R)
    pos = rng.integers(0, 400, (len(sections), N)).astype(np.int32)
    decode = all(n == 1 for n in new)
    got = batch.cache.append(tensor(k, dtype, pad), tensor(v, dtype, pad), **batch.dev, cu_q=None if decode else batch.cu_dev, max_q_len=max(new),
                             q=tensor(q, dtype, pad) if Hq else None, cos_sin=m.rope_table(400, R, device="cuda"), interleaved=inter,
                             positions=tensor(pos, "int32"), axes=axes)
    kr = reference(k, pos, axes, f, inter)
    append_reference(batch, kr, rope_bound(k, R, 1.0, inter, np.zeros_like(kr), dtype), 0)
    append_reference(batch, v, np.zeros_like(v), 1)
    if Hq:
        qr = reference(q, pos, axes, f, inter)
        assert (np.abs(f64(got) - qr) <= rope_bound(q, R, 1.0, inter, qr, dtype)).all()
    assert batch.cache.device_status() == m.MOE_OK


@pytest.mark.parametrize("Hq", [2, 40])
def test_append_axes_of_many_tokens(Hq):
    """The bits of moe_rope for q, and of one axis where positions are alike,
    on both sides of where a thread takes two heads of q."""
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(7)
    N, P, D = 2049, 64, 128
    k, v, q = (torch.randn((N, h, D), generator=gen, device="cuda").to(torch.bfloat16) for h in (2, 2, Hq))
    table, axes = m.rope_table(5000, D, device="cuda"), m.rope_axes([24, 20, 20], True)
    pos = torch.randint(0, 5000, (3, N), generator=gen, device="cuda", dtype=torch.int32)
    pages = torch.randperm(33, generator=gen, device="cuda").to(torch.int32)[None]
    batch = dict(block_table=pages, seq_lens=torch.tensor([N], dtype=torch.int32, device="cuda"),
                 cu_q=torch.tensor([0, N], dtype=torch.int32, device="cuda"), max_q_len=N, q=q, cos_sin=table)
    got = m.PagedKVCache.create(33, 2, P, D).append(k, v, **batch, positions=pos, axes=axes)
    assert torch.equal(got, m.moe_rope(q, pos, table, axes=axes))
    a, b = (m.PagedKVCache.create(33, 2, P, D) for _ in range(2))
    alike = pos[:1].expand(3, N)
    qa, qb = a.append(k, v, **batch, positions=pos[0], axes=None), b.append(k, v, **batch, positions=alike, axes=axes)
    assert torch.equal(qa, qb) and torch.equal(a.k, b.k) and torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v, b.v)


def test_append_axes_bad_positions_and_empty_slots():
    torch = torch_mod()
    rng = np.random.default_rng(37)
    lens = [0, 20, 0, 17, 1]
    batch = Batch(rng, [1] * 5, lens, 2, 16, 64)
    k, v, q = (tensor(rounded(rng, (5, h, 64), "bfloat16"), "bfloat16") for h in (2, 2, 4))
    table, axes = m.rope_table(64, 64, device="cuda"), m.rope_axes([12, 10, 10])
    pos = np.array([[-1, 19, -1, 16, 0], [-1, 3, -1, 5, 0], [-1, 2, -1, 1, 0]], np.int32)
    got = batch.cache.append(k, v, **batch.dev, q=q, cos_sin=table, positions=tensor(pos, "int32"), axes=axes)
    assert batch.cache.device_status() == m.MOE_OK
    assert torch.equal(got[[0, 2]], q[[0, 2]])
    want = m.moe_rope(q, tensor(np.maximum(pos, 0), "int32"), table, axes=axes)
    assert torch.equal(got[[1, 3, 4]], want[[1, 3, 4]])
    pos[2, 3] = 64                                     # one axis of a token that is there
    got = batch.cache.append(k, v, **batch.dev, q=q, cos_sin=table, positions=tensor(pos, "int32"), axes=axes)
    assert batch.cache.device_status() == m.MOE_ERR_BAD_POSITION
    assert torch.equal(got[3], q[3]) and torch.equal(got[1], want[1])
    page, off = batch.table[3, 1], 0                   # place 16 of its sequence, unturned
    held = ao.E4M3_VALUES[batch.cache.k[page, :, off].cpu().numpy()] * f64(batch.cache.k_scale[page])[:, None]
    assert (np.abs(held - f64(k[3])) <= np.abs(f64(k[3])) * 2.0 ** -4 + 2.0 ** -10 * f64(batch.cache.k_scale[page])[:, None]).all()


def test_a_captured_call_keeps_its_axes():
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(9)
    q = torch.randn((6, 4, 64), generator=gen, device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 90, (3, 6), generator=gen, device="cuda", dtype=torch.int32)
    table, axes = m.rope_table(90, 64, device="cuda"), [m.rope_axes([12, 10, 10]), m.rope_axes([12, 10, 10], True)]
    want = [m.moe_rope(q, pos, table, axes=a) for a in axes]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [m.moe_rope(q, pos, table, axes=a) for a in axes]
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want)) and not torch.equal(*want)
