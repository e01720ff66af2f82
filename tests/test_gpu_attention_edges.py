"""moe_rope, moe_kv_append and moe_paged_attention where their first tests do
not reach: rows that end apart, long contexts under one dominating key, streams
and graphs, slots without a sequence.  Bounds as in test_gpu_attention.py but
where a test derives its own."""
import numpy as np
import pytest

import moe_lora_expert_gb300 as m
from oracle import attention_oracle as ao
from test_gpu_attention import HALF_STEP, Batch, check_attention, f64, rounded, tensor, torch_mod

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,past,Hq,Hkv,P,D,window", [(37, 0, 24, 8, 16, 64, 0), (50, 90, 20, 10, 24, 128, 70)])
def test_units_that_end_inside_a_warp(new, past, Hq, Hkv, P, D, window):
    """Several units a CTA, each ending in a warp of which some lanes have no
    row: every unit is walked once, whatever its lanes do at the end of one."""
    torch = torch_mod()
    rng = np.random.default_rng(21)
    B = 40
    batch = Batch(rng, [new] * B, [new + past + b % 3 for b in range(B)], Hkv, P, D, std=0.5)
    q = rounded(rng, (B * new, Hq, D), "bfloat16")
    out, lse = check_attention(batch, q, "bfloat16", window=window)
    again = batch.cache.attend(tensor(q, "bfloat16"), **batch.dev, cu_q=batch.cu_dev, max_q_len=new, window=window, return_lse=True)
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    assert batch.cache.device_status() == m.MOE_OK


@pytest.mark.parametrize("new,B,Hq", [(1, 64, 16), (64, 20, 32)])     # single tokens; 256 rows a key head
@pytest.mark.parametrize("keys,rest", [(131072, 1e-3), (131072, 4e-4), (262144, 1e-3)])
def test_lse_of_many_small_weights_beside_a_large_one(new, B, Hq, keys, rest):
    """All keys but the first score zero and together have ``rest`` of the
    mass: lse = log(keys seen - 1 + exp(s_0)).  Each addition to a sum in
    float32 is off by 2^-24 of it at most, and one for each 64 keys is
    2^-24 * keys / 64 <= 2^-12: an eighth of ``rest``, in which 8 keys at a
    time would be all of it.  Both scores are exact products here."""
    torch = torch_mod()
    Hkv, P, D, scale = 8, 64, 64, 0.125
    k = torch.zeros((keys // P, Hkv, P, D), dtype=torch.uint8, device="cuda")
    k[0, :, 0, 0] = 0x38                                      # code 1
    cache = m.PagedKVCache(k, k, *[torch.ones(k.shape[:2], device="cuda") for _ in range(2)])
    q = torch.zeros((B * new, Hq, D), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = float(np.log(keys * (1 - rest) / rest) / scale)
    out, lse = cache.attend(q, torch.arange(keys // P, dtype=torch.int32, device="cuda").expand(B, -1).contiguous(),
                            torch.full((B,), keys, dtype=torch.int32, device="cuda"), max_q_len=new, scale=scale, return_lse=True,
                            cu_q=torch.arange(0, B * new + 1, new, dtype=torch.int32, device="cuda"))
    sees = keys - new + 1 + np.arange(B * new) % new
    s0 = scale * q[0, 0, 0].item()
    want = s0 + np.log1p((sees - 1) * np.exp(-s0))
    err = np.abs(f64(lse) - want[:, None])
    assert (err <= 2.0 ** -24 * keys / 64 + 2.0 ** -20 * (1 + want[:, None])).all(), float(err.max())
    assert cache.device_status() == m.MOE_OK


# ---------------------------------------------- one key that takes nearly all
#
# A weight 2^(y - b) is a float16, off by 2^-25 where it is subnormal; a key's
# exponent y stands for p v_scale = 2^y / Z.  So a key loses at most 2^-25
# |code| 2^b / Z of the output, and no more than its own part p |v|.  The
# reference b is 7 below some earlier key's exponent when it rises, so 2^b / Z
# <= 2^-7 max (p v_scale) at all times.  It falls when 64 keys that follow one
# another, and that all rows of a tile see, are more than 8 below it, which is
# looked for at one of 8 such runs at least.  So among 9 runs of 64 keys one
# made it rise, or is not that low, or made it fall: at the last of them 2^b / Z
# <= 2^8 max (p v_scale) over the 9, unless b stands 31 below the row's largest
# already.
# Keys that not all rows of a tile see are among the last 192 that a row sees:
# there b is what the runs before left, or 7 below one of their own.  The
# tests' bound has, in place of a term that knows nothing of how many keys
# there are, the sum of that over the keys.

def lost_weights(p, vs, codes):
    """That term for probabilities p [rows, keys], value scales vs [keys] and
    value codes [keys, columns]: [rows, columns]."""
    pad, D = -p.shape[1] % 64, codes.shape[1]
    runs = lambda x: np.pad(x, ((0, 0), (0, pad))).reshape(len(x), -1, 64)   # noqa: E731
    top, size = runs(p * vs).max(-1), np.pad(np.abs(codes), ((0, pad), (0, 0))).reshape(-1, 64, D)
    before = np.pad(top, ((0, 0), (8, 0)))
    nine = np.max([before[:, i:i + top.shape[1]] for i in range(9)], axis=0)
    most = top.max(-1, keepdims=True)
    at = np.minimum(2.0 ** 8 * nine, 2.0 ** -7 * most)
    for r, row in enumerate(p):
        first = max(1, (np.flatnonzero(row)[-1] - 191) // 64)         # of the runs with keys that not all rows see
        at[r, first:] = min(max(2.0 ** 8 * nine[r, first - 1], 2.0 ** -7 * top[r, first:].max()), 2.0 ** -7 * most[r, 0])
    own = np.einsum("rck,ckd->rcd", runs(p * vs), size, optimize=True)
    return np.minimum(2.0 ** -25 * (at + 2.0 ** -31 * most)[..., None] * size.sum(1), own).sum(1)


@pytest.mark.parametrize("new,B,Hq", [(1, 64, 16), (4, 32, 32), (64, 20, 32)])   # 2, 16 and 256 rows a key head
@pytest.mark.parametrize("keys,rest,std,at,shift", [
    (32768, 1e-2, 1.0, 0, 0), (32768, 1e-3, 1.0, 0, 0), (32768, 1e-3, 0.0, 5000, 0), (32768, 1e-5, 0.0, 0, 0),
    (131072, 1e-3, 0.0, 0, 0), (131072, 1e-4, 1.0, 0, 12), (32768, 1e-3, 1.0, 32000, 0),
])
def test_attention_sink(new, B, Hq, keys, rest, std, at, shift):
    """One key has all but ``rest`` of the mass and values of zero, on a page
    whose value scale is 2^shift times the others': the output is what the
    others leave.  The sequences share their pages, so that a CTA has many
    keys of a row."""
    torch = torch_mod()
    rng = np.random.default_rng(keys + at)
    Hkv, P, D, scale = 8, 64, 64, 0.125
    shape = (keys // P, Hkv, P, D)
    k = np.zeros(shape, np.uint8)
    k[..., 1:] = ao.e4m3_encode(rng.standard_normal(64 * 63) * 32).reshape(64, 63)[rng.integers(0, 64, shape[:3])]
    v = ao.e4m3_encode((1 + 0.25 * rng.standard_normal(256)) * 128)[rng.integers(0, 256, shape)]
    ks, vs = np.full(shape[:2], 2.0 ** -5, np.float32), np.full(shape[:2], 2.0 ** -7, np.float32)
    order = rng.permutation(shape[0])
    page = order[at // P]
    k[page, :, at % P] = 0
    k[page, :, at % P, 0] = ao.e4m3_encode([448.0])[0]
    v[page] = 0
    vs[page] *= 2.0 ** shift
    kv, vv = ao.E4M3_VALUES[k[order]] * 2.0 ** -5, ao.E4M3_VALUES[v[order]] * vs[order][:, :, None, None]
    kv, vv, code = (x.transpose(1, 0, 2, 3).reshape(Hkv, keys, D) for x in (kv, vv, ao.E4M3_VALUES[v[order]]))
    q = rounded(rng, (B * new, Hq, D), "bfloat16", std)
    G = Hq // Hkv
    rows = [b * new + t for b in (0, B - 1) for t in {0, new // 2, new - 1}]
    sees = np.array([keys - new + r % new for r in rows])[:, None] >= np.arange(keys)    # [rows, keys]
    tail = sees & (np.arange(keys) != at)
    # the same sink for all rows of a head: as large as the first checked row needs it
    for h in range(Hq):
        s = scale * (kv[h // G, :, 1:] @ q[rows[0], h, 1:])
        lse = np.log(np.exp(s[tail[0]] - s.max()).sum()) + s.max()
        q[:, h, 0] = (lse + np.log((1 - rest) / rest)) / (scale * 448 * 2.0 ** -5)
    qt = tensor(q, "bfloat16")
    q = f64(qt)
    cache = m.PagedKVCache(tensor(k, torch.uint8), tensor(v, torch.uint8), tensor(ks, "float32"), tensor(vs, "float32"))
    table = tensor(np.broadcast_to(order.astype(np.int32), (B, keys // P)), "int32")
    out, lse = cache.attend(qt, table, torch.full((B,), keys, dtype=torch.int32, device="cuda"),
                            cu_q=tensor(np.arange(B + 1, dtype=np.int32) * new, "int32"), max_q_len=new, scale=scale, return_lse=True)
    out, lse = f64(out), f64(lse)
    for h in range(Hq):
        s = np.where(sees, scale * (q[rows, h] @ kv[h // G].T), -np.inf)
        es = 128 * 2.0 ** -22 * scale * (np.abs(q[rows, h]) @ np.abs(kv[h // G]).T).max(-1)
        top = s.max(-1, keepdims=True)
        e = np.exp(s - top)
        p, ref_lse = e / e.sum(-1, keepdims=True), top[:, 0] + np.log(e.sum(-1))
        if h == 0:
            assert 0.5 * rest < 1 - p[0, at] < 2 * rest       # the case is what it is meant to be
        ref, spread = p @ vv[h // G], p @ np.abs(vv[h // G])
        bound = ((2.0 ** -11 + 4 * es + 2.0 ** -17)[:, None] * spread + lost_weights(p, np.repeat(vs[order, h // G], P), code[h // G])
                 + 1.01 * HALF_STEP["bfloat16"] * np.abs(ref))
        err = np.abs(out[rows, h] - ref)
        assert (err <= bound).all(), (h, float((err / np.abs(ref)).max()), float((bound / np.abs(ref)).max()))
        assert (np.abs(lse[rows, h] - ref_lse) <= es + 2.0 ** -20 * (1 + np.abs(ref_lse))).all()
    assert cache.device_status() == m.MOE_OK


# ------------------------------------------------------ workspaces and graphs

def decode_batch(seed):
    """Two sequences whose keys several CTAs share."""
    rng = np.random.default_rng(seed)
    batch = Batch(rng, [1, 1], [9000, 5000], 2, 32, 64, std=0.5)
    return batch, tensor(rounded(rng, (2, 8, 64), "bfloat16"), "bfloat16")


def workspace_of(call):
    """The workspace address that an attention call hands to the library."""
    from moe_lora_expert_gb300 import attention
    seen, real = [], attention._attend_fn

    def spy(args, handle):
        seen.append(m.PagedAttentionArgs.from_buffer_copy(args).workspace)
        return real(args, handle)

    attention._attend_fn = spy
    try:
        result = call()
    finally:
        attention._attend_fn = real
    return result, seen


def test_attention_in_a_default_capture():
    """As graphs are usually captured: a warm-up on the current stream, then
    torch.cuda.graph with its own stream and nothing prepared for it."""
    torch = torch_mod()
    batch, q = decode_batch(30)
    want = batch.cache.attend(q, **batch.dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = batch.cache.attend(q, **batch.dev)
        twice = batch.cache.attend(q, **batch.dev)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(twice, want)
    assert torch.equal(batch.cache.attend(q, **batch.dev), want)
    assert batch.cache.device_status() == m.MOE_OK


def test_graphs_replayed_on_two_streams():
    """Two captures have a workspace each (their calls share it) and may run
    at once, and beside calls on the streams that they were captured on."""
    torch = torch_mod()
    batches = [decode_batch(31), decode_batch(32)]
    wants = [b.cache.attend(q, **b.dev) for b, q in batches]
    graphs, outs, used = [], [], []
    for b, q in batches:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            out, seen = workspace_of(lambda: [b.cache.attend(q, **b.dev) for _ in range(4)])
        outs.append(out)
        assert len(set(seen)) == 1
        used.append(seen[0])
    current = torch.cuda.current_stream().cuda_stream
    assert len({*used, batches[0][0].cache.workspace(current)[0]}) == 3
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = [b.cache.attend(q, **b.dev) for b, q in batches]
        torch.cuda.synchronize()
        for out, want, e in zip(outs, wants, eager):
            assert all(torch.equal(o, want) for o in out) and torch.equal(e, want)


def test_caches_share_a_streams_workspace():
    """A cache for each layer costs no workspace of its own, and a workspace
    belongs to its stream from the first word on: nothing waits for another."""
    torch = torch_mod()
    (a, qa), (b, qb) = decode_batch(33), decode_batch(34)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    want_a, want_b = a.cache.attend(qa, **a.dev), b.cache.attend(qb, **b.dev)
    for stream in (None, side):
        outs, seen = workspace_of(lambda: [a.cache.attend(qa, **a.dev, stream=stream), b.cache.attend(qb, **b.dev, stream=stream)])
        torch.cuda.synchronize()
        assert len(set(seen)) == 1 and torch.equal(outs[0], want_a) and torch.equal(outs[1], want_b)


def test_workspace_init_refuses():
    lib = m.lib()
    n = lib.moe_paged_attention_workspace_size()
    for pointer, size in ((None, n), (64, n), (256, n - 1)):
        assert lib.moe_paged_attention_workspace_init(pointer, size, None) == m.MOE_ERR_WORKSPACE
    assert lib.moe_stream_capture_id(None, None) == m.MOE_ERR_NULL


# ----------------------------------------------------------------- the status

def test_status_of_calls_on_other_streams():
    """A problem of a call that still waits on another stream is reported, once."""
    torch = torch_mod()
    batch, q = decode_batch(35)
    side = torch.cuda.Stream()
    bad = torch.full_like(batch.dev["block_table"], batch.pages + 1)
    torch.cuda.synchronize()
    batch.cache.attend(q, **batch.dev, stream=side)     # what a first call loads and allocates may wait for the device
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)                  # about 50 ms
    batch.cache.attend(q, bad, batch.dev["seq_lens"], stream=side)
    assert batch.cache.device_status() == m.MOE_ERR_BAD_PAGE
    assert batch.cache.device_status() == m.MOE_OK


def test_status_of_a_cache_made_on_a_busy_stream():
    """The status word is cleared before the cache can be used anywhere."""
    torch = torch_mod()
    batch, _ = decode_batch(36)
    k = torch.zeros((2, 2, 64), dtype=torch.bfloat16, device="cuda")
    bad = torch.full_like(batch.dev["block_table"], batch.pages + 1)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    batch.cache.append(k, k, **batch.dev, stream=side)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    cache = m.PagedKVCache(batch.cache.k, batch.cache.v, batch.cache.k_scale, batch.cache.v_scale)
    cache.append(k, k, bad, batch.dev["seq_lens"], stream=side)
    assert cache.device_status() == m.MOE_ERR_BAD_PAGE


# --------------------------------------------------------------------- append

@pytest.mark.parametrize("given", [False, True])
def test_append_passes_over_empty_slots(given):
    """A decode batch of fixed size with slots that hold no sequence: nothing
    is written for those, their q is copied, and no problem is reported, so
    that a real one is."""
    torch = torch_mod()
    rng = np.random.default_rng(37)
    lens = [0, 20, 0, 17, 1]
    batch = Batch(rng, [1] * 5, lens, 2, 16, 64)
    k, v, q = (rounded(rng, (5, h, 64), "bfloat16") for h in (2, 2, 4))
    table = m.rope_table(64, 64, device="cuda")
    pos = np.array([n - 1 for n in lens], np.int32)
    before = [x.clone() for x in (batch.cache.k, batch.cache.v, batch.cache.k_scale, batch.cache.v_scale)]
    kw = dict(positions=tensor(pos, "int32")) if given else {}
    got = batch.cache.append(tensor(k, "bfloat16"), tensor(v, "bfloat16"), **batch.dev, q=tensor(q, "bfloat16"), cos_sin=table, **kw)
    assert batch.cache.device_status() == m.MOE_OK
    real = [b for b, n in enumerate(lens) if n]
    alone = m.PagedKVCache(*before)
    want = alone.append(tensor(k[real], "bfloat16"), tensor(v[real], "bfloat16"), batch.dev["block_table"][real].contiguous(),
                        batch.dev["seq_lens"][real].contiguous(), q=tensor(q[real], "bfloat16"), cos_sin=table)
    assert torch.equal(got[real], want) and (f64(got)[[0, 2]] == q[[0, 2]]).all()
    for a, b in ((batch.cache.k, alone.k), (batch.cache.v, alone.v), (batch.cache.k_scale, alone.k_scale),
                 (batch.cache.v_scale, alone.v_scale)):
        assert torch.equal(a, b)
    out = batch.cache.attend(got, **batch.dev)
    assert (f64(out)[[0, 2]] == 0).all() and batch.cache.device_status() == m.MOE_OK
    # a negative length, and a token without a place in its sequence, still are problems
    batch.cache.append(tensor(k, "bfloat16"), tensor(v, "bfloat16"), batch.dev["block_table"], batch.dev["seq_lens"] - 1)
    assert batch.cache.device_status() == m.MOE_ERR_BAD_POSITION
    batch.cache.append(tensor(k, "bfloat16"), tensor(v, "bfloat16"), **batch.dev, cu_q=batch.cu_dev, max_q_len=1)
    assert batch.cache.device_status() == m.MOE_ERR_BAD_POSITION


# ------------------------------------------------------------------------ NaN

@pytest.mark.parametrize("D,Hq,Hkv,window", [(64, 16, 16, 0), (128, 16, 4, 9000)])
def test_attention_one_nan_on_a_long_context(D, Hq, Hkv, window):
    """A NaN value that some rows of a unit see and others do not costs the
    unit's CTA a look at that tile, not at every key of its later units: no
    wait of 10 ms runs out, and only what sees it changes."""
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(38)
    new, past, P = 5120, 15360, 64
    pages = (new + past) // P
    shape = (pages, Hkv, P, D)
    k, v = ((torch.randn(shape, generator=gen, device="cuda") * 40).to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2))
    cache = m.PagedKVCache(k, v, *[torch.full(shape[:2], 2.0 ** -6, device="cuda") for _ in range(2)])
    q = torch.randn((new, Hq, D), generator=gen, device="cuda").to(torch.bfloat16)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    args = dict(block_table=order[None].contiguous(), seq_lens=tensor(np.array([new + past], np.int32), "int32"),
                cu_q=tensor(np.array([0, new], np.int32), "int32"), window=window, return_lse=True, wait_timeout_ms=10)
    clean, lse = cache.attend(q, **args)
    assert cache.device_status() == m.MOE_OK
    # in the middle of a unit that is late in its sequence, and so among the first to be done, and of an early one
    where = [past + new - 100, past + 300]
    for i, j in enumerate(where):
        v[order[j // P].long(), :, j % P, 33 + 16 * i] = 0x7F if i else 0xFF
    out, lse_nan = cache.attend(q, **args)
    assert cache.device_status() == m.MOE_OK
    assert torch.equal(lse, lse_nan)
    at = past + torch.arange(new, device="cuda")
    want = clean.clone()
    for i, j in enumerate(where):
        sees = (at >= j) & ((at < j + window) if window else True)
        want[sees, :, 33 + 16 * i] = float("nan")
    assert torch.equal(out.isnan(), want.isnan()) and torch.equal(out.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("bad", [0, 13])
def test_attention_nan_in_many_partial_tiles(bad):
    """More tiles with NaN and missing pages than a unit notes: still only the
    rows that see a NaN have it."""
    torch = torch_mod()
    rng = np.random.default_rng(39)
    batch = Batch(rng, [200], [4000], 1, 16, 64, std=0.5)
    q = rounded(rng, (200, 2, 64), "float16")
    table = batch.dev["block_table"]
    if bad:
        table[0, 1:240:bad] = -1                        # pages of most of the first 30 tiles
    clean, lse = batch.cache.attend(tensor(q, "float16"), **batch.dev, cu_q=batch.cu_dev, return_lse=True)
    for j in range(5, 4000, 128):                       # a NaN in every tile of 128 keys, in columns 0 to 31
        page = int(table[0, j // 16])
        if page >= 0:
            batch.cache.v[page, 0, j % 16, (j // 128) % 64] = 0x7F
    out, lse_nan = batch.cache.attend(tensor(q, "float16"), **batch.dev, cu_q=batch.cu_dev, return_lse=True)
    want = f64(clean)
    host = table[0].cpu().numpy()
    for j in range(5, 4000, 128):
        if host[j // 16] >= 0:
            want[np.arange(200) + 3800 >= j, :, (j // 128) % 64] = np.nan
    np.testing.assert_array_equal(f64(out), want)
    assert torch.equal(lse, lse_nan)
    assert batch.cache.device_status() == (m.MOE_ERR_BAD_PAGE if bad else m.MOE_OK)


@pytest.mark.parametrize("dtype", ["bfloat16", "float16"])
@pytest.mark.parametrize("new,lens,Hq,Hkv,D", [([120, 33], [270, 183], 6, 2, 80), ([50, 300], [700, 900], 8, 1, 128), ([3, 5], [900, 40], 8, 2, 64)])
def test_rows_do_not_depend_on_their_neighbours(dtype, new, lens, Hq, Hkv, D):
    """A sequence's output has the same bits whatever the queries of the next
    one are, which a tile may hold past its rows."""
    torch = torch_mod()
    rng = np.random.default_rng(41)
    batch = Batch(rng, new, lens, Hkv, 16, D, std=0.5)
    q = tensor(rounded(rng, (sum(new), Hq, D), dtype), dtype)
    kw = dict(**batch.dev, cu_q=batch.cu_dev, max_q_len=max(new), return_lse=True)
    out, lse = batch.cache.attend(q, **kw)
    for size in (0.0, 30.0, 1000.0):
        other = q.clone()
        other[new[0]:] *= size
        got, got_lse = batch.cache.attend(other, **kw)
        assert torch.equal(got[:new[0]], out[:new[0]]) and torch.equal(got_lse[:new[0]], lse[:new[0]])


# -------------------------------------------------------------------- strides

@pytest.mark.parametrize("dtype,scale", [("bfloat16", 0.2), ("float16", -0.2), ("bfloat16", -0.2), ("float16", 0.2)])
@pytest.mark.parametrize("new,D", [([1, 1], 64), ([3, 2], 128), ([120, 33], 80), ([300, 2], 64)])
def test_attention_broadcast_and_reversed_queries(dtype, scale, new, D):
    """Queries with strides of zero (one for all heads, one for all tokens)
    and below (tokens and heads backwards) give the bits of a copy of them,
    whichever kernel the number of rows asks for."""
    torch = torch_mod()
    rng = np.random.default_rng(40)
    Hq, Hkv, N = 6, 2, sum(new)
    batch = Batch(rng, new, [n + 150 for n in new], Hkv, 16, D, std=0.5)
    kw = dict(**batch.dev, cu_q=batch.cu_dev, max_q_len=max(new), scale=scale, return_lse=True)
    one_head = tensor(rounded(rng, (N, 1, D), dtype), dtype).expand(N, Hq, D)
    one_token = tensor(rounded(rng, (1, Hq, D), dtype), dtype).expand(N, Hq, D)
    for q in (one_head, one_token):
        out, lse = batch.cache.attend(q, **kw)
        want, want_lse = batch.cache.attend(q.contiguous(), **kw)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        ref = ao.attend(f64(q), *batch.codes, *batch.scales, batch.table, batch.lens, batch.cu, scale)[1]
        assert np.abs(f64(lse) - ref).max() < 1e-2
    # the library's own interface: from the last token and head backwards
    q = tensor(rounded(rng, (N, Hq, D), dtype), dtype)
    want, _ = batch.cache.attend(q.flip(0, 1).contiguous(), **kw)
    out = torch.empty_like(q)
    ws = batch.cache.workspace(torch.cuda.current_stream().cuda_stream)
    c = batch.cache
    a = m.PagedAttentionArgs(struct_size=248, dtype=m.MOE_DTYPE_BF16 if dtype == "bfloat16" else m.MOE_DTYPE_F16, q=q[-1, -1].data_ptr(),
                             out=out.data_ptr(), q_stride_token=-Hq * D, q_stride_head=-D, out_stride_token=Hq * D, out_stride_head=D,
                             block_table=batch.dev["block_table"].data_ptr(), seq_lens=batch.dev["seq_lens"].data_ptr(),
                             cu_q=batch.cu_dev.data_ptr(), status=c.status.data_ptr(), workspace=ws[0], workspace_bytes=ws[1], N=N, B=len(new),
                             Hq=Hq, table_width=batch.table.shape[1], max_q_len=max(new), max_seq_len=max(batch.lens), scale=scale)
    a.cache = m.KvCache(c.k.data_ptr(), c.v.data_ptr(), c.k_scale.data_ptr(), c.v_scale.data_ptr(), *c.k.stride()[:3], *c.v.stride()[:3], *c.k.shape)
    assert m.lib().moe_paged_attention(bytes(a), torch.cuda.current_stream().cuda_stream) == m.MOE_OK
    assert torch.equal(out, want) and c.device_status() == m.MOE_OK


# ---------------------------------------------------------------- wide queries

@pytest.mark.parametrize("new,lens", [([1, 1], [300, 40]), ([90, 5], [300, 40])])
@pytest.mark.parametrize("ratio", [20, 28])
def test_attention_queries_of_a_wide_range(new, lens, ratio):
    """A bf16 row with one value 2^ratio times the others, in a column where
    all keys are zero: what the others say is not lost."""
    rng = np.random.default_rng(42)
    batch = Batch(rng, new, lens, 2, 16, 64, std=0.5)
    batch.codes[0][..., 7] = 0
    batch.cache.k.copy_(tensor(batch.codes[0], torch_mod().uint8))
    q = rounded(rng, (sum(new), 4, 64), "bfloat16")
    q[..., 7] = 2.0 ** ratio
    check_attention(batch, q, "bfloat16", scale=0.3, decode=max(new) == 1)


@pytest.mark.parametrize("new,lens", [([1, 1], [300, 40]), ([90, 5], [300, 40])])
@pytest.mark.parametrize("power", [122, 100, -100, -125])
def test_attention_queries_at_the_ends_of_their_type(new, lens, power):
    """bf16 rows near the largest and smallest finite values, with key scales
    that make ordinary scores of them."""
    rng = np.random.default_rng(43)
    batch = Batch(rng, new, lens, 2, 16, 64, std=0.5)
    back = np.float32(2.0 ** (-power // 2))
    batch.scales[0] *= back
    batch.cache.k_scale.copy_(tensor(batch.scales[0], "float32"))
    q = rounded(rng, (sum(new), 4, 64), "bfloat16") * 2.0 ** power
    scale = 0.3 * 2.0 ** (-power - (-power // 2))
    check_attention(batch, f64(tensor(q, "bfloat16")), "bfloat16", scale=float(np.float32(scale)), decode=max(new) == 1)


# ------------------------------------------------------- append, once more

@pytest.mark.parametrize("P,limit", [(16, 5), (16, 1), (8, 20), (64, 33)])
def test_append_ends_at_max_q_len(P, limit):
    """A sequence with more new tokens than max_q_len: its first max_q_len
    are appended, at their places, and nothing else is written."""
    torch = torch_mod()
    rng = np.random.default_rng(44)
    new, lens = [limit + 9, 3, limit], [limit + 40, 30, limit + 1]
    batch = Batch(rng, new, lens, 2, P, 32)
    k, v = (tensor(rounded(rng, (sum(new), 2, 32), "bfloat16"), "bfloat16") for _ in range(2))
    parts = [x.clone() for x in (batch.cache.k, batch.cache.v, batch.cache.k_scale, batch.cache.v_scale)]
    batch.cache.append(k, v, **batch.dev, cu_q=batch.cu_dev, max_q_len=limit)
    keep = np.concatenate([np.arange(a, a + min(n, limit)) for a, n in zip(batch.cu, new)])
    kept = [min(n, limit) for n in new]
    want = m.PagedKVCache(*[x.clone() for x in parts])
    want.append(k[keep], v[keep], batch.dev["block_table"], tensor(np.array([e - n + t for n, e, t in zip(new, lens, kept)], np.int32), "int32"),
                cu_q=tensor(np.cumsum([0] + kept).astype(np.int32), "int32"), max_q_len=limit)
    for a, b in ((batch.cache.k, want.k), (batch.cache.v, want.v), (batch.cache.k_scale, want.k_scale), (batch.cache.v_scale, want.v_scale)):
        assert torch.equal(a, b)
    # tokens that the arrays do not hold are left out, those before them keep their places
    less = sum(new) - 2
    again = m.PagedKVCache(*[x.clone() for x in parts])
    again.append(k[:less], v[:less], **batch.dev, cu_q=batch.cu_dev, max_q_len=max(new))
    full = m.PagedKVCache(*[x.clone() for x in parts])
    full.append(k[:less], v[:less], batch.dev["block_table"], tensor(np.array([*lens[:2], lens[2] - 2], np.int32), "int32"),
                cu_q=tensor(np.array([*batch.cu[:3], less], np.int32), "int32"), max_q_len=max(new))
    assert torch.equal(again.k, full.k) and torch.equal(again.v_scale, full.v_scale)


@pytest.mark.parametrize("D", [16, 80])
def test_append_divides_by_a_scale_of_the_callers(D):
    """Pages that hold tokens under any scale keep it if it is large enough,
    and the new codes are those of x / scale: here each close to the middle of
    two codes, where x times the scale's inverse gives the other one."""
    torch = torch_mod()
    mids = (ao.E4M3_VALUES[8:0x70] + ao.E4M3_VALUES[9:0x71]) / 2
    cases = []
    for x in 1 + np.arange(128) / np.float32(128):
        for c in mids:
            s = np.float32(x) / np.float32(c)
            codes = ao.e4m3_encode([np.float32(x) / s, np.float32(x) * (np.float32(1) / s)])
            if codes[0] != codes[1]:
                cases.append((x, s, codes[0]))
    assert len(cases) > 100
    x, s, want = (np.array(t) for t in zip(*cases))
    B = len(cases)
    cache = m.PagedKVCache(*[torch.zeros((B, 1, 8, D), dtype=torch.uint8, device="cuda") for _ in range(2)],
                           *[tensor(s.astype(np.float32)[:, None], "float32") for _ in range(2)])
    k = tensor(np.broadcast_to(x.astype(np.float32)[:, None, None], (B, 1, D)), "bfloat16")
    cache.append(k, -k, torch.arange(B, dtype=torch.int32, device="cuda")[:, None].contiguous(),
                 torch.full((B,), 2, dtype=torch.int32, device="cuda"))
    assert torch.equal(cache.k_scale[:, 0].cpu(), torch.from_numpy(s.astype(np.float32)))
    assert (cache.k[:, 0, 1].cpu().numpy() == want[:, None]).all()
    assert (cache.v[:, 0, 1].cpu().numpy() == (want | 0x80)[:, None]).all()


def test_memory_of_a_call_on_another_stream_is_not_handed_out():
    """Operands that are dropped while the call still waits on its stream."""
    torch = torch_mod()
    batch, _ = decode_batch(45)
    side = torch.cuda.Stream()
    q = torch.randn((2, 8, 64), device="cuda").to(torch.bfloat16)
    want = batch.cache.attend(q, **batch.dev, stream=side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    mine, size = q.data_ptr(), q.shape
    out = batch.cache.attend(q, **batch.dev, stream=side)
    del q
    taken = [torch.empty(size, dtype=torch.bfloat16, device="cuda") for _ in range(64)]
    assert all(t.data_ptr() != mine for t in taken)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
