"""Positions of several axes, attention with a window and lasting first tokens, and attention of batches that share a
prefix: the cases that are timed, and their plain forms.

A case names one of four operators ("op"):

  axes    moe_rope with an axis (time, height, width) for each pair of columns: q and k; "inverse" is the gradient.
  append  moe_kv_append with such positions: keys (rotated) and values of new tokens into the paged e4m3 cache.
  sinks   moe_paged_attention with a sliding window and the first tokens visible to every row.
  shared  moe_paged_attention of sequences that share their first tokens, whose keys are read once for a group of them.

Shapes follow the attention half of perf/operators.py and the routed layer's batches (16 and 64 decode tokens, 2 x 2048
prefill tokens); the others are generic odd ones.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases

def _case(name, op, B, q_len, ctx, Hq, Hkv, D, P, dtype, nhd=False, R=0, A=0, turns=False, interleaved=False, inverse=False, window=0, sinks=0, shared=0,
          groups=0):
    """B sequences of up to q_len new tokens each, on top of up to ctx tokens that the cache holds already and, in groups
    of sequences, of ``shared`` tokens that all of a group begin with."""
    c = dict(op=op, B=B, q_len=q_len, ctx=ctx, Hq=Hq, Hkv=Hkv, D=D, P=P, dtype=dtype, nhd=nhd, R=R, A=A, turns=turns, interleaved=interleaved, inverse=inverse,
             window=window, sinks=sinks, shared=shared, groups=groups)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of 16 sequences that follow images: q and k of 16 tokens, where the launch counts
        _case("axes_decode_16", "axes", 16, 1, 2048, 32, 4, 128, 16, "bfloat16", R=128, A=3),
        # the prefill of 2 x 2048 tokens of text and images: a run of pairs for time, height and width each
        _case("axes_prefill_4096", "axes", 2, 2048, 0, 32, 4, 128, 16, "bfloat16", R=128, A=3),
        # the backward pass with 48 of 80 columns rotated as neighbours, the axes taking turns, float32, odd lengths
        _case("axes_grad_turns", "axes", 3, 1021, 5, 20, 20, 80, 16, "float32", R=48, A=3, turns=True, interleaved=True, inverse=True),
        # the same prefill's keys and values into fresh pages, with the queries
        _case("append_axes_4096", "append", 2, 2048, 0, 32, 4, 128, 64, "bfloat16", R=128, A=3, turns=True),
        # a chat of a quarter million tokens of which the last 4096 and the first 4 are seen: latency
        _case("sinks_decode_1", "sinks", 1, 1, 262139, 32, 4, 128, 16, "bfloat16", window=4096, sinks=4),
        # a decode step of 64 long chats: the bandwidth of the cache
        _case("sinks_decode_64", "sinks", 64, 1, 32767, 32, 4, 128, 64, "bfloat16", window=8192, sinks=64),
        # the prefill of 2 x 2048 tokens in a window
        _case("sinks_prefill_4096", "sinks", 2, 2048, 0, 32, 4, 128, 64, "bfloat16", window=1024, sinks=4),
        # ragged chunks of up to 1000 tokens on up to 8191 earlier ones, 64-wide heads, pages of 48, float16, first tokens that end inside a tile
        _case("sinks_chunk_ragged", "sinks", 4, 1000, 8191, 20, 5, 64, 48, "float16", nhd=True, window=3001, sinks=131),
        # two instructions, four answers each, of one token: small, latency
        _case("shared_decode_8", "shared", 8, 1, 300, 32, 4, 128, 16, "bfloat16", shared=2048, groups=2),
        # a decode step of 64 requests on one instruction of 8192 tokens
        _case("shared_decode_64", "shared", 64, 1, 1023, 32, 4, 128, 64, "bfloat16", shared=8192, groups=1),
        # drafts of 4 tokens for 20 requests on 3 documents whose length is no multiple of anything, 64-wide heads, pages of 24, float16
        _case("shared_draft_20", "shared", 20, 4, 701, 20, 5, 64, 24, "float16", nhd=True, shared=15001, groups=3),
        # a decode step of 128 requests on one document: the largest
        _case("shared_decode_128", "shared", 128, 1, 2047, 32, 4, 128, 64, "bfloat16", shared=32768, groups=1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("axes", "append", "sinks", "sinks", "shared", "shared"))
    D = rng.choice((64, 80, 96, 128, 128))
    Hkv = rng.choice((1, 2, 4, 5, 8))
    Hq = Hkv * rng.choice((1, 2, 3, 4, 5, 8) if Hkv < 8 else (1, 2, 4, 5))
    P = rng.choice((16, 16, 24, 32, 48, 64, 128))
    dtype = rng.choice(("bfloat16", "bfloat16", "float16"))
    nhd = rng.random() < 0.4
    if op in ("axes", "append"):
        R, A = rng.choice((D, D, D // 2)), rng.choice((2, 3, 3))
        turns, interleaved = rng.random() < 0.4, rng.random() < 0.4
        inverse = op == "axes" and rng.random() < 0.4
        if op == "axes":
            dtype = rng.choice((dtype, "float32"))
        q_len = rng.choice((1, _log_int(rng, 2, 2048)))
        B = _log_int(rng, 1, max(1, min(64, 4096 // q_len)))
        return _case(None, op, B, q_len, _log_int(rng, 1, 4096), Hq, Hkv, D, P, dtype, nhd, R, A, turns, interleaved, inverse)
    if op == "sinks":
        sinks = _log_int(rng, 1, 600)
        if rng.random() < 0.6:  # single tokens, or the few that a draft proposes
            q_len = rng.choice((1, 1, 1, rng.randint(2, 8)))
            B = _log_int(rng, 1, 64)
            ctx = _log_int(rng, 1, min(262144, 960_000_000 // (B * Hkv * D)))
            return _case(None, op, B, q_len, ctx, Hq, Hkv, D, P, dtype, nhd, window=_log_int(rng, 16, 8192), sinks=sinks)
        q_len = _log_int(rng, 16, 2048)  # chunks of a prompt
        B = _log_int(rng, 1, max(1, min(8, 4096 // q_len, (1 << 28) // (q_len * q_len * Hq))))
        ctx = rng.choice((0, _log_int(rng, 1, 8192)))
        ctx = min(ctx, max(0, (1 << 27) // (B * q_len * Hq) - q_len // 2))
        return _case(None, op, B, q_len, ctx, Hq, Hkv, D, P, dtype, nhd, window=_log_int(rng, 16, 4096), sinks=sinks)
    q_len = rng.choice((1, 1, 1, rng.randint(2, 8)))
    B = _log_int(rng, 2, 128 // q_len)
    groups = rng.choice((1, 1, _log_int(rng, 1, B)))
    shared = _log_int(rng, 16, min(32768, (1 << 17) // groups))
    ctx = _log_int(rng, 1, 2047)
    return _case(None, op, B, q_len, ctx, Hq, Hkv, D, P, dtype, nhd, shared=shared, groups=groups)


def _lens(c):
    """(new tokens, all tokens) of each sequence: the first has the full sizes, the others between a quarter and all."""
    part = [1.0 - 0.75 * ((0.6180339887 * b) % 1.0) for b in range(c["B"])]
    new = [max(1, int(c["q_len"] * f)) for f in part]
    even = c["ctx"] == 0
    if even:
        new = [c["q_len"]] * c["B"]
    held = [0 if even else int(c["ctx"] * f) for f in reversed(part[1:] + part[:1])]
    return new, [n + h + s for n, h, s in zip(new, held, _shared(c)[1])]


def _shared(c):
    """The groups' first sequences (and the end of the last), and the shared tokens of each sequence."""
    G, B = c["groups"], c["B"]
    if G == 0:
        return [], [0] * B
    first = [g * B // G for g in range(G + 1)]
    return first, [_shared_len(c, g) for g in range(G) for _ in range(first[g], first[g + 1])]


def _shared_len(c, g):
    return max(1, int(c["shared"] * (1.0 - 0.5 * ((0.6180339887 * g) % 1.0))))


def _axes(c):
    """The axis of each pair: a run for each axis, or turns while an axis has pairs left.  Three axes: time has fewer
    pairs than height and width in runs, more in turns."""
    n, A = c["R"] // 2, c["A"]
    if A == 2:
        sizes = [n - n // 2, n // 2]
    elif c["turns"]:
        sizes = [n - 2 * (5 * n // 16), 5 * n // 16, 5 * n // 16]
    else:
        sizes = [n - 2 * (3 * n // 8), 3 * n // 8, 3 * n // 8]
    if not c["turns"]:
        return [a for a in range(A) for _ in range(sizes[a])]
    got, left = [], list(sizes)
    while len(got) < n:
        for a in range(A):
            if left[a] > 0:
                left[a] -= 1
                got.append(a)
    return got


def _seen(c):
    """For each sequence, how many keys any of its rows sees, and how many (row, key) pairs there are."""
    got = []
    for n, s in zip(*_lens(c)):
        w, k = c["window"] or s, c["sinks"]
        first = max(0, s - n + 1 - w)
        at = np.arange(s - n, s, dtype=np.int64)
        got.append((s - first + min(first, k), int((np.minimum(at + 1, w) + np.minimum(np.maximum(at + 1 - w, 0), k)).sum())))
    return got


def work(case):
    c = case
    b = {"bfloat16": 2, "float16": 2, "float32": 4}[c["dtype"]]
    new, lens = _lens(c)
    N, heads = sum(new), c["Hq"] + c["Hkv"]
    table = N * (c["R"] * 4 + 4 * c["A"])  # each pair's cosine and sine, and the positions
    if c["op"] == "axes":
        return {"bytes": 2 * N * heads * c["D"] * b + table, "flops": 3 * N * heads * c["R"]}
    if c["op"] == "append":
        pages = sum(-(-s // c["P"]) - (s - n) // c["P"] for n, s in zip(new, lens))
        kv = 2 * N * c["Hkv"] * c["D"] * (b + 1) + 2 * 8 * pages * c["Hkv"]
        return {"bytes": kv + 2 * N * c["Hq"] * c["D"] * b + table, "flops": 3 * N * heads * c["R"] + 4 * N * c["Hkv"] * c["D"]}
    seen = _seen(c)
    keys, pairs = sum(k for k, _ in seen), sum(p for _, p in seen)
    first, each = _shared(c)
    keys -= sum(each) - sum(each[i] for i in first[:-1])  # a group's shared keys are read once
    cache = keys * c["Hkv"] * (2 * c["D"] + 8.0 / c["P"])
    return {"bytes": cache + N * c["Hq"] * (2 * c["D"] * b + 4), "flops": 4 * c["D"] * pairs * c["Hq"]}


# ------------------------------------------------------------------ inputs

def _frequencies(c):
    """The R / 2 angles per position in 64 bits: one falling line of them over all pairs, or for an image's two axes a line for each."""
    if c["A"] == 2:
        axes = _axes(c)
        size = [axes.count(0), axes.count(1)]
        at, got = [0, 0], []
        for a in axes:
            got.append(10000.0 ** (-at[a] / size[a]))
            at[a] += 1
        return np.array(got)
    return 10000.0 ** (-np.arange(0, c["R"], 2, dtype=np.float64) / c["R"])


def _media(n, start, A, rng):
    """Positions [A, n] of a sequence: text, whose axes are alike, and images and short videos as grids, each thing after all before it."""
    parts, have, at = [], 0, start
    while have < n:
        if A == 3:
            k = rng.integers(8, 60)
            parts.append(np.broadcast_to(at + np.arange(k), (3, k)))
            have, at = have + k, at + k
        t, h, w = (1 if A == 2 else rng.integers(1, 5)), rng.integers(4, 25), rng.integers(4, 25)
        grid = np.stack(np.meshgrid(np.arange(t), np.arange(h), np.arange(w), indexing="ij")).reshape(3, -1)[3 - A:]
        parts.append((at if A == 3 else 0) + grid)
        have, at = have + t * h * w, at + max(t, h, w)
    return np.concatenate(parts, axis=1)[:, :n]


def _positions(c, rng):
    new, lens = _lens(c)
    if c["q_len"] == 1 and c["A"] == 3:  # text that goes on after what came before
        return np.broadcast_to(np.array([s - 1 for s in lens]), (3, c["B"]))
    return np.concatenate([_media(n, (s - n) // 2, c["A"], rng) for n, s in zip(new, lens)], axis=1)


def _normal(shape, g, dev, dtype):
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)


def _codes(pages, c, g, dev):
    """Codes and scales of a cache that holds normal values whose size differs from head to head and page to page."""
    shape = (pages, c["Hkv"], c["P"], c["D"])
    codes = torch.empty(shape, dtype=torch.float8_e4m3fn, device=dev)
    scale = torch.exp2(torch.randint(-8, -5, shape[:2], generator=g, device=dev).float())
    step = max(1, (1 << 27) // (c["Hkv"] * c["P"] * c["D"]))
    for i in range(0, pages, step):
        x = torch.randn((min(step, pages - i), *shape[1:]), generator=g, device=dev)
        codes[i : i + step] = (x / scale[i : i + step, :, None, None]).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return codes, scale


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = getattr(torch, c["dtype"])
    new, lens = _lens(c)
    N, B, P = sum(new), c["B"], c["P"]
    s = dict(c, N=N, max_q=max(new), max_len=max(lens), scale=c["D"] ** -0.5)
    s["q"] = _normal((N, c["Hq"], c["D"]), g, dev, dt)
    if c["A"]:
        s["k"] = _normal((N, c["Hkv"], c["D"]), g, dev, dt)
        s["axes"] = bytes(_axes(c))
        s["axis_of_pair"] = torch.tensor(_axes(c), device=dev)
        pos = np.ascontiguousarray(_positions(c, np.random.default_rng(seed)), dtype=np.int32)
        s["positions"] = torch.from_numpy(pos).to(dev)
        at = torch.arange(int(pos.max()) + 1, dtype=torch.float64, device=dev)[:, None] * torch.from_numpy(_frequencies(c)).to(dev)
        s["cos_sin"] = torch.cat([at.cos(), at.sin()], dim=1).float()
    if c["op"] == "axes":
        return s
    s["cu_q"] = torch.from_numpy(np.cumsum([0] + new).astype(np.int32)).to(dev)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    first, each = _shared(c)
    # the whole pages of what a group shares are the same pages, the others lie anywhere; entries past the end are -1
    table, pages, copies = np.full((B, -(-max(lens) // P)), -1, dtype=np.int32), 0, []
    for b, (e, k) in enumerate(zip(lens, each)):
        lead = max([f for f in first[:-1] if f <= b], default=b)
        same = k // P if lead < b else 0
        table[b, :same] = table[lead, :same]
        more = -(-e // P) - same
        table[b, same : same + more] = np.arange(pages, pages + more)
        pages += more
        if lead < b and k % P:  # the page in which it ends is a copy
            copies.append((lead, b, same))
    order = torch.randperm(pages, generator=g, device=dev).int()
    table = torch.from_numpy(table).to(dev)
    table = torch.where(table < 0, table, order[table.clamp(min=0).long()])
    s["block_table"] = table
    for x in "kv":
        codes, scale = _codes(pages, c, g, dev)
        if copies:
            lead, b, at = torch.tensor(copies, device=dev).T
            into, of = table[b, at].long(), table[lead, at].long()
            codes.view(torch.uint8)[into] = codes.view(torch.uint8)[of]
            scale[into] = scale[of]
        if c["nhd"]:  # a page holds its tokens' heads one after another
            codes = codes.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(torch.float8_e4m3fn)
        s[x + "_codes"], s[x + "_scale"] = codes, scale
    if c["groups"]:
        s["shared_seqs"] = torch.tensor(first, dtype=torch.int32, device=dev)
        s["shared_lens"] = torch.tensor([each[i] for i in first[:-1]], dtype=torch.int32, device=dev)
        s["max_shared_q"] = max(sum(new[i:j]) for i, j in zip(first, first[1:]))
    if c["op"] == "append":  # a sixteenth as large scales on some pages: there the new tokens make the scale grow
        few = torch.rand(s["k_scale"].shape, generator=g, device=dev) < 0.3
        s["k_scale"] = torch.where(few, s["k_scale"] / 16, s["k_scale"])
        s["v"] = _normal((N, c["Hkv"], c["D"]), g, dev, dt)
    return s


# ------------------------------------------------------------------ the plain forms

def _rotate(x, s):
    """x [N, H, D] in 32 bits, its first R columns rotated, each pair by the position on its axis."""
    x, R = x.float(), s["R"]
    pair = torch.arange(R // 2, device=x.device)
    at = s["positions"].long()[s["axis_of_pair"]].T  # [N, R / 2]
    cos, sin = s["cos_sin"][at, pair][:, None], s["cos_sin"][at, R // 2 + pair][:, None]
    if s["inverse"]:
        sin = -sin
    if s["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., : R // 2], x[..., R // 2 : R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., R:]], dim=-1)


def _places(s):
    """The sequence and the place in it of each new token."""
    token = torch.arange(s["N"], dtype=torch.int32, device=s["cu_q"].device)
    seq = (torch.searchsorted(s["cu_q"], token, right=True) - 1).long()
    return seq, (s["seq_lens"][seq] - s["cu_q"][seq + 1] + token).long()


def _plain_axes(s):
    dt = s["q"].dtype
    return [_rotate(x, s).to(dt) for x in (s["q"], s["k"])]


def _plain_append_one(x, codes, scale, page, off, first_page, first_off):
    """x [N, Hkv, D] in 32 bits into codes [pages, Hkv, P, D] at (page, off); the scales are powers of two."""
    m, e = torch.frexp(x.abs().amax(-1))  # [N, Hkv]; 448 = 0.875 * 2 ** 9
    need = torch.exp2((e - torch.where(m <= 0.875, 9, 8)).clamp(min=-42).float())
    touched = torch.zeros_like(scale).index_reduce_(0, page, need, "amax")
    fresh = torch.zeros(scale.shape[0], dtype=torch.bool, device=x.device).index_fill_(0, page, True)
    fresh[first_page] = first_off == 0
    grown = torch.maximum(torch.where(fresh[:, None], 0.0, scale), touched)
    ratio = (scale / grown)[first_page][:, :, None, None]  # what the first page of each sequence holds already
    held = torch.arange(codes.shape[2], device=x.device)[None, None, :, None] < first_off[:, None, None, None]
    old = codes.view(torch.uint8)
    was = codes.view(torch.uint8)[first_page].view(torch.float8_e4m3fn)
    old[first_page] = torch.where(held, (was.float() * ratio).to(torch.float8_e4m3fn).view(torch.uint8), was.view(torch.uint8))
    old[page, :, off] = (x / grown[page][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_(grown)


def _plain_append(s):
    seq, place = _places(s)
    table = s["block_table"].long()
    page, off = table[seq, place // s["P"]], place % s["P"]
    start = s["seq_lens"].long() - (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    first_page, first_off = table.gather(1, (start // s["P"])[:, None])[:, 0], start % s["P"]
    _plain_append_one(_rotate(s["k"], s), s["k_codes"], s["k_scale"], page, off, first_page, first_off)
    _plain_append_one(s["v"].float(), s["v_codes"], s["v_scale"], page, off, first_page, first_off)
    # codes are float8 values and their scales stand beside them: together what the cache stands for
    return dict(q=_rotate(s["q"], s).to(s["q"].dtype), k_codes=s["k_codes"], v_codes=s["v_codes"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _gathered(codes, scale, table):
    """[B, Hkv, keys, D] in 32 bits."""
    x = codes.view(torch.uint8)[table].view(torch.float8_e4m3fn).float().mul_(scale[table][..., None, None])
    return x.transpose(1, 2).flatten(2, 3)


def _plain_attend(s):
    G, Hkv, D, B, T = s["Hq"] // s["Hkv"], s["Hkv"], s["D"], s["B"], s["max_q"]
    table = s["block_table"].clamp(min=0).long()
    count = (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    step = torch.arange(T, device=table.device)
    rows = (s["cu_q"][:-1, None].long() + step).clamp(max=s["N"] - 1)
    q = s["q"].float()[rows].view(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
    score = (q @ _gathered(s["k_codes"], s["k_scale"], table).transpose(-1, -2)).mul_(s["scale"]).view(B, Hkv, G, T, -1)
    at = (s["seq_lens"].long() - count)[:, None] + step  # [B, T]: each row's position
    key = torch.arange(score.shape[-1], device=table.device)
    seen = (key > at[..., None] - (s["window"] or 1 << 40)) | (key < s["sinks"])
    seen = (key <= at[..., None]) & seen & (step < count[:, None])[..., None]
    score = score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, Hkv, G * T, -1) @ _gathered(s["v_codes"], s["v_scale"], table)).view(B, Hkv, G, T, D)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + total.log())[..., 0]
    seq, place = _places(s)
    t = place - (s["seq_lens"].long() - count)[seq]
    return dict(out=out.permute(0, 3, 1, 2, 4)[seq, t].reshape(s["N"], s["Hq"], D).to(s["q"].dtype), lse=lse.permute(0, 3, 1, 2)[seq, t].reshape(s["N"], s["Hq"]))


# ------------------------------------------------------------------ one pass

def _cache(s):
    """The handle that a user's program keeps for its cache."""
    if "cache" not in s:
        import moe_lora_expert_gb300 as m

        s["cache"] = m.PagedKVCache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"])
    return s["cache"]


def run(state):
    s = state
    if not own:
        return {"axes": _plain_axes, "append": _plain_append}.get(s["op"], _plain_attend)(s)
    if s["op"] == "axes":
        import moe_lora_expert_gb300 as m

        return list(m.moe_rope(s["q"], s["positions"], s["cos_sin"], k=s["k"], interleaved=s["interleaved"], inverse=s["inverse"], axes=s["axes"]))
    if s["op"] == "append":
        q = _cache(s).append(s["k"], s["v"], s["block_table"], s["seq_lens"], cu_q=s["cu_q"], max_q_len=s["max_q"], q=s["q"], cos_sin=s["cos_sin"],
                             interleaved=s["interleaved"], positions=s["positions"], axes=s["axes"])
        return dict(q=q, k_codes=s["k_codes"], v_codes=s["v_codes"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    how = dict(window=s["window"], sinks=s["sinks"])
    if s["op"] == "shared":
        how = dict(shared_lens=s["shared_lens"], shared_seqs=s["shared_seqs"], max_shared_q=s["max_shared_q"])
    out, lse = _cache(s).attend(s["q"], s["block_table"], s["seq_lens"], cu_q=s["cu_q"], max_q_len=s["max_q"], max_seq_len=s["max_len"], scale=s["scale"],
                                return_lse=True, **how)
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------ in 64 bits

def _exact_turn(x, s, sign):
    """x [n, H, D] in 64 bits, with the angles from their definition."""
    f = torch.from_numpy(_frequencies(s)).to(x.device)
    on = torch.stack([s["positions"][a].to(torch.float64) for a in _axes(s)], dim=1)  # [n, R / 2]
    angle = (on * f)[:, None, :]
    z = torch.polar(torch.ones_like(angle), sign * angle)
    head, rest = x[..., : s["R"]], x[..., s["R"] :]
    pairs = head.unflatten(-1, (-1, 2)) if s["interleaved"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    return torch.cat([(turned if s["interleaved"] else turned.transpose(-1, -2)).flatten(-2), rest], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    d = lambda x: x.to(torch.float64)  # noqa: E731
    if c["op"] == "axes":
        return [_exact_turn(d(s[x]), s, -1.0 if c["inverse"] else 1.0) for x in ("q", "k")]
    new, lens = _lens(c)
    if c["op"] == "append":
        table = s["block_table"].tolist()
        got = dict(q=_exact_turn(d(s["q"]), s, 1.0))
        for name, x in (("k", _exact_turn(d(s["k"]), s, 1.0)), ("v", d(s["v"]))):
            codes, scale = d(s[name + "_codes"]), d(s[name + "_scale"])
            at = 0
            for b, (n, e) in enumerate(zip(new, lens)):
                p = e - n
                while p < e:  # one page at a time
                    page, off = table[b][p // c["P"]], p % c["P"]
                    k = min(c["P"] - off, e - p)
                    y = x[at : at + k]
                    was = scale[page] if off else torch.zeros_like(scale[page])
                    big = y.abs().amax((0, 2)).clamp(min=1e-300)
                    now = torch.maximum(was, torch.exp2(torch.ceil(torch.log2(big / 448)).clamp(min=-42)))
                    codes[page, :, :off] = _to_e4m3(codes[page, :, :off] * (was / now)[:, None, None])
                    codes[page, :, off : off + k] = _to_e4m3(y.transpose(0, 1) / now[:, None, None])
                    scale[page] = now
                    p, at = p + k, at + k
            got[name + "_codes"], got[name + "_scale"] = codes, scale
        return got
    outs, lses, at = [], [], 0
    for b, (n, e) in enumerate(zip(new, lens)):
        pages = s["block_table"][b, : -(-e // c["P"])].long()
        q = d(s["q"][at : at + n])
        at += n
        row = torch.arange(e - n, e, device=q.device)[:, None]
        key = torch.arange(e, device=q.device)[None]
        hidden = (key > row) | ((key <= row - c["window"]) & (key >= c["sinks"]) if c["window"] else torch.zeros_like(key, dtype=torch.bool))
        k, v = ((d(s[x + "_codes"].view(torch.uint8)[pages].view(torch.float8_e4m3fn)) * d(s[x + "_scale"][pages])[:, :, None, None]).transpose(0, 1).flatten(1, 2)
                for x in "kv")
        some = slice(0, e)
        if n == 1 and c["window"]:  # one row: only the keys that it sees
            some = (~hidden[0]).nonzero()[:, 0]
        hidden = hidden[:, some]
        each = c["Hq"] // c["Hkv"]
        for h in range(c["Hkv"]):
            kh, vh = k[h][some], v[h][some]
            score = (torch.einsum("nhd,kd->hnk", q[:, h * each : (h + 1) * each], kh) * s["scale"]).masked_fill(hidden, float("-inf"))
            lses.append(torch.logsumexp(score, -1))
            outs.append(torch.softmax(score, -1) @ vh)
    # a list of [heads of one key head, rows, ...] for each sequence and key head
    H = c["Hkv"]
    join = lambda xs: torch.cat([torch.cat(xs[i : i + H]).transpose(0, 1) for i in range(0, len(xs), H)])  # noqa: E731
    return dict(out=join(outs), lse=join(lses))


def _to_e4m3(x):
    """The nearest values that e4m3 has (ties to the even code), in 64 bits."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0**-6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)
