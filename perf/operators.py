"""Rotary positions, the 8-bit paged cache and the attention over it: the cases that are timed, and their plain forms.

A case names one of three operators ("op"):

  rope    moe_rope: q and k rotated by their positions; "inverse" is the gradient.
  append  moe_kv_append: the keys (rotated) and values of new tokens into the paged e4m3 cache, one scale for each
          (page, head), with the queries rotated in the same call.
  attend  moe_paged_attention: causal attention of the new tokens over that cache, with the log-sum-exp of each row.

Shapes follow the routed layer of workloads.py where they can (hidden 2048: 4096 prefill tokens as 2 x 2048, 16 and 64
decode tokens); the others are generic odd ones.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases

def _case(name, op, B, q_len, ctx, Hq, Hkv, D, R, P, dtype, nhd=False, interleaved=False, inverse=False, window=0, scaling="none"):
    """B sequences of up to q_len new tokens each, on top of up to ctx tokens that the cache holds already."""
    c = dict(op=op, B=B, q_len=q_len, ctx=ctx, Hq=Hq, Hkv=Hkv, D=D, R=R, P=P, dtype=dtype, nhd=nhd, interleaved=interleaved, inverse=inverse, window=window,
             scaling=scaling)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one decode step of 16 sequences: 16 tokens' q and k, where the launch counts
        _case("rope_decode_16", "rope", 16, 1, 2048, 32, 4, 128, 128, 16, "bfloat16"),
        # a prefill of 2 x 2048 tokens with the positions of a context stretched four times (yarn)
        _case("rope_prefill_4096", "rope", 2, 2048, 0, 32, 4, 128, 128, 16, "bfloat16", scaling="yarn"),
        # the backward pass of a model that rotates 32 of 80 columns in neighbouring pairs, float32, odd lengths
        _case("rope_grad_partial", "rope", 3, 1021, 5, 20, 20, 80, 32, 16, "float32", interleaved=True, inverse=True, scaling="linear"),
        # one decode step of 64 sequences: one token each onto pages that are partly full
        _case("append_decode_64", "append", 64, 1, 4096, 32, 4, 128, 128, 16, "bfloat16"),
        # a prefill of 2 x 2048 tokens into fresh pages
        _case("append_prefill_4096", "append", 2, 2048, 0, 32, 4, 128, 128, 64, "bfloat16"),
        # ragged chunks that begin and end inside pages of 24 tokens, tokens before heads in a page, half of the head rotated
        _case("append_ragged", "append", 7, 701, 333, 15, 5, 80, 48, 24, "float16", nhd=True, interleaved=True, scaling="llama3"),
        # one user's next token at a short context: latency
        _case("attend_decode_1", "attend", 1, 1, 1021, 32, 4, 128, 128, 16, "bfloat16"),
        # a decode step of 16 sequences of ragged contexts up to 4096
        _case("attend_decode_16", "attend", 16, 1, 4095, 32, 4, 128, 128, 16, "bfloat16"),
        # a decode step of 64 sequences with long contexts: the bandwidth of the cache
        _case("attend_decode_64", "attend", 64, 1, 32767, 32, 4, 128, 128, 64, "bfloat16"),
        # one token on a context of a quarter million: the split over the long axis
        _case("attend_decode_long", "attend", 1, 1, 262139, 32, 4, 128, 128, 32, "bfloat16"),
        # the prefill of 2 x 2048 tokens
        _case("attend_prefill_4096", "attend", 2, 2048, 0, 32, 4, 128, 128, 64, "bfloat16"),
        # ragged chunks of up to 1000 tokens on up to 8191 earlier ones, sliding window, 64-wide heads, pages of 48, float16
        _case("attend_chunk_window", "attend", 4, 1000, 8191, 20, 5, 64, 64, 48, "float16", nhd=True, window=4096),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "attend", "attend"))
    D = rng.choice((64, 80, 96, 128, 128))
    R = rng.choice((D, D, D // 2))
    Hkv = rng.choice((1, 2, 4, 5, 8))
    Hq = Hkv * rng.choice((1, 2, 3, 4, 5, 8) if Hkv < 8 else (1, 2, 4, 5))
    D = 128 if Hq * D > 2048 else D
    P = rng.choice((16, 16, 24, 32, 48, 64, 128))
    dtype = rng.choice(("bfloat16", "bfloat16", "float16"))
    nhd, interleaved = rng.random() < 0.4, rng.random() < 0.4
    scaling = rng.choice(("none", "linear", "yarn", "llama3"))
    window, inverse = 0, False
    if op == "rope":
        inverse = rng.random() < 0.4
        dtype = rng.choice((dtype, "float32"))
        q_len = _log_int(rng, 1, 2048)
        B = _log_int(rng, 1, max(1, 4096 // q_len))
        ctx = _log_int(rng, 1, 30000)
    elif op == "append":
        q_len = rng.choice((1, _log_int(rng, 2, 2048)))
        B = _log_int(rng, 1, max(1, min(64, 4096 // q_len)))
        ctx = _log_int(rng, 1, 4096)
    elif rng.random() < 0.6:  # single tokens, or the few that a draft proposes
        q_len = rng.choice((1, 1, 1, rng.randint(2, 8)))
        B = _log_int(rng, 1, 64)
        ctx = _log_int(rng, 1, min(262144, 960_000_000 // (B * Hkv * D)))
        window = rng.choice((0, 0, 0, 1 + ctx // 3))
    else:  # chunks of a prompt
        q_len = _log_int(rng, 16, 2048)
        B = _log_int(rng, 1, max(1, min(8, 4096 // q_len, (1 << 28) // (q_len * q_len * Hq))))
        ctx = rng.choice((0, _log_int(rng, 1, 8192)))
        ctx = min(ctx, max(0, (1 << 27) // (B * q_len * Hq) - q_len // 2))
        window = rng.choice((0, 0, 0, 1 + (ctx + q_len) // 3))
    return _case(None, op, B, q_len, ctx, Hq, Hkv, D, R, P, dtype, nhd, interleaved, inverse, window, scaling)


def _lens(c):
    """(new tokens, tokens after them) of each sequence: the first has the full sizes, the others between a quarter and all."""
    part = [1.0 - 0.75 * ((0.6180339887 * b) % 1.0) for b in range(c["B"])]
    new = [max(1, int(c["q_len"] * f)) for f in part]
    even = c["ctx"] == 0
    if even:
        new = [c["q_len"]] * c["B"]
    return new, [n + (0 if even else int(c["ctx"] * f)) for n, f in zip(new, reversed(part[1:] + part[:1]))]


def _seen(c):
    """For each sequence, how many keys of the cache any of its rows sees, and how many (row, key) pairs there are."""
    got = []
    for n, s in zip(*_lens(c)):
        w = c["window"] or s
        first = max(0, s - n + 1 - w)
        at = np.arange(s - n, s, dtype=np.int64)
        got.append((s - first, int(np.minimum(at + 1, w).sum())))
    return got


def work(case):
    c = case
    b = {"bfloat16": 2, "float16": 2, "float32": 4}[c["dtype"]]
    N, heads = sum(_lens(c)[0]), c["Hq"] + c["Hkv"]
    table = N * (c["R"] * 4 + 4)
    if c["op"] == "rope":
        return {"bytes": 2 * N * heads * c["D"] * b + table, "flops": 3 * N * heads * c["R"]}
    if c["op"] == "append":
        pages = sum(-(-s // c["P"]) - (s - n) // c["P"] for n, s in zip(*_lens(c)))
        kv = 2 * N * c["Hkv"] * c["D"] * (b + 1) + 2 * 8 * pages * c["Hkv"]
        return {"bytes": kv + 2 * N * c["Hq"] * c["D"] * b + table, "flops": 3 * N * heads * c["R"] + 4 * N * c["Hkv"] * c["D"]}
    seen = _seen(c)
    keys, pairs = sum(k for k, _ in seen), sum(p for _, p in seen)
    cache = keys * c["Hkv"] * (2 * c["D"] + 8.0 / c["P"])
    return {"bytes": cache + N * c["Hq"] * (2 * c["D"] * b + 4), "flops": 4 * c["D"] * pairs * c["Hq"]}


# ------------------------------------------------------------------ inputs

def _frequencies(R, scaling):
    """The R / 2 angles per position, and the factor on cos and sin, in 64 bits."""
    base = 10000.0
    f = base ** (-np.arange(0, R, 2, dtype=np.float64) / R)
    if scaling == "linear":
        return f / 4.0, 1.0
    if scaling == "yarn":  # stretched 4 times from 4096: fast angles kept, slow ones divided, a ramp between
        turn = lambda r: R * math.log(4096 / (r * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(turn(32)), 0), min(math.ceil(turn(1)), R - 1)
        ramp = np.clip((np.arange(R // 2) - lo) / max(hi - lo, 1e-3), 0, 1)
        return f * (1 - ramp) + f / 4.0 * ramp, 0.1 * math.log(4.0) + 1.0
    if scaling == "llama3":  # stretched 8 times from 8192, between wavelengths of 8192 and 8192 / 4
        wave = 2 * math.pi / f
        smooth = np.clip((8192 / wave - 1.0) / (4.0 - 1.0), 0, 1)
        return f / 8.0 * (1 - smooth) + f * smooth, 1.0
    return f, 1.0


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
    if c["nhd"]:  # a page holds its tokens' heads one after another
        codes = codes.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2).view(torch.float8_e4m3fn)
    return codes, scale


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = getattr(torch, c["dtype"])
    new, lens = _lens(c)
    N = sum(new)
    s = dict(c, N=N, max_q=max(new), max_len=max(lens), scale=c["D"] ** -0.5)
    s["q"] = _normal((N, c["Hq"], c["D"]), g, dev, dt)
    if c["op"] != "attend":
        s["k"] = _normal((N, c["Hkv"], c["D"]), g, dev, dt)
        f, m = _frequencies(c["R"], c["scaling"])
        at = torch.arange(max(lens), dtype=torch.float64, device=dev)[:, None] * torch.from_numpy(f).to(dev)
        s["cos_sin"] = torch.cat([at.cos() * m, at.sin() * m], dim=1).float()
    cu = np.cumsum([0] + new)
    s["positions"] = torch.from_numpy(np.concatenate([np.arange(e - n, e) for n, e in zip(new, lens)]).astype(np.int32)).to(dev)
    if c["op"] == "rope":
        return s
    s["cu_q"] = torch.from_numpy(cu.astype(np.int32)).to(dev)
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    wide = -(-max(lens) // c["P"])
    held = torch.tensor([-(-e // c["P"]) for e in lens], device=dev)[:, None] > torch.arange(wide, device=dev)
    pages = int(held.sum())
    table = torch.full((c["B"], wide), -1, dtype=torch.int32, device=dev)
    table[held] = torch.randperm(pages, generator=g, device=dev).int()  # the pages lie anywhere; entries past the end are -1
    s["block_table"] = table
    s["k_codes"], s["k_scale"] = _codes(pages, c, g, dev)
    s["v_codes"], s["v_scale"] = _codes(pages, c, g, dev)
    if c["op"] == "append":  # a sixteenth as large scales on some pages: there the new tokens make the scale grow
        few = torch.rand(s["k_scale"].shape, generator=g, device=dev) < 0.3
        s["k_scale"] = torch.where(few, s["k_scale"] / 16, s["k_scale"])
        s["v"] = _normal((N, c["Hkv"], c["D"]), g, dev, dt)
    return s


# ------------------------------------------------------------------ the plain forms

def _rotate(x, positions, cos_sin, R, interleaved, inverse):
    """x [N, H, D] in 32 bits, its first R columns rotated."""
    x = x.float()
    cos, sin = cos_sin[positions.long()][:, None, :].split(R // 2, dim=-1)
    if inverse:
        sin = -sin
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., : R // 2], x[..., R // 2 : R]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., R:]], dim=-1)


def _places(s):
    """The sequence and the position of each new token."""
    seq = torch.searchsorted(s["cu_q"], torch.arange(s["N"], dtype=torch.int32, device=s["cu_q"].device), right=True) - 1
    return seq, s["positions"].long()


def _plain_rope(s):
    dt = s["q"].dtype
    return [_rotate(x, s["positions"], s["cos_sin"], s["R"], s["interleaved"], s["inverse"]).to(dt) for x in (s["q"], s["k"])]


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
    seq, pos = _places(s)
    table = s["block_table"].long()
    page, off = table[seq, pos // s["P"]], pos % s["P"]
    start = s["seq_lens"].long() - (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    first_page, first_off = table.gather(1, (start // s["P"])[:, None])[:, 0], start % s["P"]
    turn = lambda x: _rotate(x, s["positions"], s["cos_sin"], s["R"], s["interleaved"], False)  # noqa: E731
    _plain_append_one(turn(s["k"]), s["k_codes"], s["k_scale"], page, off, first_page, first_off)
    _plain_append_one(s["v"].float(), s["v_codes"], s["v_scale"], page, off, first_page, first_off)
    # codes are float8 values and their scales stand beside them: together what the cache stands for
    return dict(q=turn(s["q"]).to(s["q"].dtype), k_codes=s["k_codes"], v_codes=s["v_codes"], k_scale=s["k_scale"], v_scale=s["v_scale"])


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
    seen = (key <= at[..., None]) & (key > at[..., None] - (s["window"] or 1 << 40)) & (step < count[:, None])[..., None]
    score = score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, Hkv, G * T, -1) @ _gathered(s["v_codes"], s["v_scale"], table)).view(B, Hkv, G, T, D)
    out = torch.where(total > 0, out / total, 0.0)
    lse = (top + total.log())[..., 0]
    seq, pos = _places(s)
    t = pos - (s["seq_lens"].long() - count)[seq]
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
        return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)
    if s["op"] == "rope":
        import moe_lora_expert_gb300 as m

        return list(m.moe_rope(s["q"], s["positions"], s["cos_sin"], k=s["k"], interleaved=s["interleaved"], inverse=s["inverse"]))
    if s["op"] == "append":
        q = _cache(s).append(s["k"], s["v"], s["block_table"], s["seq_lens"], cu_q=s["cu_q"], max_q_len=s["max_q"], q=s["q"], cos_sin=s["cos_sin"],
                             interleaved=s["interleaved"])
        return dict(q=q, k_codes=s["k_codes"], v_codes=s["v_codes"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    out, lse = _cache(s).attend(s["q"], s["block_table"], s["seq_lens"], cu_q=s["cu_q"], max_q_len=s["max_q"], max_seq_len=s["max_len"], scale=s["scale"],
                                window=s["window"], return_lse=True)
    return dict(out=out, lse=lse)


# ------------------------------------------------------------------ in 64 bits

def _exact_turn(x, pos, c, sign):
    """x [n, H, D] in 64 bits, with the angles from their definition."""
    f, m = _frequencies(c["R"], c["scaling"])
    angle = pos[:, None, None] * torch.from_numpy(f).to(x.device)
    z = torch.polar(torch.full_like(angle, m), sign * angle)
    head, rest = x[..., : c["R"]], x[..., c["R"] :]
    pairs = head.unflatten(-1, (-1, 2)) if c["interleaved"] else head.unflatten(-1, (2, -1)).transpose(-1, -2)
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z)
    return torch.cat([(turned if c["interleaved"] else turned.transpose(-1, -2)).flatten(-2), rest], -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    d = lambda x: x.to(torch.float64)  # noqa: E731
    pos = d(s["positions"])
    if c["op"] == "rope":
        return [_exact_turn(d(s[x]), pos, c, -1.0 if c["inverse"] else 1.0) for x in ("q", "k")]
    new, lens = _lens(c)
    table = s["block_table"].tolist()
    if c["op"] == "append":
        got = dict(q=_exact_turn(d(s["q"]), pos, c, 1.0))
        for name, x in (("k", _exact_turn(d(s["k"]), pos, c, 1.0)), ("v", d(s["v"]))):
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
        hidden = (key > row) | ((key <= row - c["window"]) if c["window"] else torch.zeros_like(key, dtype=torch.bool))
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
        for h in range(c["Hq"]):
            kv, first = divmod(h, c["Hq"] // c["Hkv"])
            if first == 0:
                k, v = ((d(s[x + "_codes"].view(torch.uint8)[pages, kv].view(torch.float8_e4m3fn)) * d(s[x + "_scale"][pages, kv])[:, None, None]).flatten(0, 1)[:e]
                        for x in "kv")
            score = ((q[:, h] @ k.T) * s["scale"]).masked_fill(hidden, float("-inf"))
            lse[:, h] = torch.logsumexp(score, -1)
            out[:, h] = torch.softmax(score, -1) @ v
        outs.append(out)
        lses.append(lse)
    return dict(out=torch.cat(outs), lse=torch.cat(lses))


def _to_e4m3(x):
    """The nearest values that e4m3 has (ties to the even code), in 64 bits."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0**-6)))
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)
