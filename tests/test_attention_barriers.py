"""The order that the prefix pass's barriers keep between its roles, on the CPU:
every interleaving of a small model of it ends.

The model: pieces of one key tile each, one after another in a CTA.  A barrier
completes a phase when it has its count of arrivals, and a wait names a phase by
its parity alone, so a role that is late by two phases waits for one that may
never come.  Counts, and who arrives, are taken from the source.
"""
import re

import pytest

from test_attention_source import body, code

STAGES, SLOTS = 2, 4
SOFTMAX, CONVERT = 2, 2          # warps of the model; 8 and 4 in the kernel


def source():
    """(arrivals that end a phase of q_empty, whether the converting warps are
    among them) in the prefix pass."""
    text = code("prefill_attention.cu")
    count = re.search(r"mbar_init\(&s\.q_empty, (.*?)\);", text).group(1)
    count = re.sub(r"kIsPrefix \? (\w+) : (\w+)", r"(\1 if kIsPrefix else \2)", count).replace("/", "//")
    count = eval(count, {"kTileRows": 128, "kIsPrefix": True})
    converting = text[text.index("else if (warp >= kConvertWarp && warp < kMmaWarp)"):]
    converting = body(converting, "else if")
    return count, "mbar_arrive(&s.q_empty)" in converting


def roles(units, converters_arrive):
    """Each role as a list of steps: ("wait", barrier, phase) or ("arrive", barrier).
    Copies arrive on their own, right when they are issued."""
    load, mma = [], []
    soft, convert = ([[] for _ in range(n)] for n in (SOFTMAX, CONVERT))
    for u in range(units):
        for v in (0, 1):
            n = 2 * u + v
            st = n % STAGES
            if n >= STAGES:
                load.append(("wait", f"code_empty{st}", n // STAGES - 1))
            load.append(("arrive", f"code_full{st}"))
            if v == 0:
                if u > 0:
                    load.append(("wait", "q_empty", u - 1))
                load.append(("arrive", "q_raw"))
            for warp in convert:
                warp.append(("wait", f"code_full{st}", n // STAGES))
                if n >= SLOTS:
                    warp.append(("wait", f"empty{n % SLOTS}", n // SLOTS - 1))
                warp += [("arrive", f"code_empty{st}"), ("arrive", f"full{n % SLOTS}")]
                if v == 0:
                    warp.append(("wait", "q_raw", u))
                    if converters_arrive:
                        warp.append(("arrive", "q_empty"))
        for warp in soft:
            warp += [("wait", "q_raw", u), ("arrive", "q_full"), ("arrive", "q_empty"), ("wait", "s_full", u), ("arrive", "p_full"), ("wait", "o_full", u)]
        k, v = 2 * u, 2 * u + 1
        mma += [("wait", "q_full", u), ("wait", f"full{k % SLOTS}", k // SLOTS), ("arrive", "s_full"), ("arrive", f"empty{k % SLOTS}"), ("arrive", "q_empty"),
                ("wait", f"full{v % SLOTS}", v // SLOTS), ("wait", "p_full", u), ("arrive", f"empty{v % SLOTS}"), ("arrive", "o_full")]
    return [load, mma, *soft, *convert]


def stuck(units, converters_arrive):
    """A state from which no role can go on though some have not ended, or None."""
    steps = roles(units, converters_arrive)
    count = {"q_full": SOFTMAX, "p_full": SOFTMAX, "q_empty": 1 + SOFTMAX + (CONVERT if converters_arrive else 0)}
    for i in range(STAGES):
        count[f"code_empty{i}"] = CONVERT
    for i in range(SLOTS):
        count[f"full{i}"] = CONVERT
    names = sorted({s[1] for role in steps for s in role})
    index = {n: i for i, n in enumerate(names)}
    seen, todo = set(), [(tuple(0 for _ in steps), tuple(0 for _ in names))]
    while todo:
        at, arrived = todo.pop()
        if (at, arrived) in seen:
            continue
        seen.add((at, arrived))
        moved = False
        for r, role in enumerate(steps):
            if at[r] == len(role):
                continue
            kind, name, *phase = role[at[r]]
            i, each = index[name], count.get(name, 1)
            if kind == "wait" and (arrived[i] // each) % 2 == phase[0] % 2:      # the phase of that parity is the one under way
                continue
            moved = True
            new = arrived if kind == "wait" else arrived[:i] + (arrived[i] + 1,) + arrived[i + 1:]
            todo.append((at[:r] + (at[r] + 1,) + at[r + 1:], new))
        if not moved and any(a < len(role) for a, role in zip(at, steps)):
            return at
    return None


def test_the_model_sees_a_missing_arrival():
    """Without the converting warps' word the queries of the next piece may come
    before such a warp has looked for this one's."""
    assert stuck(2, converters_arrive=False) is not None


@pytest.mark.parametrize("units", [1, 2, 3, 4])
def test_every_order_of_pieces_of_one_tile_ends(units):
    count, converters_arrive = source()
    assert count == 1 + 8 + (4 if converters_arrive else 0)      # the products, the rows' warps, the converting warps
    assert stuck(units, converters_arrive) is None
