"""Which calls over shared prefixes are the plain call, by the sizes that the host
has, and the scratch that the others need, without a GPU."""
import pytest

import moe_lora_expert_gb300 as m
from test_attention_forms_host import shared
from test_attention_host import FAKE, attend_args, lib  # noqa: F401


def scratch(lib, over=None, more=None, cache=None):  # noqa: F811
    """Bytes for a call of 4 sequences on 4 key heads with 8 query heads each and
    contexts of up to 2^20 tokens, or what differs from it."""
    args = attend_args(lib, cache_over=cache, **{"max_seq_len": 1 << 20, "table_width": 1 << 16, **(over or {})})
    return lib.moe_paged_attention_shared_partial_size(bytes(args), shared(lib, **{"groups": 1, "seqs": None, **(more or {})}))


def test_scratch_of_a_call_that_shares(lib):  # noqa: F811
    want = scratch(lib)
    assert want >= lib.moe_shared_prefix_partial_size(4, 32, 128, 1) > 0
    assert scratch(lib, more={"partial": None, "partial_bytes": 0}) == want        # its own are not read


@pytest.mark.parametrize("over,more", [
    ({"max_seq_len": 128}, {}),                                                    # short contexts
    ({"N": 2, "B": 2}, {}), ({}, {"max_tokens": 3}),                               # few rows in a group
    ({"N": 4096, "max_q_len": 1024, "cu_q": FAKE}, {"max_tokens": 4096}),          # many in each sequence
    ({}, {"groups": 0}), ({}, {"max_tokens": 0}), ({"N": 0, "B": 0}, {}),
    ({"table_width": 1 << 30}, {}),                                                # tables past what the kernels count
    ({"q": None}, {}), ({"window": 5}, {}), ({}, {"struct_size": 8}), ({}, {"groups": -1})])   # refused by the call
def test_no_scratch_for_the_plain_call(lib, over, more):  # noqa: F811
    assert scratch(lib, over, more) == 0


def test_no_scratch_without_arguments(lib):  # noqa: F811
    assert lib.moe_paged_attention_shared_partial_size(None, shared(lib)) == lib.moe_paged_attention_shared_partial_size(bytes(attend_args(lib)), None) == 0


@pytest.mark.parametrize("more", [dict(partial=None, partial_bytes=0), dict(partial=None), dict(partial=FAKE + 16), dict(partial_bytes=64)])
def test_a_call_that_shares_is_refused_without_scratch(lib, more):  # noqa: F811
    args = attend_args(lib, max_seq_len=1 << 20, table_width=1 << 16)
    assert lib.moe_paged_attention_shared(bytes(args), shared(lib, groups=1, seqs=None, **more), None) == m.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("heads", [1, 2, 3])
def test_few_key_heads_may_leave_a_piece_on_each_sm(lib, heads):  # noqa: F811
    """One unit for each key head, cut for 152 SMs: 32 pieces would leave most idle."""
    rows, row = 4 * 8 * heads, 4 * 128 + 8
    size = scratch(lib, over={"Hq": 8 * heads}, cache={"kv_heads": heads})
    pieces = (size - 4) // (rows * row) - 1
    assert size == (pieces + 1) * rows * row + 4 and pieces == 160 // heads


@pytest.mark.parametrize("B,groups,heads,most,longest,pays", [
    (8, 1, 4, None, 2349, False), (8, 2, 4, 4, 2349, False),                  # the plain call is done before three kernels are launched
    (8, 1, 4, None, 16685, True), (8, 1, 1, None, 16685, False), (8, 1, 1, None, 65837, True),
    (64, 1, 4, None, 1 << 20, True), (64, 1, 4, None, 9216, True), (64, 1, 4, None, 2349, False),
    (32, 16, 4, None, 65837, False), (32, 16, 4, 2, 65837, False),            # groups of two, with the bound and without
    (16, 8, 4, None, 65837, False), (8, 4, 4, None, 65837, False),
    (32, 8, 4, 4, 4397, False), (32, 8, 4, 4, 16685, True), (64, 16, 4, 4, 65837, False),
    (64, 8, 4, 8, 1325, False), (64, 8, 4, 8, 8493, True), (320, 40, 4, 8, 8493, True),
    (9, 4, 4, 9, 1 << 20, False), (9, 4, 2, 9, 1 << 20, True), (9, 4, 2, 3, 1 << 20, False)])   # an uneven list of few units
def test_which_calls_share(lib, B, groups, heads, most, longest, pays):  # noqa: F811
    """One new token a sequence, 8 query heads a key head: both sides are measured beside the rule."""
    got = scratch(lib, over={"B": B, "N": B, "Hq": 8 * heads, "max_seq_len": longest}, cache={"kv_heads": heads},
                  more={"groups": groups, "seqs": FAKE, "max_tokens": B if most is None else most})
    assert (got > 0) == pays
