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
