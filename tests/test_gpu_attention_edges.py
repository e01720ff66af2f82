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
