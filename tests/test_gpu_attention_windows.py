"""Windows of any size, against the float64 oracle."""
import numpy as np
import pytest

import moe_lora_expert_gb300 as m
from test_gpu_attention import Batch, rounded, tensor
from test_gpu_attention_forms import compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new,lens", [([6, 1], [4, 30]), ([200, 3], [150, 1])])
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 7), (2 ** 31 - 3, 0), (1 << 30, 2)])
def test_a_window_past_any_position(new, lens, window, sinks):
    """As no window at all, with more new tokens than the sequence holds too,
    whose first rows come before the first key and see none."""
    rng = np.random.default_rng(window % 97 + sinks)
    batch = Batch(rng, new, lens, 2, 16, 64, std=0.5)
    q = rounded(rng, (sum(new), 8, 64), "bfloat16")
    out, lse = batch.cache.attend(tensor(q, "bfloat16"), **batch.dev, cu_q=batch.cu_dev, max_q_len=max(new), window=window, sinks=sinks, return_lse=True)
    compare(out, lse, batch, q, "bfloat16")
    assert batch.cache.device_status() == m.MOE_OK


@pytest.mark.parametrize("new,lens,window,sinks", [([60], [3000], 2500, 300), ([40, 3], [2600, 700], 900, 5)])
def test_many_rows_with_sinks_whose_wait_runs_out(new, lens, window, sinks):
    """Chunks whose units several CTAs have parts of: no key tile comes, the
    status says so, and the joins of the calls that follow are right."""
    rng = np.random.default_rng(sum(lens))
    batch = Batch(rng, new, lens, 1, 16, 64, std=0.5)
    q = rounded(rng, (sum(new), 16, 64), "bfloat16")
    args = dict(q=tensor(q, "bfloat16"), **batch.dev, cu_q=batch.cu_dev, max_q_len=max(new), window=window, sinks=sinks)
    batch.cache.attend(**args, wait_timeout_ms=20, debug_flags=m.MOE_DEBUG_STALL_ATTENTION)
    assert batch.cache.device_status() == m.MOE_ERR_DEVICE_TIMEOUT
    for _ in range(2):
        out, lse = batch.cache.attend(**args, return_lse=True)
        assert batch.cache.device_status() == m.MOE_OK
        compare(out, lse, batch, q, "bfloat16", window=window, sinks=sinks)
