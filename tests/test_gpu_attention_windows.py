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
