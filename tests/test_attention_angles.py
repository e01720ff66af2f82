"""rope_frequencies: what it refuses, without a GPU."""
import pytest

import moe_lora_expert_gb300 as m


@pytest.mark.parametrize("bad", [
    dict(scaling={"factor": 4.0}),                                                # no kind
    dict(scaling={"kind": "yarn", "factor": 4.0}), dict(scaling={"kind": "llama3", "factor": 8.0}),   # no trained length
    dict(scaling={"kind": "yarn", "factor": 4.0, "original": 0}), dict(scaling={"kind": "llama3", "factor": 8.0, "original": -1}),
    dict(scaling={"kind": "yarn", "factor": 4.0, "original": 4096, "beta_fast": 0}),
    dict(scaling={"kind": "yarn", "factor": 4.0, "original": 4096, "beta_slow": -1}),
    dict(scaling={"kind": "llama3", "factor": 8.0, "original": 8192, "low": 4, "high": 4}),
    dict(scaling={"kind": "linear", "factor": float("inf")}), dict(scaling={"kind": "ntk", "factor": float("nan")}),
    dict(base=0.0), dict(base=-10000.0), dict(base=1.0, scaling={"kind": "yarn", "factor": 4.0, "original": 4096}),
])
def test_scaling_that_has_no_angles_is_refused(bad):
    with pytest.raises(ValueError):
        m.rope_frequencies(64, **bad)


def test_the_modules_example_runs_where_its_calls_do():
    """The table of the module's own example is made where the cache is."""
    import moe_lora_expert_gb300.attention as attention
    lines = [ln for ln in attention.__doc__.splitlines() if "rope_table(" in ln]
    assert len(lines) == 1 and 'device="cuda"' in lines[0]
