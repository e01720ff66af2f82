"""What may be given as the axes of a rotation's pairs, on the CPU."""
import numpy as np
import pytest

import moe_lora_expert_gb300 as m
from test_attention_devices import fake  # noqa: F401
from test_rope_axes_host import AXES_CALLS, calls, run  # noqa: F401


@pytest.mark.parametrize("name", AXES_CALLS)
@pytest.mark.parametrize("axes", [32, np.int64(32), np.zeros(4, np.int64), [0.5] * 32, [0] * 31 + [256], [-1] + [0] * 31])
def test_axes_that_name_no_axis_for_each_pair(calls, name, axes):  # noqa: F811
    """A number is not so many pairs of the first axis, nor an array's memory its values."""
    with pytest.raises(ValueError):
        run(name, axes=axes)
    assert not calls[0]


@pytest.mark.parametrize("name", AXES_CALLS)
@pytest.mark.parametrize("kind", [list, tuple, bytearray, lambda x: np.array(list(x)), lambda x: np.array(list(x), np.uint8)])
def test_axes_of_any_sequence(calls, name, kind):  # noqa: F811
    want = m.rope_axes([10, 11, 11], turns=True)
    run(name, axes=kind(want))
    assert bytes(m.RopeAxes.from_buffer_copy(calls[0][0][3]).axis_of_pair[:32]) == want
