"""Rules that the attention half's CUDA sources keep, checked on their text:
faults that a run may or may not show."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "moe_lora_expert_gb300", "csrc")


def code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, head):
    """The braces' content that follows ``head``."""
    at = text.index("{", text.index(head))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at + 1:i]
    raise AssertionError(head)


def test_warps_name_the_lanes_they_wait_for():
    """__activemask() names the lanes that happen to be there, not those that
    will come: nothing that lanes share may be ordered by it."""
    for name in os.listdir(CSRC):
        assert "__activemask" not in code(name), name


def test_a_shared_walk_is_stepped_between_barriers():
    """All lanes are done with a piece before any reads the walk, and have read
    it before any writes the next piece."""
    steps = re.findall(r"__syncwarp\(lanes\)|Walk w = \*at|\*at = w", body(code("prefill_attention.cu"), "bool walk_next("))
    assert steps == ["__syncwarp(lanes)", "Walk w = *at", "__syncwarp(lanes)", "*at = w", "__syncwarp(lanes)"]


def test_tmem_is_accessed_by_whole_warps():
    """tcgen05's allocation and loads are one instruction of all lanes; what
    comes before them (rows that are written, an arrival by one lane) is not."""
    text = code("prefill_attention.cu")
    summed = body(text, "auto summed = ")
    assert 0 <= summed.find("__syncwarp()") < summed.index("tmem_ld32(")
    assert re.search(r"__syncwarp\(\);\s*tmem_alloc\(", text)
    assert re.search(r"mbar_arrive\(&s\.p_full\[i\]\[h\]\);\s*__syncwarp\(\);", text)
