"""Host check of how the tensor-core chunk attention (csrc/tq3_chunk_mma.cu) ends, on its source: no correct
call makes one of its waits run out, so the GPU tests only run the path on which none does.

Whichever role's wait ran out, products may be in flight: the warps that issued some have to wait for them
before the tensor memory is freed, and no role may go on to the next segment, whose queries are written where
those products read.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_quantization_b200", "csrc")


def body(source, head):
    """The text between the braces of the function whose definition starts with `head`."""
    at = source.index("{", source.index(")", source.index(head)))
    depth = 0
    for i in range(at, len(source)):
        depth += {"{": 1, "}": -1}.get(source[i], 0)
        if depth == 0:
            return source[at:i + 1]
    raise AssertionError(head)


@pytest.fixture(scope="module")
def source():
    with open(os.path.join(CSRC, "tq3_chunk_mma.cu")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_products_are_waited_for_before_tensor_memory_is_freed(source):
    kernel = body(source, "chunk_kernel(const")
    commit, wait = kernel.index("mma_commit(&sh.drain"), kernel.index("mbar_wait_bounded(&sh.drain")
    meet, free = kernel.rindex("__syncthreads()"), kernel.index("tmem_dealloc")
    assert commit < wait < meet < free
    # the condition that guards the drain: whoever issued products, whether or not a wait ran out
    condition = kernel[kernel.rindex("if (", 0, commit):commit]
    assert "issued" in condition and "dead" not in condition
    assert "elect_one()" in condition  # a commit covers the products of the thread that makes it
    role = body(source, "bool issue_role(")
    assert "n_s += mine" in role and role.rstrip("} \n").endswith("return n_s > 0;")


@pytest.mark.parametrize("role", ["softmax_role", "decode_role", "issue_role"])
def test_all_roles_leave_when_one_wait_has_run_out(source, role):
    # every role enters its next segment through next_segment alone, and tells it of its own waits
    text = body(source, role + "(const")
    assert "more = next_segment<kWide>(a, sh, dead)" in text and "while (!w.done())" not in text
    between = body(source, "bool next_segment(")
    told, meet, seen = between.index("sh.dead = 1"), between.index("__syncthreads()"), between.index("sh.dead != 0")
    assert told < meet < seen < between.index("w.next(a)")
    assert "return !over && !w.done();" in between
