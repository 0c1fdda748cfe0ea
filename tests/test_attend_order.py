"""The order of the tensor-memory accesses in the attention's source: loads and stores of tensor memory (tcgen05.ld, .st)
run asynchronously and come in no order among themselves but by a wait, and a wrong order mostly gives the right result
all the same, so that no run of the kernel shows it."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "gated_deltanet_verify_gb300", "csrc", "attend.cu")


@pytest.fixture(scope="module")
def steps():
    """(line, name) of the calls that matter, in the kernel's text."""
    text = open(SOURCE).read()
    text = text[text.index("attend_tc_kernel("):text.index("cudaError_t launch(")]
    text = re.sub(r"//[^\n]*", "", text)
    names = r"\b(tmem_ld32|tmem_st16|tmem_st32|wait_ld|wait_st|rows_sync|fence_before|fence_after)\("
    return [(text.count("\n", 0, m.start()), m.group(1)) for m in re.finditer(names, text)]


def test_no_store_between_a_load_and_its_wait(steps):
    pending = None
    for at, name in steps:
        if name.startswith("tmem_ld"):
            pending = at
        elif name == "wait_ld":
            pending = None
        elif name.startswith("tmem_st"):
            assert pending is None, f"a store {at - pending} lines behind a load that nothing has waited for"


def test_the_other_threads_store_is_fenced(steps):
    """Two threads share a row's scores, and the weights of one go over scores of the other: from a load's wait to the barrier
    between the two there is a fence, and another one from the barrier to the store."""
    names = [name for _, name in steps]
    first = names.index("tmem_ld32")
    between = names[first:names.index("rows_sync", first)]
    assert "fence_before" in between[between.index("wait_ld"):]
    behind = names[names.index("rows_sync", first):]
    assert "fence_after" in behind[:behind.index("tmem_st32")]
