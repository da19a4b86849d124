"""Blocks of a cluster are scheduled together but need not have started together: shared memory
of another block is accessed after a barrier of the cluster alone. Read from the sources, as such
an access is undefined, not an error."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "linear_cross_entropy_gemm_gb300", "csrc")


def source(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def body(text, name):
    """The function's body: from the brace after its parameters to the one that closes it."""
    at = text.index("{", re.search(rf"\b{name}\([^;{{]*{{", text).start())
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i]
    raise AssertionError(name)


def test_the_sum_of_shares_waits_for_the_first_block():
    text = body(source("rms_norm.cu"), "share_sum_kernel")
    remote = text.index("map_shared_rank")
    assert text.count("cluster_arrive()") == text.count("cluster_wait()") == 1
    # All threads arrive at the start and wait before the first store to another block.
    assert text.index("if (blocks > 1) cluster_arrive();") < text.index("griddep_wait()")
    assert text.index("if (blocks > 1) cluster_wait();") < text.index("if (warp == 0)") < remote
