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


def test_the_sampler_waits_for_all_blocks():
    text = source("sample.cu")
    kernel, run, find = (body(text, name) for name in ("sample_kernel", "run", "find_top"))
    assert text.count("cluster_arrive()") == text.count("cluster_wait()") == 1
    arrive = kernel.index("if (a.cluster > 1) cluster_arrive();")
    assert arrive < kernel.index("griddep_wait()") < kernel.index("r.run(row)") and "return" not in kernel
    # Nothing before find_top takes a barrier or another block's memory, or leaves.
    before = run[:run.index("find_top(")]
    assert not re.search(r"of_block|sync\(\)|reduce<|gather|return", before.replace("__syncthreads()", ""))
    # In it the wait, by all threads, precedes the first store.
    wait = find.index("if (a.cluster > 1) cluster_wait();")
    assert wait < find.index("of_block(") and find[:wait].count("{") == find[:wait].count("}") + 1
    assert "return" not in find[:wait]


def test_other_blocks_memory_is_taken_after_a_barrier():
    """Of the kernels that map another block's memory: the first mapping follows a cluster barrier."""
    for name in ("block_small.cu", "pair_engine.cuh", "gemm_engine.cuh", "rms_norm.cu"):
        for kernel in re.split(r"__global__", source(name))[1:]:
            for mapped in list(re.finditer(r"mapa_shared\(|map_shared_rank\(", kernel))[:1]:
                assert re.search(r"cluster_sync\(\)|cluster_wait\(\)", kernel[:mapped.start()]), name
