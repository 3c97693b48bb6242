"""Rules of the operators' kernels that no run can show to be kept: which block starts first, and what a compiler may
move, differ from run to run.  Read from the sources (no GPU needed)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def source(name):
    with open(os.path.join(ROOT, "video_dit_sparse_gb300", "csrc", name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_no_block_has_a_duty_by_its_number():
    """A kernel that takes over blocks which have not started may run any unit in any block, and block 0 may never
    start: a block's number only says which unit it begins with."""
    text = source("sa_masked.cu")
    kernel = text[text.index("__device__ __forceinline__ void share_out"):text.index("sa_masked_join_kernel")]
    assert "request_block" in kernel
    assert re.findall(r"[^\n]*blockIdx[^\n]*", kernel) == ["    int64_t g = blockIdx.x;"]


def test_results_of_a_running_kernel_are_read_by_plain_loads():
    """A kernel launched beside the one ahead of it reads that one's results after its wait.  A read-only load promises
    that nothing writes the data while the kernel runs, so the compiler may move it ahead of the wait."""
    text = source("sa_masked.cu") + source("sa_cache.cu")
    assert text.count("wait_for_earlier_kernel();") == 4
    loads = re.findall(r"__ldg\((?:[^()]|\((?:[^()]|\([^()]*\))*\))*\)", text)
    assert len(loads) > 5  # (the pattern finds them)
    assert [x for x in loads if re.search(r"\bkept\b|part_o|part_lse|part_first", x)] == []
    quads = text[text.index("sa_masked_join_quads_kernel"):text.index("void masked_plan")]
    assert "__ldg" not in quads  # (its rows are read through a pointer of their own)
