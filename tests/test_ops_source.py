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
