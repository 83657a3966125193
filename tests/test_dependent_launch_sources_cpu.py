"""Kernels that are launched while the launch before them still runs (programmatic dependent launch): what a call before
them on the stream wrote is there only behind griddepcontrol.wait, which no test of results shows reliably."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deepseek_sparse_mla_indexer_gb300", "csrc")


def _body(name, kernel):
    """The code of a kernel, without comments."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    at = re.search(kernel + r"\([^{]*\)\s*\{", code)
    depth, i = 1, at.end()
    while depth:
        depth += {"{": 1, "}": -1}.get(code[i], 0)
        i += 1
    return code[at.end():i]


@pytest.mark.parametrize("array", ["q_nope", "q_rope", "kv", "indices"])
def test_sparse_attention_reads_behind_its_wait(array):
    workers = _body("sparse_mla_tc.cu", "sparse_mla_tc_kernel").split("} else {", 1)[1]  # warp 1 reads no global memory
    assert workers.index("pdl_wait()") < workers.index("p." + array)
