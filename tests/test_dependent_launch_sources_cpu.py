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


@pytest.mark.parametrize("name,kernel", [("mla_project.cu", "head_product_kernel"), ("mla_project.cu", "pair_product_kernel"),
                                         ("mla_prefill.cu", "mla_prefill_kernel")])
def test_bounded_waits_begin_behind_the_launch_before(name, kernel):
    # every warp passes the wait (it stands outside any branch) before its first wait that may run out
    body = _body(name, kernel)
    at = body.index("pdl_wait()")
    assert body[:at].count("{") == body[:at].count("}") and "mla_wait(" not in body[:at]
