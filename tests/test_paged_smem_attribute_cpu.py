"""How much shared memory a kernel may use is set once, to the most that any call needs.  Set from a call's own
size, it is lowered by another host thread between that thread's setting and its launch, which is then refused."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deepseek_sparse_mla_indexer_gb300", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


@pytest.mark.parametrize("name", ["paged_mla.cu", "paged_mla_tc.cu", "mla_key_weights.cu", "mla_key_weights_tc.cu", "evict.cu"])
def test_the_limit_does_not_follow_the_call(name):
    assert "cudaFuncSetAttribute" not in _code(name)  # max_dynamic_smem asks once per device
    assert "max_dynamic_smem" in _code(name)
