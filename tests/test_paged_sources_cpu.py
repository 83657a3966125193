"""What the library's sources may not hold: the library is loaded by single- and multi-GPU programs
alike, and a call cannot see whether the memory that it is given is this GPU's own."""
import glob
import os

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deepseek_sparse_mla_indexer_gb300", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*")))


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.basename(s) for s in SOURCES])
def test_no_load_writes_into_several_thread_blocks(path):
    with open(path, encoding="utf-8") as f:
        assert "multicast" not in f.read().lower()


def test_there_are_sources_to_look_at():
    assert any(s.endswith("paged_mla_tc.cu") for s in SOURCES)
