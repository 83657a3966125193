"""Calls of nsa_evict_compact that the binding refuses before it computes with their sizes (no GPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def nsa():
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("slots,page_size", [(0, 64), (64, 0), (64, -1), (65, 64)])
def test_compaction_of_no_whole_pages(nsa, slots, page_size):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError):
        nsa.nsa_evict_compact(i(1, 8), i(1), i(1), 16, i(1, 4), page_size, [torch.zeros(slots, 4)], None,
                              torch.empty(64, dtype=torch.uint8))
