"""Rows that nsa_evict_compact cannot follow (a page outside the cache, a position past the length, one out of
order): the row stays, and its total with it.  Bytes and totals are compared for equality."""
import numpy as np
import pytest
import torch

from tests._paged import page_table, slots_of
from tests.test_gpu_evict import _arrays, _compact, _expect, _same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def nsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


LENS, PS = [100, 100, 100], 16


def _case(seed):
    g = torch.Generator().manual_seed(seed)
    table, pages = page_table(LENS, PS, g)
    arrays, total = _arrays(pages * PS, g, "serving"), torch.rand((3, 100), generator=g) + 1
    return table, pages, arrays, total, np.tile(np.arange(50, dtype=np.int32) * 2, (3, 1))


def _expect_but(arrays, total, table, keep, stay):
    """The moved arrays and totals, with rows `stay` = [(request, positions)] as they were."""
    safe = keep.copy()
    for b, at in stay:
        safe[b, at] = at  # any valid source: put back below
    want, wt = _expect(arrays, total, table, PS, safe, [50] * 3, LENS)
    for b, at in stay:
        s = slots_of(table[b], 100, PS)
        for w, a in zip(want, arrays):
            w[s[at]] = a[s[at]]
        wt[b, at] = total[b, at]
    return want, wt


def test_a_source_page_outside_the_cache(nsa):
    table, pages, arrays, total, keep = _case(41)
    bad = table.clone()
    bad[0, 5] = pages  # positions 80 .. 95 of request 0: sources of rows 40 .. 47
    got, gt, code = _compact(nsa, arrays, total, bad, PS, keep, [50] * 3, LENS, 100)
    want, wt = _expect_but(arrays, total, table, keep, [(0, np.arange(40, 48))])
    assert code == nsa.ERR_BOUNDS
    assert _same(got, want)
    assert torch.equal(gt, wt)


def test_a_destination_page_outside_the_cache(nsa):
    table, pages, arrays, total, keep = _case(42)
    bad = table.clone()
    bad[1, 1] = -1  # positions 16 .. 31 of request 1: sources of rows 8 .. 15, destinations of rows 16 .. 31
    got, gt, code = _compact(nsa, arrays, total, bad, PS, keep, [50] * 3, LENS, 100)
    want, wt = _expect_but(arrays, total, table, keep, [(1, np.arange(8, 32))])
    assert code == nsa.ERR_BOUNDS
    assert _same(got, want)
    assert torch.equal(gt, wt)


def test_totals_alone_need_no_pages(nsa):
    table, pages, _, total, keep = _case(43)
    got, gt, code = _compact(nsa, [], total, torch.full_like(table, -1), PS, keep, [50] * 3, LENS, 100)
    assert code == 0
    assert torch.equal(gt, _expect([], total, table, PS, keep, [50] * 3, LENS)[1])


def test_a_position_past_the_length_and_one_out_of_order(nsa):
    table, pages, arrays, total, keep = _case(44)
    keep[0, 49], keep[1, 10] = 100, 18
    got, gt, code = _compact(nsa, arrays, total, table, PS, keep, [50] * 3, LENS, 100)
    want, wt = _expect_but(arrays, total, table, keep, [(0, np.array([49])), (1, np.array([10]))])
    assert code == nsa.ERR_BOUNDS
    assert _same(got, want)
    assert torch.equal(gt, wt)
