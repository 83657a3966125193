"""Row widths that nsa_paged_mla and nsa_mla_key_weights refuse, alike and before any launch (no GPU)."""
import pytest

from tests.test_paged_abi_cpu import _paged


@pytest.fixture(scope="module")
def nsa():
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("dl,dr", [(1688, 64), (1752, 0), (1, 1751), (8192, 64), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_rows_wider_than_the_kernels_hold(nsa, weights, dl, dr):
    assert _paged(nsa, weights, dl=dl, dr=dr) == nsa.ERR_UNSUPPORTED
    assert _paged(nsa, weights, qdt=0, kdt=0, dl=dl, dr=dr) == nsa.ERR_UNSUPPORTED


def test_no_workspace_for_what_is_refused(nsa):
    assert nsa.nsa_paged_mla_workspace_bytes(1, 1, 2 ** 20, 2 ** 20, 2, 100) == 0     # 2^21 columns a request
    assert nsa.nsa_paged_mla_workspace_bytes(1, 1, 1, 1, 65536, 100) == 0
    assert nsa.nsa_paged_mla_workspace_bytes(1, 2, 1, 1, 16, 2 ** 30 + 1) == 0
    assert nsa.nsa_paged_mla_workspace_bytes(1, 1, 2 ** 26, 1, 128, 100) == 0         # 2^33 query heads
