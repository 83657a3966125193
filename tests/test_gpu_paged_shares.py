"""nsa_paged_mla and nsa_mla_key_weights where a thread block's share of the work holds many tiles
and several requests, so that shares begin and end inside, between and at the edges of requests.
Tolerances are those of test_gpu_paged_mla."""
import pytest
import torch

from tests._paged import Problem
from tests.test_gpu_paged_mla import _check, _check_weights, _run, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def nsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


CASES = {
    "mixed": [(i * 397) % 1700 if i % 9 else 0 for i in range(150)],
    "tiny among long": [1 if i % 3 else 3000 - 17 * i for i in range(70)],
    "one tile each": [1 + (i * 31) % 128 for i in range(700)],
    "more than threads": [(i * 37) % 300 for i in range(1000)],
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("kv,n,H", [("bf16", 1, 16), ("bf16", 2, 16), ("bf16", 1, 128), ("bf16", 1, 192), ("fp8", 1, 16),
                                    ("fp8", 1, 64), ("fp8", 1, 128), ("fp8", 4, 64)])
def test_attention(nsa, name, kv, n, H):
    lens = CASES[name] if n * H <= 32 else CASES[name][:: 4]
    p = Problem(lens, n=n, H=H, kv=kv, seed=21)
    out, lse, code = _run(nsa, p)
    assert code == 0
    _check(p, out, lse)


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("kv,n,H", [("bf16", 1, 16), ("bf16", 2, 96), ("fp8", 1, 16), ("fp8", 1, 80), ("fp8", 3, 64)])
def test_weights(nsa, name, kv, n, H):
    lens = CASES[name] if n * H <= 32 else CASES[name][:: 4]
    p = Problem(lens, n=n, H=H, kv=kv, seed=22)
    lse = p.attention()[1].float()
    total = torch.zeros((p.B, p.max_len), device="cuda")
    assert _weights(nsa, p, lse, total) == 0
    _check_weights(p, lse, total)
