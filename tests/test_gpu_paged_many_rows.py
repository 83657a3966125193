"""nsa_paged_mla and nsa_mla_key_weights with many rows a request: prompt chunks and windows of queries, ragged ones
padded with rows of length 0.  Tolerances are those of test_gpu_paged_mla."""
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


def _problem(kv, n, H, ps, q_lens, ctx):
    """Request b: its last q_lens[b] tokens are rows of their own lengths, in front of rows of length 0."""
    row_len = []
    for q, c in zip(q_lens, ctx):
        row_len += [0] * (n - q) + [c - (q - 1 - i) for i in range(q)]
    return Problem(ctx, n=n, H=H, kv=kv, ps=ps, seed=n + H, row_len=row_len)


CASES = [(37, 3, 64, [37, 1, 20], [300, 150, 37]), (70, 16, 64, [70, 64], [500, 64]), (9, 128, 64, [9, 0, 4], [257, 40, 640]),
         (128, 16, 16, [128], [128]), (13, 5, 7, [13, 2], [40, 33]), (5, 128, 32, [5], [1200]), (2, 96, 64, [2, 1], [300, 700])]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("n,H,ps,q_lens,ctx", CASES)
def test_attention(nsa, kv, n, H, ps, q_lens, ctx):
    p = _problem(kv, n, H, ps, q_lens, ctx)
    out, lse, code = _run(nsa, p)
    assert code == 0
    _check(p, out, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("n,H,ps,q_lens,ctx", CASES)
def test_weights(nsa, kv, n, H, ps, q_lens, ctx):
    p = _problem(kv, n, H, ps, q_lens, ctx)
    lse = p.attention()[1].float()
    total = torch.zeros((p.B, p.max_len), device="cuda")
    assert _weights(nsa, p, lse, total) == 0
    _check_weights(p, lse, total)
