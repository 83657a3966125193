"""nsa_paged_mla's workspace: one allocated for the largest shape of a serving loop serves every smaller one."""
import random

import pytest
import torch

from tests._paged import Problem
from tests.test_gpu_paged_mla import _check, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def nsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("kv,dt", [("bf16", 1), ("fp8", 2)])
def test_a_verify_workspace_serves_decode(nsa, kv, dt):
    ws = nsa.alloc_paged_mla_workspace(1, dt, 32 * 4, 4, 128, 32768)
    for n, H in ((1, 128), (1, 64), (2, 128), (1, 16), (3, 100)):
        p = Problem([5000, 0, 129, 700], n=n, H=H, kv=kv, seed=n * 1000 + H)
        out, lse, code = _run(nsa, p, ws=ws)
        assert code == 0
        _check(p, out, lse)


@pytest.mark.parametrize("dt", [1, 2])
def test_no_larger_shape_needs_less(nsa, dt):
    rng = random.Random(9)
    log = lambda lo, hi: round(lo * (hi / lo) ** rng.random())
    for _ in range(4000):
        B, n, H, ml = log(1, 300), log(1, 8), log(1, 200), log(1, 200000)
        small = (B * n, n, H, ml)
        more = [x + rng.choice([0, 0, 1, x, 3 * x]) for x in (B, n, H, ml)]
        large = (more[0] * more[1], more[1], more[2], more[3])
        assert nsa.nsa_paged_mla_workspace_bytes(1, dt, *small) <= nsa.nsa_paged_mla_workspace_bytes(1, dt, *large), (small, large)
