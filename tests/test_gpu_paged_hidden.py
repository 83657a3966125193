"""nsa_paged_mla where some rows of a request may not see what others see, and where most
requests of a batch are empty.  Tolerances are those of test_gpu_paged_mla."""
import copy
import math
import time

import pytest
import torch

from tests._paged import Problem, slots_of
from tests.test_gpu_paged_mla import _check, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def nsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


def _spoil(p, b, pos, what):
    """A value that is not finite in the latent of a position of request b (fp8: by its scale or code)."""
    s = int(slots_of(p.table[b], pos + 1, p.ps)[pos])
    if p.kv_dt == 2:
        if math.isnan(what):
            p.kv[s, 130] = 0x7f
        else:
            p.kv[s, p.dl:p.dl + 16].view(torch.float32)[2] = what
    else:
        for d in (0, 77, 511):
            p.kv[s, d] = what


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("kv,n,H", [("bf16", 2, 8), ("bf16", 2, 16), ("bf16", 4, 16), ("bf16", 3, 20), ("bf16", 2, 128),
                                    ("fp8", 2, 8), ("fp8", 2, 16), ("fp8", 4, 16), ("fp8", 4, 32), ("fp8", 2, 128),
                                    ("f32", 2, 3)])
def test_what_is_not_finite_reaches_only_the_rows_that_see_it(nsa, kv, n, H, what):
    lens = [130, 1, 300, 128, 64]
    row_len = []
    for b, l in enumerate(lens):
        # the drafts of a verify step; in request 2 the first row is much shorter than the others
        row_len += [max(0, l - (n - 1 - i)) if b != 2 or i > 0 else 40 for i in range(n)]
    p = Problem(lens, n=n, H=H, kv=kv, seed=11, row_len=row_len)
    spoiled = {0: [129], 2: [60, 200], 4: [63]}
    for b, at in spoiled.items():
        for pos in at:
            _spoil(p, b, pos, what)
    seeing = torch.tensor([any(pos < row_len[b * n + i] for pos in spoiled.get(b, []))
                           for b in range(len(lens)) for i in range(n)])
    assert seeing.any() and not seeing.all()
    out, lse, code = _run(nsa, p)
    assert code == 0
    # the rows that see it are not finite somewhere (a score of -inf alone has no weight)
    if math.isnan(what):
        assert torch.isnan(out[seeing.cuda()]).any(-1).all() and torch.isnan(lse[seeing.cuda()]).all()
    # the others are as if the positions were not there
    rest = copy.copy(p)
    rest.row_len = torch.where(seeing, 0, p.row_len)
    out[seeing.cuda()], lse[seeing.cuda()] = 0, -math.inf
    _check(rest, out, lse)


@pytest.mark.parametrize("kv,H", [("fp8", 128), ("fp8", 64), ("bf16", 128)])
def test_a_few_requests_among_many_empty_ones(nsa, kv, H):
    """A padded batch: the rows of the empty requests become 0 / -inf, and no thread block waits for
    what another of its warps has long passed (a bounded wait that runs out takes a second)."""
    lens = [0] * 1200
    for b, l in ((7, 40000), (501, 129), (1190, 5000)):
        lens[b] = l
    p = Problem(lens, H=H, kv=kv, seed=12)
    p.q = p.q[:1].expand(p.R, -1, -1).contiguous()  # only three rows see a key
    _run(nsa, p)
    torch.cuda.synchronize()
    q = p.q.cuda()
    t0 = time.perf_counter()
    out, lse, code = _run(nsa, p, q=q)
    took = time.perf_counter() - t0
    assert code == 0 and took < 0.5, took
    empty = p.row_len.cuda() == 0
    assert not out[empty].any() and torch.isneginf(lse[empty]).all()
    keep = [7, 501, 1190]
    few = copy.copy(p)
    few.lens, few.B, few.R = [lens[b] for b in keep], 3, 3
    few.table, few.row_len, few.q = p.table[keep], p.row_len[keep], p.q[keep]
    _check(few, out[keep], lse[keep])
