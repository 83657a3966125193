"""The paged operators on a cache whose rows lie past the reach of 32-bit byte offsets: the same
problem at the front of a small cache gives the same bits."""
import pytest
import torch

from tests._paged import SCALE, Problem, slots_of
from tests.test_gpu_paged_mla import _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def nsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


def _far(p):
    """p's cache behind 2^32 bytes of a larger one, and the page table that finds it."""
    row = p.kv.shape[1] * p.kv.element_size()
    skip = -(-(2 ** 32 + 2 ** 20) // (row * p.ps))  # pages
    kv = torch.empty(((skip + p.pages) * p.ps, p.kv.shape[1]), dtype=p.kv.dtype, device="cuda")
    kv[skip * p.ps:] = p.kv.cuda()
    return kv, (p.table + skip).cuda(), skip


@pytest.mark.parametrize("kv,n,H,ps", [("bf16", 1, 16, 64), ("bf16", 1, 128, 64), ("fp8", 1, 16, 64), ("fp8", 4, 16, 16),
                                       ("fp8", 2, 128, 64), ("fp8", 1, 128, 64), ("bf16", 1, 4, 7)])
def test_attention_weights_and_compaction(nsa, kv, n, H, ps):
    lens = [700, 0, 129, 1500]
    p = Problem(lens, n=n, H=H, kv=kv, ps=ps, seed=31)
    out, lse, code = _run(nsa, p)
    assert code == 0
    far, table, skip = _far(p)
    q, rl = p.q.cuda(), p.row_len.cuda()
    ws = nsa.alloc_paged_mla_workspace(p.q_dt, p.kv_dt, p.R, n, H, p.max_len)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    nsa.nsa_paged_mla(p.q_dt, p.kv_dt, q[..., :512], q[..., 512:], far, ps, table, rl, n, p.max_len, SCALE, out2, lse2,
                      ws, status)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)

    totals = []
    for cache, t in ((p.kv.cuda(), p.table.cuda()), (far, table)):
        total = torch.zeros((p.B, p.max_len), device="cuda")
        nsa.nsa_mla_key_weights(p.q_dt, p.kv_dt, q[..., :512], q[..., 512:], cache, ps, t, rl, n, p.max_len, SCALE, lse,
                                total, status)
        totals.append(total)
    assert torch.equal(*totals)

    old = torch.tensor(lens, dtype=torch.int32, device="cuda")
    keep = torch.empty((p.B, 200), dtype=torch.int32, device="cuda")
    new = torch.empty(p.B, dtype=torch.int32, device="cuda")
    nsa.nsa_evict_select(totals[0], old, p.max_len, 4, 16, 200, keep, new, status)
    nsa.nsa_evict_compact(keep, new, old, p.max_len, table, ps, [far], totals[1], nsa.alloc_evict_workspace(p.B, p.max_len),
                          status)
    assert nsa.nsa_status_read(status) == 0
    for b in range(p.B):
        got = far[(slots_of(p.table[b], int(new[b]), ps) + skip * ps).cuda()]
        kept = keep[b, :int(new[b])].cpu().long()
        want = p.kv[slots_of(p.table[b], lens[b], ps)[kept]]
        assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))
