"""nsa_paged_mla's fp8 path through the clusters' scratch: rings that wrap many times, several pieces a share, calls
that run beside each other, and positions that only some rows see.  Tolerances are those of test_gpu_paged_mla."""
import math

import pytest
import torch

from tests._paged import SCALE, Problem, slots_of
from tests.test_gpu_paged_mla import _check, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def nsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("n,H", [(1, 40), (1, 64), (1, 128), (2, 96), (2, 128), (4, 128)])
def test_long_requests_give_equal_bits(nsa, n, H):
    p = Problem([60001, 777, 20000], n=n, H=H, kv="fp8", seed=51)
    first = _run(nsa, p)
    assert first[2] == 0
    _check(p, first[0], first[1])
    for _ in range(8):
        out, lse, code = _run(nsa, p)
        assert code == 0 and torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("n,H", [(1, 64), (1, 128), (4, 128)])
def test_captured_replayed_and_on_another_stream(nsa, n, H):
    p = Problem([9000, 3000, 0, 700], n=n, H=H, kv="fp8", seed=52)
    want = _run(nsa, p)
    assert want[2] == 0
    q, kv, t, rl = p.q.cuda(), p.kv.cuda(), p.table.cuda(), p.row_len.cuda()
    outs = [torch.zeros((p.R, p.H, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lses = [torch.zeros((p.R, p.H), device="cuda") for _ in range(2)]
    ws = [nsa.alloc_paged_mla_workspace(1, 2, p.R, n, p.H, p.max_len) for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda i: nsa.nsa_paged_mla(1, 2, q[..., :512], q[..., 512:], kv, 64, t, rl, n, p.max_len, SCALE, outs[i], lses[i], ws[i],
                                       status)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(0)
    torch.cuda.synchronize()
    for _ in range(5):  # replayed on one stream while the same call runs on another
        for x in (*outs, *lses):
            x.zero_()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            call(1)
        torch.cuda.synchronize()
        assert nsa.nsa_status_read(status) == 0
        for o, l in zip(outs, lses):
            assert torch.equal(o, want[0]) and torch.equal(l, want[1])


@pytest.mark.parametrize("kv,H", [("fp8", 8), ("fp8", 32), ("fp8", 128), ("bf16", 8), ("bf16", 64)])
def test_infinities_far_apart_in_a_split_request(nsa, kv, H):
    """Scores of -inf that one row of a long request sees and the other does not, in many shares."""
    L, short = 20011, 5000
    p = Problem([L], n=2, H=H, kv=kv, seed=53, row_len=[short, L])
    at = [4000, 5001, 9500, 9501, 15000, 20010]
    if kv == "fp8":
        p.q[..., 256:384] = -(p.q[..., 256:384].abs() + 0.125)
    else:
        p.q[..., 5] = p.q[..., 5].abs() + 0.125
    for pos in at:
        s = int(slots_of(p.table[0], pos + 1, p.ps)[pos])
        if kv == "fp8":
            p.kv[s, 256:384] = 0x38  # 1.0
            p.kv[s, 512:528].view(torch.float32)[2] = math.inf
        else:
            p.kv[s, 5] = -math.inf
    bad = slice(256, 384) if kv == "fp8" else slice(5, 6)
    ok = torch.ones(512, dtype=torch.bool)
    ok[bad] = False
    out, lse, code = _run(nsa, p)
    assert code == 0
    out, lse = out.double().cpu(), lse.double().cpu()
    for r in range(2):
        x, k = p.scores(r)
        want = torch.logsumexp(x, 1)
        fin = torch.where(torch.isfinite(k), k, torch.zeros_like(k))
        e = float((p.q[r].double().abs() @ fin.abs().T).max()) * SCALE * 577 * 2.0 ** -24
        pr = torch.exp(x - want[:, None])
        exp = pr @ fin[:, :512]
        assert ((lse[r] - want).abs() <= 2 * e + 2.0 ** -22 * (2 + want.abs())).all()
        assert torch.isnan(out[r][:, bad]).all() and torch.isfinite(out[r][:, ok]).all()  # both rows see position 4000
        tol = (2.0 ** -8 + 4 * e) * (pr @ fin[:, :512].abs()) + 2.0 ** -8 * exp.abs() + 2.0 ** -20
        assert ((out[r] - exp).abs() <= tol)[:, ok].all()
    # without the one that both see, only the longer row has them
    s = int(slots_of(p.table[0], 4001, p.ps)[4000])
    if kv == "fp8":
        p.kv[s, 512:528].view(torch.float32)[2] = 1.0
    else:
        p.kv[s, 5] = 0.25
    out, lse, code = _run(nsa, p)
    assert code == 0 and torch.isfinite(out[0]).all() and torch.isfinite(lse).all()
    assert torch.isnan(out[1][:, bad]).all() and torch.isfinite(out[1][:, ok.cuda()]).all()
