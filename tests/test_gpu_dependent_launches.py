"""Calls right behind the ones that write their inputs, over one set of buffers: each may start under the end of the launch
before it, and none may read before that launch's results are there."""
import pytest
import torch

import deepseek_sparse_mla_indexer_gb300 as nsa
import workloads as W
from deepseek_sparse_mla_indexer_gb300.step import SparseAttentionStep
from tests import _forms as F

pytestmark = pytest.mark.gpu
D = "cuda"

STEPS = {
    "128 heads, bf16": dict(seq_lens=[300, 2100, 77, 2500], H=128, kv_dtype=W.DT_BF16, seed=31),
    "16 heads, fp8": dict(seq_lens=[300, 2100, 77, 2500, 1, 640], H=16, kv_dtype=W.DT_E4M3, seed=32),
}
# the calls between the queries' way into the latent space and the attention that reads them
ORDERS = {
    "absorb, attention": ("metadata", "indexer", "topk_transform", "absorb", "attention"),
    "absorb, indexer, top-k, attention": ("metadata", "absorb", "indexer", "topk_transform", "attention"),
    "absorb, metadata, indexer, top-k, attention": ("absorb", "metadata", "indexer", "topk_transform", "attention"),
}


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("name", STEPS)
def test_absorb_sparse_attention_project(name, order, captured):
    wl = W.make_workload("chain", mode=W.MODE_DECODE, topk=2048, page_size=64, Hi=64, Di=128, idx_dtype=W.DT_E4M3, d_latent=512,
                         d_rope=64, q_dtype=W.DT_BF16, sm_scale=W.SM_SCALE_V32, **STEPS[name])
    step = SparseAttentionStep(wl, D)
    g = torch.Generator().manual_seed(wl.R)
    N, R, H = 24, step.R, step.H
    src, w = F.rand(g, N, R, H, 192).to(D), F.weight(g, H).to(D)
    q, back = torch.empty_like(src[0]), torch.empty((R, H, 128), dtype=F.BF, device=D)
    step.q_nope, step.q_rope = torch.empty((R, H, 512), dtype=F.BF, device=D), q[..., 128:]
    calls = dict(absorb=lambda: nsa.nsa_mla_absorb_q(q[..., :128], w, step.q_nope, step.status),
                 **{n: getattr(step, n) for n in ("metadata", "indexer", "topk_transform", "attention")})

    def run(i, wait, into):
        for f in (lambda: q.copy_(src[i]), *(calls[c] for c in ORDERS[order]),
                  lambda: nsa.nsa_mla_project_v(step.out, w, back, step.status),
                  lambda: [a.copy_(b) for a, b in zip(into, (step.out, step.lse, back))]):
            f()
            if wait:
                torch.cuda.synchronize()

    results = lambda: [tuple(torch.empty_like(t) for t in (step.out, step.lse, back)) for _ in range(N)]
    want, got = results(), results()
    for i in range(N):
        run(i, True, want[i])
    assert step.status_code() == 0
    assert not torch.equal(want[0][0], want[1][0])
    if captured:
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=s):
            for i in range(N):
                run(i, False, got[i])
        graph.replay()
        graph.replay()
    else:
        for i in range(N):
            run(i, False, got[i])
    torch.cuda.synchronize()
    assert step.status_code() == 0
    for i in range(N):
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b)


def _long_calls():
    """Calls with bounded waits: (results, call)."""
    g = torch.Generator().manual_seed(3)
    H, R = 4, 33
    empty = lambda *s: torch.empty(s, dtype=F.BF, device=D)
    q, w, cache = F.rand(g, R, H, 192).to(D), F.weight(g, H).to(D), F.rand(g, 300, 576).to(D)
    lat, back, out = F.rand(g, R, H, 512).to(D), empty(R, H, 128), empty(R, H, 128)
    q_lat, lse, ws = empty(R, H, 512), torch.empty((R, H), device=D), nsa.alloc_mla_prefill_workspace()
    kv, rope, cq, ck = F.rand(g, 300, H, 256).to(D), F.rand(g, 300, 64).to(D), F.starts([R]).to(D), F.starts([300]).to(D)

    def expand(m, H, w):
        slots = (torch.arange(m) % 300).to(torch.int32).to(D)
        kv_out, rope_out, ws = empty(m, H, 256), empty(m, 64), nsa.alloc_mla_expand_workspace(m)
        return (kv_out, rope_out), lambda st: nsa.nsa_mla_expand_kv(nsa.DT_BF16, cache, slots, w, kv_out, rope_out, ws, st)

    return {
        "absorb": ((q_lat,), lambda st: nsa.nsa_mla_absorb_q(q[..., :128], w, q_lat, st)),
        "project": ((back,), lambda st: nsa.nsa_mla_project_v(lat, w, back, st)),
        "expand": expand(100, H, w),
        "expand on pairs of CTAs": expand(2050, 27, F.weight(g, 27).to(D)),
        "prefill": ((out, lse), lambda st: nsa.nsa_mla_prefill(q[..., :128], q[..., 128:], kv[..., :128], rope, kv[..., 128:], cq, ck,
                                                               True, F.SCALE, out, lse, ws, st)),
    }


@pytest.mark.parametrize("name", ["absorb", "project", "expand", "expand on pairs of CTAs", "prefill"])
def test_behind_a_launch_that_lets_it_start_and_runs_on(name):
    results, call = _long_calls()[name]
    waited, status = (torch.zeros(1, dtype=torch.int32, device=D) for _ in range(2))
    call(status)
    want = [t.clone() for t in results]
    for t in results:
        t.fill_(7)
    nsa.nsa_check_bounded_wait(waited, 3_000_000_000)  # 1.5 s; the kernels' own waits give up after 2e9 clocks
    call(status)
    torch.cuda.synchronize()
    assert nsa.nsa_status_read(waited) == nsa.ERR_TIMEOUT and nsa.nsa_status_read(status) == 0
    for a, b in zip(results, want):
        assert torch.equal(a, b)
