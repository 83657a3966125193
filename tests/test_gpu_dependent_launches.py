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
