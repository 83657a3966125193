"""Calls of latent attention's two forms at their edges: offsets past 32 bits, results at 16-byte addresses, a thousand
requests, requests that overlap, rows of one stride, queries that are not finite."""
import pytest
import torch

import deepseek_sparse_mla_indexer_gb300 as nsa
from tests import _forms as F

pytestmark = pytest.mark.gpu
D = "cuda"


def _prefill(q, kv, k_rope, cu_q, cu_k, causal, out=None, lse=None, status=None):
    out = torch.full((q.shape[0], q.shape[1], 128), 7.0, dtype=F.BF, device=D) if out is None else out
    lse = torch.full(q.shape[:2], 7.0, device=D) if lse is None else lse
    nsa.nsa_mla_prefill(q[..., :128], q[..., 128:], kv[..., :128], k_rope, kv[..., 128:], cu_q.to(D), cu_k.to(D), causal, F.SCALE,
                        out, lse, nsa.alloc_mla_prefill_workspace(), status)
    return out, lse


def test_keys_behind_two_to_the_31_values():
    H, far, nk, nq = 128, 70000, 300, 3  # 70000 x 128 x 256 = 2.3e9
    g = torch.Generator().manual_seed(1)
    kv, k_rope = torch.zeros((far + nk, H, 256), dtype=F.BF, device=D), torch.zeros((far + nk, 64), dtype=F.BF, device=D)
    q, tail, rope = F.rand(g, nq, H, 192), F.rand(g, nk, H, 256), F.rand(g, nk, 64)
    kv[far:], k_rope[far:] = tail.to(D), rope.to(D)
    cu_q, cu_k = torch.tensor([0, 0, nq], dtype=torch.int32), torch.tensor([0, far, far + nk], dtype=torch.int32)
    out, lse = _prefill(q.to(D), kv, k_rope, cu_q, cu_k, True)
    o, l, to, tl = F.attention(q, tail, rope, [nq], [nk], True)
    F.close(lse, l, tl, "lse")
    F.close(out, o, to, "out")


def test_queries_behind_two_to_the_31_values():
    H, far, n = 128, 131300, 5  # 131300 x 128 x 128 = 2.15e9
    g = torch.Generator().manual_seed(2)
    q = torch.zeros((far + n, H, 192), dtype=F.BF, device=D)
    last, kv, rope = F.rand(g, n, H, 192), F.rand(g, n, H, 256), F.rand(g, n, 64)
    q[far:] = last.to(D)
    cu_q, cu_k = torch.tensor([0, far, far + n], dtype=torch.int32), torch.tensor([0, 0, n], dtype=torch.int32)
    out, lse = _prefill(q, kv.to(D), rope.to(D), cu_q, cu_k, True)
    o, l, to, tl = F.attention(last, kv, rope, [n], [n], True)
    F.close(lse[far:], l, tl, "lse")
    F.close(out[far:], o, to, "out")
    for i in range(0, far, 8192):  # rows without a key
        assert not out[i:min(far, i + 8192)].any() and (lse[i:min(far, i + 8192)] == -torch.inf).all()


def test_expanded_rows_behind_two_to_the_31_values():
    H, m = 128, 65700  # 65700 x 128 x 256 = 2.15e9
    g = torch.Generator().manual_seed(3)
    cache, w = F.rand(g, 100, 576), F.weight(g, H)
    slots = torch.arange(m, dtype=torch.int32) % 100
    out = torch.empty((m, H, 256), dtype=F.BF, device=D)
    rope = torch.empty((m, 64), dtype=F.BF, device=D)
    nsa.nsa_mla_expand_kv(nsa.DT_BF16, cache.to(D), slots.to(D), w.to(D), out, rope, nsa.alloc_mla_expand_workspace(m))
    want = cache[:, :512].double() @ w.double().T
    F.close(out[:100].view(100, -1), want, F.product_tol(cache[:, :512].double(), w.double(), want), "first rows")
    for i in range(0, m, 100):
        n = min(100, m - i)
        assert torch.equal(out[i:i + n], out[:n]) and torch.equal(rope[i:i + n], rope[:n])


@pytest.mark.parametrize("H,nq,nk", [(200, [40], [300]), (2, [6], [3000])])
def test_results_at_16_byte_addresses(H, nq, nk):
    g = torch.Generator().manual_seed(4)
    q, kv, rope = F.rand(g, sum(nq), H, 192).to(D), F.rand(g, sum(nk), H, 256).to(D), F.rand(g, sum(nk), 64).to(D)
    want = _prefill(q, kv, rope, F.starts(nq), F.starts(nk), True)
    n = sum(nq) * H * 128
    buf = torch.full((n + 16,), 7.0, dtype=F.BF, device=D)
    out = buf[8:8 + n].view(sum(nq), H, 128)
    assert out.data_ptr() % 32 == 16
    got = _prefill(q, kv, rope, F.starts(nq), F.starts(nk), True, out=out)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (buf[:8] == 7).all() and (buf[8 + n:] == 7).all()


@pytest.mark.parametrize("causal", [True, False])
def test_a_thousand_requests(causal):
    g = torch.Generator().manual_seed(5)
    nq = [int(x) for x in torch.randint(0, 4, (1000,), generator=g)]
    nk = [a + int(x) for a, x in zip(nq, torch.randint(0, 9, (1000,), generator=g))]
    nq[500], nk[500] = 300, 700
    q, kv, rope = F.rand(g, sum(nq), 1, 192), F.rand(g, sum(nk), 1, 256), F.rand(g, sum(nk), 64)
    out, lse = _prefill(q.to(D), kv.to(D), rope.to(D), F.starts(nq), F.starts(nk), causal)
    o, l, to, tl = F.attention(q, kv, rope, nq, nk, causal)
    F.close(lse, l, tl, "lse")
    F.close(out, o, to, "out")


def test_overlapping_requests_are_reported():
    # each in order by itself, together more blocks of queries than so many rows have
    g = torch.Generator().manual_seed(6)
    q, kv, rope = F.rand(g, 600, 1, 192).to(D), F.rand(g, 600, 1, 256).to(D), F.rand(g, 600, 64).to(D)
    cu = torch.tensor([0, 600, 0, 600, 0, 600, 0, 600], dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device=D)
    _prefill(q, kv, rope, cu, cu, True, status=status)
    assert nsa.nsa_status_read(status) == nsa.ERR_BOUNDS


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,nq,nk", [
    (2, [300, 5, 0, 1, 260], [9000, 700, 40, 5, 3100]),   # other numbers of parts, and none, in one call
    (1, [7, 1, 9], [6000, 0, 300]),                        # a request without a key beside a long one
    (3, [2] * 33 + [40], [900] * 33 + [5000]),             # more requests than a warp has lanes
    (16, [500], [2700]),
])
def test_parts_of_requests_of_other_lengths(H, nq, nk, causal):
    g = torch.Generator().manual_seed(9)
    q, kv, rope = F.rand(g, sum(nq), H, 192), F.rand(g, sum(nk), H, 256), F.rand(g, sum(nk), 64)
    ws = nsa.alloc_mla_prefill_workspace()
    ws.fill_(255)  # (NaN in every part that is not written)
    out, lse = torch.full((sum(nq), H, 128), 7.0, dtype=F.BF, device=D), torch.full((sum(nq), H), 7.0, device=D)
    status = torch.zeros(1, dtype=torch.int32, device=D)
    nsa.nsa_mla_prefill(q.to(D)[..., :128], q.to(D)[..., 128:], kv.to(D)[..., :128], rope.to(D), kv.to(D)[..., 128:], F.starts(nq).to(D),
                        F.starts(nk).to(D), causal, F.SCALE, out, lse, ws, status)
    assert nsa.nsa_status_read(status) == 0
    o, l, to, tl = F.attention(q, kv, rope, nq, nk, causal)
    F.close(lse, l, tl, "lse")
    F.close(out, o, to, "out")


@pytest.mark.parametrize("causal", [True, False])
def test_a_request_left_out_of_long_ones(causal):
    # few items over long rows, whose keys a good call cuts into parts
    g = torch.Generator().manual_seed(8)
    nq, nk = [40, 30, 50], [5000, 3000, 4000]
    q, kv, rope = F.rand(g, 120, 1, 192), F.rand(g, 12000, 1, 256), F.rand(g, 12000, 64)
    o, l, to, tl = F.attention(q, kv, rope, nq, nk, causal)
    for bad, left in ([0, 5000, 8000, 12001], slice(70, 120)), ([-1, 5000, 8000, 12000], slice(0, 40)), \
            ([0, 5000, 4999, 12000], slice(40, 120)):
        out, lse = torch.full((120, 1, 128), 7.0, dtype=F.BF, device=D), torch.full((120, 1), 7.0, device=D)
        status = torch.zeros(1, dtype=torch.int32, device=D)
        ws = nsa.alloc_mla_prefill_workspace()
        nsa.nsa_mla_prefill(q.to(D)[..., :128], q.to(D)[..., 128:], kv.to(D)[..., :128], rope.to(D), kv.to(D)[..., 128:],
                            F.starts(nq).to(D), torch.tensor(bad, dtype=torch.int32, device=D), causal, F.SCALE, out, lse, ws, status)
        assert nsa.nsa_status_read(status) == nsa.ERR_BOUNDS
        keep = torch.ones(120, dtype=torch.bool)
        keep[left] = False
        if bad[2] == 4999:  # (request 2 is in order, but has other keys)
            assert (out[40:70] == 7).all() and (lse[40:70] == 7).all() and not (lse[70:] == 7).any()
        else:
            assert (out[left] == 7).all() and (lse[left] == 7).all()
        F.close(lse.cpu()[keep], l[keep], tl[keep], "lse")
        F.close(out.cpu()[keep], o[keep], to[keep], "out")


def test_one_row_and_one_head_of_any_stride():
    g = torch.Generator().manual_seed(7)
    q, kv, rope = F.rand(g, 9, 1, 192).to(D), F.rand(g, 30, 1, 256).to(D), F.rand(g, 30, 64).to(D)
    cq, ck, ws = F.starts([9]).to(D), F.starts([30]).to(D), nsa.alloc_mla_prefill_workspace()
    want = _prefill(q, kv, rope, cq, ck, True)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    odd = lambda t, n, d: t.as_strided((n, 1, d), (t.stride(0), 1, 1), t.storage_offset())
    nsa.nsa_mla_prefill(odd(q, 9, 128), odd(q[..., 128:], 9, 64), odd(kv, 30, 128), rope, odd(kv[..., 128:], 30, 128), cq, ck, True,
                        F.SCALE, out, lse, ws)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    # one query, one key
    cq, ck = F.starts([1]).to(D), F.starts([1]).to(D)
    one = lambda t, d: t[:1].as_strided((1, 1, d), (3, 5, 1), t.storage_offset())
    out, lse = torch.empty((1, 1, 128), dtype=F.BF, device=D), torch.empty((1, 1), device=D)
    nsa.nsa_mla_prefill(one(q, 128), one(q[..., 128:], 64), one(kv, 128), rope[:1].as_strided((1, 64), (1, 1)), one(kv[..., 128:], 128),
                        cq, ck, True, F.SCALE, out, lse, ws)
    assert torch.equal(out, kv[:1, :, 128:])


def test_queries_that_are_not_finite_stay_alone():
    g = torch.Generator().manual_seed(8)
    q, kv, rope = F.rand(g, 200, 2, 192).to(D), F.rand(g, 400, 2, 256).to(D), F.rand(g, 400, 64).to(D)
    clean = _prefill(q, kv, rope, F.starts([200]), F.starts([400]), True)
    q[3, 1, 7], q[140, 0, 190] = float("nan"), float("inf")
    out, lse = _prefill(q, kv, rope, F.starts([200]), F.starts([400]), True)
    assert torch.isnan(out[3, 1]).all() and torch.isnan(lse[3, 1]) and torch.isnan(out[140, 0]).all() and torch.isnan(lse[140, 0])
    for a, b in ((out, clean[0]), (lse, clean[1])):
        a[3, 1], a[140, 0] = b[3, 1], b[140, 0]
        assert torch.equal(a, b)


@pytest.mark.parametrize("captured", [False, True])
def test_calls_right_behind_what_writes_their_inputs(captured):
    # one set of buffers, written and read again and again without a wait: a call that began too early shows
    g = torch.Generator().manual_seed(10)
    N, R, H, keys = 24, 33, 4, 300
    src = F.rand(g, N, R, H, 192).to(D)
    caches, w = F.rand(g, N, keys, 576).to(D), F.weight(g, H).to(D)
    slots = torch.arange(keys, dtype=torch.int32, device=D)
    cq, ck = F.starts([R]).to(D), F.starts([keys]).to(D)
    q, kv = torch.empty_like(src[0]), torch.empty_like(caches[0])
    kv_new, rope = torch.empty((keys, H, 256), dtype=F.BF, device=D), torch.empty((keys, 64), dtype=F.BF, device=D)
    lat, out, lse = torch.empty((R, H, 512), dtype=F.BF, device=D), torch.empty((R, H, 128), dtype=F.BF, device=D), torch.empty((R, H), device=D)
    back, joined, jl = torch.empty_like(out), torch.empty_like(out), torch.empty_like(lse)
    ws, wse = nsa.alloc_mla_prefill_workspace(), nsa.alloc_mla_expand_workspace(keys)

    def run(i, wait, into):
        for f in (lambda: q.copy_(src[i]), lambda: kv.copy_(caches[i]),
                  lambda: nsa.nsa_mla_expand_kv(nsa.DT_BF16, kv, slots, w, kv_new, rope, wse),
                  lambda: nsa.nsa_mla_prefill(q[..., :128], q[..., 128:], kv_new[..., :128], rope, kv_new[..., 128:], cq, ck, True,
                                              F.SCALE, out, lse, ws),
                  lambda: nsa.nsa_mla_absorb_q(q[..., :128], w, lat), lambda: nsa.nsa_mla_project_v(lat, w, back),
                  lambda: nsa.nsa_merge_attention([out, back], [lse, lse], joined, jl),
                  lambda: [a.copy_(b) for a, b in zip(into, (out, lat, back, joined, jl))]):
            f()
            if wait:
                torch.cuda.synchronize()

    results = lambda: [tuple(torch.empty_like(t) for t in (out, lat, back, joined, jl)) for _ in range(N)]
    want, got = results(), results()
    for i in range(N):
        run(i, True, want[i])
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
    for i in range(N):
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b)
