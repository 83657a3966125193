"""nsa_mla_prefill where many values are not finite: each component of a row's result is that of the values the row sees, and
the call takes a small multiple of its time."""
import pytest
import torch

import deepseek_sparse_mla_indexer_gb300 as nsa
from tests import _forms as F

pytestmark = pytest.mark.gpu
D = "cuda"
NAN, INF = float("nan"), float("inf")


def _call(q, kv, k_rope, cu_q, cu_k, causal, ws):
    out = torch.full((*q.shape[:2], 128), 7.0, dtype=F.BF, device=D)
    lse, status = torch.full(q.shape[:2], 7.0, device=D), torch.zeros(1, dtype=torch.int32, device=D)
    nsa.nsa_mla_prefill(q[..., :128], q[..., 128:], kv[..., :128], k_rope, kv[..., 128:], cu_q, cu_k, causal, F.SCALE, out, lse, ws, status)
    assert nsa.nsa_status_read(status) == 0
    return out.cpu(), lse.cpu()


def _inputs(nq, nk, H, seed):
    g = torch.Generator().manual_seed(seed)
    return F.rand(g, sum(nq), H, 192), F.rand(g, sum(nk), H, 256), F.rand(g, sum(nk), 64), g


def _check(nq, nk, H, causal, change, seed):
    q, kv, k_rope, g = _inputs(nq, nk, H, seed)
    clean = kv.clone()
    change(kv[..., 128:], g)
    ws = nsa.alloc_mla_prefill_workspace()
    cu_q, cu_k = F.starts(nq).to(D), F.starts(nk).to(D)
    _, clean_lse = _call(q.to(D), clean.to(D), k_rope.to(D), cu_q, cu_k, causal, ws)
    out, lse = _call(q.to(D), kv.to(D), k_rope.to(D), cu_q, cu_k, causal, ws)
    assert torch.equal(lse, clean_lse)
    # the formula: weights are positive, so a component is NaN if a NaN or infinities of both signs are seen, an infinity if
    # those of one sign are, and otherwise the sum over values all of which are finite
    o, _, tol, _ = F.attention(q, torch.nan_to_num(kv, nan=0, posinf=0, neginf=0), k_rope, nq, nk, causal)
    q0 = k0 = 0
    for a, b in zip(nq, nk):
        v = kv[k0:k0 + b, :, 128:]
        sees = (torch.arange(b)[None, :] <= torch.arange(b - a, b)[:, None]) if causal else torch.ones((a, b), dtype=torch.bool)
        nan, pos, neg = (torch.einsum("qt,thd->qhd", sees.float(), x.float()) > 0 for x in (torch.isnan(v), v == INF, v == -INF))
        want = o[q0:q0 + a]
        want[pos], want[neg] = INF, -INF
        want[nan | (pos & neg)] = NAN
        q0, k0 = q0 + a, k0 + b
    F.close(out, o, tol, "out")


def _sprinkled(share):
    def change(v, g):
        u = torch.rand(v.shape, generator=g)
        for i, x in enumerate((NAN, INF, -INF)):
            v[(u >= i * share) & (u < (i + 1) * share)] = x
    return change


CHANGES = {
    "all NaN": lambda v, g: v.fill_(NAN), "all infinite": lambda v, g: v.fill_(-INF),
    "a few": _sprinkled(0.0005), "some": _sprinkled(0.004), "many": _sprinkled(0.2),
}
CASES = {
    "a prompt": ([300], [300]), "after a prefix": ([140, 1], [500, 130]), "ends inside a step": ([257, 60, 5], [257, 190, 3]),
    "in parts": ([130], [2600]), "parts of other lengths": ([7, 40], [3000, 700]),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("what", CHANGES)
@pytest.mark.parametrize("name", CASES)
def test_components_are_those_of_the_values_seen(name, what, causal):
    _check(*CASES[name], 2, causal, CHANGES[what], seed=41)


@pytest.mark.parametrize("what", ["all NaN", "all infinite", "many"])
def test_the_call_takes_a_small_multiple_of_its_time(what):
    # a block of queries is done twice and its masked keys are read once more: about twice the time.  Each masked score
    # taken again for each component was hundreds of times
    n, H = 2048, 16
    q, kv, k_rope, g = _inputs([n], [n], H, 42)
    ws, cu, args = nsa.alloc_mla_prefill_workspace(), F.starts([n]).to(D), [q.to(D), None, k_rope.to(D)]
    out, lse = torch.empty((n, H, 128), dtype=F.BF, device=D), torch.empty((n, H), device=D)

    def best(kv):
        times = []
        for _ in range(8):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(4):
                nsa.nsa_mla_prefill(args[0][..., :128], args[0][..., 128:], kv[..., :128], args[2], kv[..., 128:], cu, cu, True, F.SCALE,
                                    out, lse, ws)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    clean = best(kv.to(D))
    CHANGES[what](kv[..., 128:], g)
    assert best(kv.to(D)) < 5 * clean


@pytest.mark.parametrize("name,nq,nk,causal,at", [
    ("in one part", [300], [300], True, 3), ("in steps that all rows see", [130], [700], False, 5),
    ("in a share that sees nothing else", [3], [5000], False, slice(0, 900)), ("the last key", [40], [2100], True, 2060),
])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_weight_0_and_a_value_that_is_not_finite(name, nq, nk, causal, at, bad):
    # whether that component shows it is not defined; the others, and lse, are those of the other keys
    q, kv, k_rope, _ = _inputs(nq, nk, 2, 43)
    q[..., 0] = q[..., 0].abs() + 0.1
    kv[at, :, 0] = -INF
    finite = kv.clone()
    kv[at, :, 128 + 9] = bad
    ws, cu_q, cu_k = nsa.alloc_mla_prefill_workspace(), F.starts(nq).to(D), F.starts(nk).to(D)
    want, got = (_call(q.to(D), x.to(D), k_rope.to(D), cu_q, cu_k, causal, ws) for x in (finite, kv))
    assert torch.equal(got[1], want[1])
    other = torch.arange(128) != 9
    assert torch.equal(got[0][..., other], want[0][..., other])
    a, b = got[0][..., 9], want[0][..., 9]
    assert (~torch.isfinite(a) | (a == b)).all() and torch.isfinite(want[0]).all()


@pytest.mark.parametrize("nq,nk,causal,at", [([300], [300], True, 3), ([130], [700], False, 5), ([3], [5000], False, slice(0, 900)),
                                             ([40], [2100], True, 2060)])
def test_a_weight_that_is_0_in_32_bits_and_an_infinity(nq, nk, causal, at):
    # scores about 300 below the others: the formula's weight is not 0, that of 32 bits is
    q, kv, k_rope, _ = _inputs(nq, nk, 2, 44)
    q[..., 0] = 16.0
    kv[at, :, 0] = -300.0
    finite = kv.clone()
    kv[at, :, 128 + 9] = INF
    ws, cu_q, cu_k = nsa.alloc_mla_prefill_workspace(), F.starts(nq).to(D), F.starts(nk).to(D)
    want, got = (_call(q.to(D), x.to(D), k_rope.to(D), cu_q, cu_k, causal, ws) for x in (finite, kv))
    assert torch.equal(got[1], want[1]) and torch.isfinite(want[0]).all()
    other = torch.arange(128) != 9
    assert torch.equal(got[0][..., other], want[0][..., other])
    a, b = got[0][..., 9], want[0][..., 9]
    assert (~torch.isfinite(a) | (a == b)).all()
