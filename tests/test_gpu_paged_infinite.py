"""nsa_paged_mla and nsa_mla_key_weights where a position that a row sees has a score of -inf (an infinity in
its latent): the position has no weight, lse is that of the other positions, and 0 x inf makes the output
NaN in exactly the components that are not finite, whatever the other rows of the request see and however
the positions are split.  A row all of whose scores are -inf has lse -inf and outputs 0 (NaN in those components).
Tolerances are those of test_gpu_paged_mla, with the sums taken over what is finite."""
import math

import pytest
import torch

from tests._paged import SCALE, Problem, slots_of
from tests.test_gpu_paged_mla import _run, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def nsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


SHAPES = [("bf16", 2, 8, 64), ("bf16", 2, 16, 64), ("bf16", 4, 16, 64), ("bf16", 2, 128, 64), ("bf16", 2, 7, 5),
          ("fp8", 2, 8, 64), ("fp8", 2, 16, 64), ("fp8", 4, 16, 64), ("fp8", 2, 128, 64), ("fp8", 4, 128, 64),
          ("fp8", 3, 4, 3), ("f32", 2, 3, 16)]


def _problem(kv, n, H, ps):
    lens = [130, 1, 300, 129, 64, 700]
    row_len = []
    for b, l in enumerate(lens):
        # the drafts of a verify step; in request 2 the first row is much shorter than the others
        row_len += [max(0, l - (n - 1 - i)) if b != 2 or i > 0 else 40 for i in range(n)]
    p = Problem(lens, n=n, H=H, kv=kv, ps=ps, seed=17, row_len=row_len)
    # a position all of whose scores are -inf: one component -inf where the queries are positive, or (e4m3 has no
    # infinity) a block of equal codes with an infinite scale where they are negative
    if kv == "fp8":
        p.q[..., 256:384] = -(p.q[..., 256:384].abs() + 0.125)
    else:
        p.q[..., 5] = p.q[..., 5].abs() + 0.125
    # seen by the last row alone; the only one; seen by all rows and by all but the first; alone in its tile; in a whole tile
    for b, at in ((0, [129]), (1, [0]), (2, [3, 200, 299]), (3, [128]), (5, [100, 400])):
        for pos in at:
            s = int(slots_of(p.table[b], pos + 1, p.ps)[pos])
            if kv == "fp8":
                p.kv[s, 256:384] = 0x38  # 1.0
                p.kv[s, 512:528].view(torch.float32)[2] = math.inf
            else:
                p.kv[s, 5] = -math.inf
    return p


def _err(p, r, k):
    return float((p.q[r].double().abs() @ k.abs().T).max()) * SCALE * 577 * 2.0 ** -24


@pytest.mark.parametrize("kv,n,H,ps", SHAPES)
def test_attention(nsa, kv, n, H, ps):
    p = _problem(kv, n, H, ps)
    out, lse, code = _run(nsa, p)
    assert code == 0
    out, lse = out.double().cpu(), lse.double().cpu()
    for r in range(p.R):
        if int(p.row_len[r]) == 0:
            assert not out[r].any() and torch.isneginf(lse[r]).all()
            continue
        x, k = p.scores(r)
        assert not torch.isnan(x).any()
        want = torch.logsumexp(x, 1)
        pr = torch.exp(x - torch.where(torch.isinf(want), torch.zeros_like(want), want)[:, None])
        exp = pr @ k[:, :p.dl]
        fin = torch.where(torch.isfinite(k), k, torch.zeros_like(k))
        e = _err(p, r, fin)
        none = torch.isneginf(want)
        assert torch.equal(torch.isneginf(lse[r]), none), (r, lse[r])
        assert ((lse[r] - want).abs() <= 2 * e + 2.0 ** -22 * (2 + want.abs()))[~none].all(), (r, lse[r], want)
        assert torch.equal(torch.isnan(out[r]), torch.isnan(exp)), (r, torch.isnan(out[r]).sum(), torch.isnan(exp).sum())
        ok = ~torch.isnan(exp)
        if p.q_dt == 0:
            tol = (2.0 ** -18 + 4 * e) * (1 + exp.abs())
        else:
            tol = (2.0 ** -8 + 4 * e) * (pr @ fin[:, :p.dl].abs()) + 2.0 ** -8 * exp.abs() + 2.0 ** -20
        assert ((out[r] - exp).abs() <= tol)[ok].all(), r


@pytest.mark.parametrize("kv,n,H,ps", SHAPES)
def test_weights(nsa, kv, n, H, ps):
    p = _problem(kv, n, H, ps)
    lse = torch.full((p.R, p.H), -math.inf)
    want = torch.zeros((p.B, p.max_len), dtype=torch.float64)
    e = 0.0
    for r in range(p.R):
        if int(p.row_len[r]) == 0:
            continue
        x, k = p.scores(r)
        lse[r] = torch.logsumexp(x, 1).float()
        if not torch.isinf(lse[r]).any():
            want[r // n, :x.shape[1]] += torch.exp(x - lse[r].double()[:, None]).sum(0)
            e = max(e, _err(p, r, torch.where(torch.isfinite(k), k, torch.zeros_like(k))))
    total = torch.zeros((p.B, p.max_len), device="cuda")
    assert _weights(nsa, p, lse, total) == 0
    rel = 2 * e + 64 * 2.0 ** -23 + (p.n * p.H + 8) * 2.0 ** -24
    assert ((total.double().cpu() - want).abs() <= rel * want + 1e-30).all()
