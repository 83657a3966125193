"""nsa_merge_attention against 64 bits, in place, and with parts that saw no key."""
import pytest
import torch

import deepseek_sparse_mla_indexer_gb300 as nsa
from tests import _forms as F

pytestmark = pytest.mark.gpu


def _parts(n, shape, dtype, seed, none=0.3):
    g = torch.Generator().manual_seed(seed)
    parts = [F.rand(g, *shape, dtype=dtype) for _ in range(n)]
    lses = [torch.randn(shape[:-1], generator=g) * 3 for _ in range(n)]
    for p, l in zip(parts, lses):
        gone = torch.rand(shape[:-1], generator=g) < none
        l[gone] = -torch.inf
        p[gone] = float("nan")  # not looked at
    return parts, lses


def _check(out, lse, parts, lses, out_dtype):
    o, l, size = F.merge(parts, lses)
    # a weight: exp of a difference of lse below 2^5 in fp32 and their sum, a few steps; n products and sums
    rel = (32 + 4 * len(parts) + 8) * 2.0 ** -23
    half = F.EPS_BF if out_dtype == F.BF else 2.0 ** -24
    F.close(lse, l, rel + torch.nan_to_num(l.abs(), posinf=0, neginf=0) * 2.0 ** -22, "lse")
    F.close(out, o, rel * size * (1 + half) + half * o.abs() + 1e-30, "out")


@pytest.mark.parametrize("dtypes", [(F.BF, F.BF), (F.F32, F.F32), (F.F32, F.BF)], ids=["bf16", "f32", "f32 to bf16"])
@pytest.mark.parametrize("n", range(1, 9))
def test_parts(n, dtypes):
    parts, lses = _parts(n, (7, 3, 128), dtypes[0], n)
    out = torch.empty((7, 3, 128), dtype=dtypes[1], device="cuda")
    lse = torch.empty((7, 3), device="cuda")
    nsa.nsa_merge_attention([p.cuda() for p in parts], [l.cuda() for l in lses], out, lse)
    _check(out, lse, parts, lses, dtypes[1])


@pytest.mark.parametrize("D", [8, 24, 64, 200, 512, 1000, 2048])
@pytest.mark.parametrize("rows", [1, 5, 300])
def test_widths(rows, D):
    parts, lses = _parts(3, (rows, D), F.BF, D)
    out, lse = torch.full((rows + 1, D), 7.0, dtype=F.BF, device="cuda"), torch.full((rows + 1,), 7.0, device="cuda")
    nsa.nsa_merge_attention([p.cuda() for p in parts], [l.cuda() for l in lses], out[:rows], lse[:rows])
    _check(out[:rows], lse[:rows], parts, lses, F.BF)
    assert (out[rows:] == 7).all() and (lse[rows:] == 7).all()


@pytest.mark.parametrize("dtype", [F.BF, F.F32])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_in_place(at, dtype):
    parts, lses = _parts(3, (513, 5, 128), dtype, 9)
    pd, ld = [p.cuda() for p in parts], [l.cuda() for l in lses]
    nsa.nsa_merge_attention(pd, ld, pd[at], ld[at])
    _check(pd[at], ld[at], parts, lses, dtype)


def test_no_key_anywhere_and_lse_that_are_not_finite():
    parts = [torch.ones((5, 16), device="cuda") * (i + 1) for i in range(2)]
    inf = float("inf")
    lses = [torch.tensor(x, device="cuda") for x in ([-inf, float("nan"), inf, 0.0, -inf], [-inf, 0.0, 0.0, -inf, float("nan")])]
    out, lse = torch.empty((5, 16), device="cuda"), torch.empty(5, device="cuda")
    nsa.nsa_merge_attention(parts, lses, out, lse)
    assert (out[0] == 0).all() and lse[0] == -inf
    assert torch.isnan(out[[1, 2, 4]]).all() and torch.isnan(lse[[1, 2, 4]]).all()
    assert (out[3] == 1).all() and lse[3] == 0


def test_far_apart_and_equal_calls():
    parts, lses = _parts(2, (100, 128), F.BF, 12, none=0)
    lses[1] = lses[0] - 500.0
    out, lse = torch.empty((100, 128), dtype=F.BF, device="cuda"), torch.empty(100, device="cuda")
    nsa.nsa_merge_attention([p.cuda() for p in parts], [l.cuda() for l in lses], out, lse)
    assert torch.equal(out.cpu(), parts[0]) and torch.equal(lse.cpu(), lses[0])


def test_no_rows():
    e, l = torch.empty((0, 128), dtype=F.BF, device="cuda"), torch.empty(0, device="cuda")
    nsa.nsa_merge_attention([e, e], [l, l], e.clone(), l.clone())


@pytest.mark.parametrize("dtypes", [(F.BF, F.BF), (F.F32, F.F32), (F.F32, F.BF)], ids=["bf16", "f32", "f32 to bf16"])
@pytest.mark.parametrize("n", [2, 3, 8])
def test_values_near_the_end_of_the_range(n, dtypes):
    # an average of finite values is finite, although their sum is not
    g = torch.Generator().manual_seed(n)
    parts = [(F.rand(g, 9, 64).sign() * 2.0 ** 127 * (1 + torch.rand((9, 1), generator=g) / 2)).to(dtypes[0]) for _ in range(n)]
    parts[1:4] = [parts[0].clone() for _ in parts[1:4]]
    lses = [torch.randn(9, generator=g) for _ in range(n)]
    out, lse = torch.empty((9, 64), dtype=dtypes[1], device="cuda"), torch.empty(9, device="cuda")
    nsa.nsa_merge_attention([p.cuda() for p in parts], [l.cuda() for l in lses], out, lse)
    assert torch.isfinite(out).all()
    _check(out, lse, parts, lses, dtypes[1])
