"""The products with the up-projection (nsa_mla_expand_kv, nsa_mla_absorb_q, nsa_mla_project_v) against 64 bits."""
import pytest
import torch

import deepseek_sparse_mla_indexer_gb300 as nsa
from tests import _forms as F
from tests import _paged as P

pytestmark = pytest.mark.gpu

ROWS = [1, 2, 15, 16, 17, 33, 64, 100, 129, 255, 256, 257, 1000]


def _cache(g, kv, slots):
    x = torch.randn((slots, 576), generator=g)
    return P.fp8_rows(x, 512, 64) if kv == "fp8" else x.to(F.BF)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("m,H", [(m, 1) for m in ROWS] + [(1, 16), (77, 5), (300, 3), (700, 16)] +
                         [(257, 128), (3651, 16), (2050, 27)])  # these on pairs of CTAs
def test_expand(kv, m, H):
    g = torch.Generator().manual_seed(m)
    cache, w = _cache(g, kv, m + 9), F.weight(g, H)
    slots = torch.randperm(m + 9, generator=g)[:m].to(torch.int32)
    slots[m // 2] = -1  # padding
    out = torch.full((m, H, 256), 7.0, dtype=F.BF, device="cuda")
    rope = torch.full((m, 64), 7.0, dtype=F.BF, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    dt = nsa.DT_E4M3 if kv == "fp8" else nsa.DT_BF16
    nsa.nsa_mla_expand_kv(dt, cache.cuda(), slots.cuda(), w.cuda(), out, rope, nsa.alloc_mla_expand_workspace(m), status)
    assert nsa.nsa_status_read(status) == 0
    rows = P.row_values(cache, 2 if kv == "fp8" else 1, 512, 64)[slots.long()]
    rows[m // 2] = 0
    want = rows[:, :512] @ w.double().T
    F.close(out.view(m, -1), want, F.product_tol(rows[:, :512], w.double(), want), "kv")
    assert torch.equal(rope.cpu().double(), rows[:, 512:])


def test_expand_reports_slots_outside():
    g = torch.Generator().manual_seed(1)
    cache, w = _cache(g, "bf16", 20), F.weight(g, 2)
    slots = torch.tensor([3, 20, 19, 1 << 30], dtype=torch.int32)
    out, rope = torch.full((4, 2, 256), 7.0, dtype=F.BF, device="cuda"), torch.full((4, 64), 7.0, dtype=F.BF, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    nsa.nsa_mla_expand_kv(nsa.DT_BF16, cache.cuda(), slots.cuda(), w.cuda(), out, rope, nsa.alloc_mla_expand_workspace(4), status)
    assert nsa.nsa_status_read(status) == nsa.ERR_BOUNDS
    for i in (1, 3):
        assert (out[i] == 0).all() and (rope[i] == 0).all()
    for i in (0, 2):
        assert torch.equal(rope[i].cpu(), cache[int(slots[i]), 512:])


def test_expand_writes_its_rows_alone_and_a_larger_workspace_serves():
    g = torch.Generator().manual_seed(2)
    cache, w = _cache(g, "bf16", 64), F.weight(g, 3)
    out = torch.full((40, 3, 256), 7.0, dtype=F.BF, device="cuda")
    rope = torch.full((40, 64), 7.0, dtype=F.BF, device="cuda")
    ws = nsa.alloc_mla_expand_workspace(1000)
    slots = torch.arange(33, dtype=torch.int32, device="cuda")
    nsa.nsa_mla_expand_kv(nsa.DT_BF16, cache.cuda(), slots, w.cuda(), out[:33], rope[:33], ws)
    assert (out[33:] == 7).all() and (rope[33:] == 7).all()
    first = out[:33].clone()
    nsa.nsa_mla_expand_kv(nsa.DT_BF16, cache.cuda(), slots, w.cuda(), out[:33], rope[:33], ws)
    assert torch.equal(first, out[:33])


@pytest.mark.parametrize("R,H", [(r, 2) for r in ROWS] + [(1, 128), (32, 128), (5, 17), (3, 1)])
@pytest.mark.parametrize("op", ["absorb", "project"])
def test_head_products(op, R, H):
    g = torch.Generator().manual_seed(R * 100 + H)
    w = F.weight(g, H)
    if op == "absorb":
        x, out = F.rand(g, R, H, 192)[..., :128], torch.full((R + 2, H, 512), 7.0, dtype=F.BF, device="cuda")
        nsa.nsa_mla_absorb_q(x.cuda(), w.cuda(), out[:R])
    else:
        x, out = F.rand(g, R, H, 512), torch.full((R + 2, H, 128), 7.0, dtype=F.BF, device="cuda")
        nsa.nsa_mla_project_v(x.cuda(), w.cuda(), out[:R])
    w64 = w.double().view(H, 256, 512)
    for h in range(H):
        wh = w64[h, :128].T if op == "absorb" else w64[h, 128:]
        want = x[:, h].double() @ wh.T
        F.close(out[:R, h], want, F.product_tol(x[:, h].double(), wh, want), f"head {h}")
    assert (out[R:] == 7).all()


@pytest.mark.parametrize("op", ["absorb", "project"])
def test_strides_and_order(op):
    g = torch.Generator().manual_seed(3)
    R, H, K = 37, 6, 128 if op == "absorb" else 512
    w = F.weight(g, H).cuda()
    call = nsa.nsa_mla_absorb_q if op == "absorb" else nsa.nsa_mla_project_v
    xs = {"packed": F.rand(g, R, H, K)}
    xs["heads first"] = xs["packed"].transpose(0, 1).contiguous().transpose(0, 1)
    wide = torch.zeros((R, H, K + 24), dtype=F.BF)
    wide[..., 8:K + 8] = xs["packed"]
    xs["inside wide rows"] = wide[..., 8:K + 8]
    got = {}
    for name, x in xs.items():
        if name == "packed":
            d = x.cuda()
        elif name == "heads first":
            d = x.transpose(0, 1).contiguous().cuda().transpose(0, 1)
        else:
            d = wide.cuda()[..., 8:K + 8]
        out = torch.empty((R, H, 512 if op == "absorb" else 128), dtype=F.BF, device="cuda")
        call(d, w, out)
        got[name] = out.cpu()
    assert torch.equal(got["packed"], got["heads first"]) and torch.equal(got["packed"], got["inside wide rows"])


@pytest.mark.parametrize("op", ["absorb", "project"])
def test_one_row_and_one_head_of_any_stride(op):
    g = torch.Generator().manual_seed(4)
    K = 128 if op == "absorb" else 512
    call = nsa.nsa_mla_absorb_q if op == "absorb" else nsa.nsa_mla_project_v
    w = F.weight(g, 1).cuda()
    x = F.rand(g, 5, 1, K).cuda()
    a, b = (torch.empty((n, 1, 640 - K), dtype=F.BF, device="cuda") for n in (5, 1))
    call(x.as_strided((5, 1, K), (K, 3, 1)), w, a)
    call(x[2:3].as_strided((1, 1, K), (1, 0, 1), x[2:3].storage_offset()), w, b)
    assert torch.equal(a[2:3], b)


@pytest.mark.parametrize("op", ["absorb", "project"])
def test_not_finite_stays_in_its_row(op):
    g = torch.Generator().manual_seed(5)
    R, H, K = 20, 2, 128 if op == "absorb" else 512
    call = nsa.nsa_mla_absorb_q if op == "absorb" else nsa.nsa_mla_project_v
    w, x = F.weight(g, H).cuda(), F.rand(g, R, H, K).cuda()
    a, b = (torch.empty((R, H, 640 - K), dtype=F.BF, device="cuda") for _ in range(2))
    call(x, w, a)
    x[7, 1, 3] = float("nan")
    call(x, w, b)
    assert torch.isnan(b[7, 1]).all()
    b[7, 1] = a[7, 1]
    assert torch.equal(a, b)
