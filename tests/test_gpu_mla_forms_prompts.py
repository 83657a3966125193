"""Latent attention's two forms at the sizes of prompts: the products' wide tiles with heads and strides of their own, attention
whose heads go in sections (several rounds of items, the last section smaller)."""
import pytest
import torch

import deepseek_sparse_mla_indexer_gb300 as nsa
from tests import _forms as F

pytestmark = pytest.mark.gpu
D = "cuda"


def _strided(x, layout):
    """The same values [R, H, K] on the GPU in another layout."""
    if layout == "packed":
        return x.to(D)
    if layout == "heads first":
        return x.transpose(0, 1).contiguous().to(D).transpose(0, 1)
    wide = torch.full((*x.shape[:2], x.shape[2] + 24), 3.0, dtype=F.BF, device=D)
    wide[..., 8:-16] = x.to(D)
    return wide[..., 8:-16]


# tiles of 64, 128 and 256 rows, the last one not full, on 148 .. 160 SMs
@pytest.mark.parametrize("layout", ["packed", "heads first", "inside wide rows"])
@pytest.mark.parametrize("R,H", [(520, 16), (700, 16), (900, 9), (1001, 16), (129, 128), (4001, 16)])
@pytest.mark.parametrize("op", ["absorb", "project"])
def test_head_products_of_many_rows(op, R, H, layout):
    g = torch.Generator().manual_seed(R + H)
    K = 128 if op == "absorb" else 512
    w, x = F.weight(g, H), F.rand(g, R, H, K)
    out = torch.full((R + 2, H, 640 - K), 7.0, dtype=F.BF, device=D)
    status = torch.zeros(1, dtype=torch.int32, device=D)
    (nsa.nsa_mla_absorb_q if op == "absorb" else nsa.nsa_mla_project_v)(_strided(x, layout), w.to(D), out[:R], status)
    assert nsa.nsa_status_read(status) == 0 and (out[R:] == 7).all()
    w64 = w.double().view(H, 256, 512)
    rows = torch.arange(R) if R < 1000 else torch.cat([torch.randperm(R, generator=g)[:200], torch.arange(R - 40, R)])
    for h in range(H):
        wh = w64[h, :128].T if op == "absorb" else w64[h, 128:]
        want = x[rows, h].double() @ wh.T
        F.close(out[rows.to(D), h], want, F.product_tol(x[rows, h].double(), wh, want), f"head {h}")


@pytest.mark.parametrize("op", ["absorb", "project"])
def test_a_single_head_of_a_far_stride(op):
    g = torch.Generator().manual_seed(4)
    K = 128 if op == "absorb" else 512
    call = nsa.nsa_mla_absorb_q if op == "absorb" else nsa.nsa_mla_project_v
    w, x = F.weight(g, 1).to(D), F.rand(g, 5, 1, K).to(D)
    a, b = (torch.empty((5, 1, 640 - K), dtype=F.BF, device=D) for _ in range(2))
    call(x, w, a)
    call(x.as_strided((5, 1, K), (K, 1 << 40, 1)), w, b)
    assert torch.equal(a, b)


def _reference(q, k, v, seen):
    """F.attention's (out, lse, tol_out, tol_lse) for rows q [n, 192] of one head, row i over the first seen[i] keys."""
    x, dx = (q @ k.T) * F.SCALE, (q.abs() @ k.abs().T) * F.SCALE * (192 * 2.0 ** -23 + 2.0 ** -21)
    hide = torch.arange(len(k))[None, :] >= seen[:, None]
    x, dx = x.masked_fill(hide, -torch.inf), dx.masked_fill(hide, 0.0)
    d = dx.amax(-1, keepdim=True) + 2.0 ** -20
    lse = torch.logsumexp(x, -1, keepdim=True)
    p = torch.exp(x - lse)
    out, size = p @ v, p @ v.abs()
    tol = (F.EPS_BF + 2 * d + len(k) * 2.0 ** -23) * size * (1 + F.EPS_BF) + F.EPS_BF * out.abs()
    return out, lse[:, 0], tol, d[:, 0] + lse[:, 0].abs() * 2.0 ** -22


# heads are cut into sections where their keys do not fit in L2 together and each section fills the SMs four times:
# 25 heads of a prompt go as 13 and 12, 45 of three requests and 81 over a long prefix as halves one apart
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,nq,nk", [(25, [8192], [8192]), (45, [2500, 700, 1], [4500, 3700, 900]), (81, [2000], [11000])])
def test_attention_in_sections_of_heads(H, nq, nk, causal):
    g = torch.Generator(device=D).manual_seed(H)
    q, kv, k_rope = (torch.randn(s, generator=g, device=D, dtype=F.BF) for s in ((sum(nq), H, 192), (sum(nk), H, 256), (sum(nk), 64)))
    out, lse = torch.full((sum(nq), H, 128), 7.0, dtype=F.BF, device=D), torch.full((sum(nq), H), 7.0, device=D)
    status = torch.zeros(1, dtype=torch.int32, device=D)
    nsa.nsa_mla_prefill(q[..., :128], q[..., 128:], kv[..., :128], k_rope, kv[..., 128:], F.starts(nq).to(D), F.starts(nk).to(D), causal,
                        F.SCALE, out, lse, nsa.alloc_mla_prefill_workspace(), status)
    assert nsa.nsa_status_read(status) == 0
    assert not (lse == 7).any() and torch.isfinite(lse).all() and torch.isfinite(out).all()
    pick = torch.Generator().manual_seed(1)
    q0 = k0 = 0
    for a, b in zip(nq, nk):
        rope = k_rope[k0:k0 + b].cpu().double()
        for h in range(H):
            rows = torch.unique(torch.cat([torch.randint(0, a, (6,), generator=pick), torch.tensor([0, a - 1, a // 2])]))
            at = (q0 + rows).to(D)
            k = torch.cat([kv[k0:k0 + b, h, :128].cpu().double(), rope], 1)
            o, l, to, tl = _reference(q[at, h].cpu().double(), k, kv[k0:k0 + b, h, 128:].cpu().double(),
                                      b - a + rows + 1 if causal else torch.full_like(rows, b))
            F.close(lse[at, h], l, tl, f"lse of head {h}")
            F.close(out[at, h], o, to, f"out of head {h}")
        q0, k0 = q0 + a, k0 + b
