"""Latent attention's two forms as a serving loop runs them together: a prompt's chunk is written to the paged cache, its
prefix expanded chunk by chunk, attended and joined; the same queries absorbed, attended in the latent space and projected."""
import pytest
import torch

import deepseek_sparse_mla_indexer_gb300 as nsa
from tests import _forms as F
from tests import _paged as P

pytestmark = pytest.mark.gpu
D = "cuda"


class Layer:
    """Two requests over one paged cache: prefixes of different lengths, then a chunk of new tokens each."""

    def __init__(self, kv, prefix, new, H, ps=16, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.prefix, self.new, self.H, self.ps = prefix, new, H, ps
        self.lens = [a + b for a, b in zip(prefix, new)]
        table, pages = P.page_table(self.lens, ps, g)
        self.table, self.dt = table.to(D), nsa.DT_E4M3 if kv == "fp8" else nsa.DT_BF16
        self.w = F.weight(g, H)
        rows = [F.rand(g, n, 576) for n in self.lens]
        self.q = F.rand(g, sum(new), H, 192)
        self.cache = torch.zeros((pages * ps, 656), dtype=torch.uint8, device=D) if kv == "fp8" else \
            torch.zeros((pages * ps, 576), dtype=F.BF, device=D)
        self.slots = [P.slots_of(table[b], n, ps).to(torch.int32) for b, n in enumerate(self.lens)]
        status = torch.zeros(1, dtype=torch.int32, device=D)
        for r, s in zip(rows, self.slots):
            r = r.to(D)
            nsa.nsa_set_mla_kv(self.dt, r[:, :512], r[:, 512:], s.to(D), self.cache, status)
        assert nsa.nsa_status_read(status) == 0
        # what the cache holds, in 64 bits, and what it expands to; the kernels' keys and values are rounded to bf16
        self.rows = [P.row_values(self.cache.cpu(), self.dt, 512, 64)[s.long()] for s in self.slots]

    def exact(self):
        """(out, lse) of the new tokens over prefix and chunk without any rounding, and for each form the bound
        (out, lse) of what its roundings to bf16 do, half a step EPS_BF each.
        Expanded: a key's rounding moves a score by EPS_BF scale sum |q| |k| at most, d, so a weight by e^(2 d) - 1 of
        itself; values, weights, each part's result and the joined one are rounded too.
        Absorbed: a query's rounding moves a score by EPS_BF scale sum |q W_k| |c|; weights and the attended latent are
        rounded, of magnitude sum p |c| at most, and go through W_v: |W_v| sum p |c|; then the result.
        fp32 sums and 2^x add less than EPS_BF / 8 of the same magnitudes (512 products: 2^-14)."""
        w = self.w.double().view(self.H, 256, 512)
        outs, lses, expanded, absorbed, q0 = [], [], [], [], 0
        for rows, p, n in zip(self.rows, self.prefix, self.new):
            q, c = self.q[q0:q0 + n].double(), rows[:, :512]
            kv = torch.einsum("tl,hfl->thf", c, w)
            q_lat = torch.einsum("qhd,hdl->qhl", q[..., :128], w[:, :128])
            rope = torch.einsum("qhd,td->qht", q[..., 128:], rows[:, 512:])
            hidden = torch.arange(p + n)[None, None, :] > torch.arange(p, p + n)[:, None, None]
            x = ((torch.einsum("qhl,tl->qht", q_lat, c) + rope) * F.SCALE).masked_fill(hidden, -torch.inf)
            lse = torch.logsumexp(x, -1)
            weights = torch.exp(x - lse[..., None])
            out = torch.einsum("qht,thd->qhd", weights, kv[..., 128:])
            both = torch.einsum("qhd,td->qht", q[..., 128:].abs(), rows[:, 512:].abs()) / 8
            for bounds, keys, size in (
                    (expanded, torch.einsum("qhd,thd->qht", q[..., :128].abs(), kv[..., :128].abs()),
                     torch.einsum("qht,thd->qhd", weights, kv[..., 128:].abs())),
                    (absorbed, torch.einsum("qhl,tl->qht", q_lat.abs(), c.abs()),
                     torch.einsum("qhl,hfl->qhf", torch.einsum("qht,tl->qhl", weights, c.abs()), w[:, 128:].abs()))):
                d = (((keys * 9 / 8 + both) * F.EPS_BF * F.SCALE).masked_fill(hidden, 0).amax(-1) + 2.0 ** -14)[..., None]
                bounds.append((size * (torch.expm1(2 * d) + 5 * F.EPS_BF) + 2 * F.EPS_BF * out.abs(), d[..., 0] + lse.abs() * 2.0 ** -20))
            outs.append(out), lses.append(lse)
            q0 += n
        return torch.cat(outs), torch.cat(lses), *([torch.cat(t) for t in zip(*b)] for b in (expanded, absorbed))


def _expanded(L, chunk):
    status = torch.zeros(1, dtype=torch.int32, device=D)
    H, total_q = L.H, sum(L.new)
    q, cu_q, w = L.q.to(D), F.starts(L.new).to(D), L.w.to(D)
    ws, parts, lses = nsa.alloc_mla_prefill_workspace(), [], []

    def attend(slots, lens, causal):
        m = sum(lens)
        kv, k_rope = torch.empty((m, H, 256), dtype=F.BF, device=D), torch.empty((m, 64), dtype=F.BF, device=D)
        out, lse = torch.empty((total_q, H, 128), dtype=F.BF, device=D), torch.empty((total_q, H), device=D)
        nsa.nsa_mla_expand_kv(L.dt, L.cache, slots, w, kv, k_rope, nsa.alloc_mla_expand_workspace(m), status)
        nsa.nsa_mla_prefill(q[..., :128], q[..., 128:], kv[..., :128], k_rope, kv[..., 128:], cu_q, F.starts(lens).to(D), causal,
                            F.SCALE, out, lse, ws, status)
        parts.append(out), lses.append(lse)

    slot_table = torch.zeros((len(L.lens), max(L.lens)), dtype=torch.int32)
    for b, s in enumerate(L.slots):
        slot_table[b, :len(s)] = s
    slot_table = slot_table.to(D)
    attend(torch.cat([s[p:] for s, p in zip(L.slots, L.prefix)]).to(D), L.new, True)
    for c in range(0, max(L.prefix), chunk):
        lens = [max(0, min(chunk, p - c)) for p in L.prefix]
        flat = torch.empty(sum(lens), dtype=torch.int32, device=D)
        nsa.nsa_flatten_page_table(slot_table[:, c:].contiguous(), torch.tensor(lens, dtype=torch.int32, device=D),
                                   F.starts(lens)[:-1].contiguous().to(D), flat, status)
        attend(flat, lens, False)
    while len(parts) > 1:  # up to eight at a time, in place
        n = min(8, len(parts))
        nsa.nsa_merge_attention(parts[:n], lses[:n], parts[0], lses[0])
        parts[1:n], lses[1:n] = [], []
    assert nsa.nsa_status_read(status) == 0
    return parts[0], lses[0]


def _absorbed(L):
    status = torch.zeros(1, dtype=torch.int32, device=D)
    H, R = L.H, sum(L.new)
    q, w = L.q.to(D), L.w.to(D)
    q_lat, lat, out = (torch.empty((R, H, d), dtype=F.BF, device=D) for d in (512, 512, 128))
    lse = torch.empty((R, H), device=D)
    nsa.nsa_mla_absorb_q(q[..., :128], w, q_lat, status)
    n = max(L.new)  # requests with fewer rows are padded with rows of length 0
    at = torch.cat([torch.arange(k) + b * n for b, k in enumerate(L.new)]).to(D)
    qn, qr = torch.zeros((len(L.new) * n, H, 512), dtype=F.BF, device=D), torch.zeros((len(L.new) * n, H, 64), dtype=F.BF, device=D)
    qn[at], qr[at] = q_lat, q[..., 128:]
    row_len = torch.zeros(len(L.new) * n, dtype=torch.int32, device=D)
    row_len[at] = torch.cat([torch.arange(p + 1, p + k + 1) for p, k in zip(L.prefix, L.new)]).to(torch.int32).to(D)
    o, l = torch.empty_like(qn), torch.empty(qn.shape[:2], device=D)
    nsa.nsa_paged_mla(nsa.DT_BF16, L.dt, qn, qr, L.cache, L.ps, L.table, row_len, n, max(L.lens), F.SCALE, o, l,
                      nsa.alloc_paged_mla_workspace(nsa.DT_BF16, L.dt, qn.shape[0], n, H, max(L.lens)), status)
    lat.copy_(o[at]), lse.copy_(l[at])
    nsa.nsa_mla_project_v(lat, w, out, status)
    assert nsa.nsa_status_read(status) == 0
    return out, lse


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("prefix,new,chunk", [([0, 0], [40, 7], 64), ([300, 77], [33, 50], 100), ([1000, 5], [20, 1], 100),
                                              ([130, 131], [1, 1], 50)])
def test_both_forms(kv, prefix, new, chunk):
    L = Layer(kv, prefix, new, H=16, seed=len(new) + sum(prefix))
    out, lse, expanded, absorbed = L.exact()
    for name, (o, l), (tol_o, tol_l) in (("expanded", _expanded(L, chunk), expanded), ("absorbed", _absorbed(L), absorbed)):
        F.close(l, lse, tol_l, name + " lse")
        F.close(o, out, tol_o, name + " out")


def test_captured_and_replayed():
    L = Layer("bf16", [300, 77], [33, 50], H=16, seed=5)
    want = _expanded(L, 400)
    H, R, m = L.H, 83, sum(L.lens)
    q, w = L.q.to(D), L.w.to(D)
    flat = torch.cat(L.slots).to(D)
    kv, rope = torch.zeros((m, H, 256), dtype=F.BF, device=D), torch.zeros((m, 64), dtype=F.BF, device=D)
    out, lse = torch.zeros((R, H, 128), dtype=F.BF, device=D), torch.zeros((R, H), device=D)
    q_lat = torch.zeros((R, H, 512), dtype=F.BF, device=D)
    ws, ews = nsa.alloc_mla_prefill_workspace(), nsa.alloc_mla_expand_workspace(m)
    cu_q, cu_k = F.starts(L.new).to(D), F.starts(L.lens).to(D)

    def step():
        nsa.nsa_mla_absorb_q(q[..., :128], w, q_lat)
        nsa.nsa_mla_expand_kv(L.dt, L.cache, flat, w, kv, rope, ews)
        nsa.nsa_mla_prefill(q[..., :128], q[..., 128:], kv[..., :128], rope, kv[..., 128:], cu_q, cu_k, True, F.SCALE, out, lse, ws)

    step()
    eager = [t.clone() for t in (kv, rope, out, lse, q_lat)]
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            step()
    for _ in range(3):
        for t in (kv, rope, out, lse, q_lat):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, (kv, rope, out, lse, q_lat)))
    # prefix and chunk in one causal call; the chunks joined
    o, l, (tol_o, tol_l), _ = L.exact()
    for got in ((out, lse), want):
        F.close(got[1], l, tol_l, "lse")
        F.close(got[0], o, tol_o, "out")
