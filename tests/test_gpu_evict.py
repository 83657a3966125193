"""nsa_evict_select and nsa_evict_compact on the GPU against plain Python, and a run of
attention, weights, selection and compaction together.  Everything but the attention is
whole numbers or moved bytes: compared for equality."""
import numpy as np
import pytest
import torch

from tests._paged import SCALE, Problem, page_table, select, slots_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def nsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


def _select(nsa, total, lens, sinks, recent, budget, max_len=None, keep=None):
    B = len(lens)
    keep = torch.full((B, budget), -7, dtype=torch.int32, device="cuda") if keep is None else keep
    new = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    nsa.nsa_evict_select(total, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                         total.shape[1] if max_len is None else max_len, sinks, recent, budget, keep, new, status)
    return keep.cpu().numpy(), new.cpu().numpy(), nsa.nsa_status_read(status)


def _totals(kind, B, W, seed):
    g = np.random.default_rng(seed)
    if kind == "heavy":
        t = np.exp(2 * g.standard_normal((B, W)))
    elif kind == "ties":
        t = g.integers(0, 5, (B, W)).astype(np.float64)
    elif kind == "equal":
        t = np.full((B, W), 0.25)
    elif kind == "zeros":
        t = np.where(g.random((B, W)) < 0.5, -0.0, 0.0)
    else:  # every kind of value
        t = g.standard_normal((B, W))
        t[g.random((B, W)) < 0.1] = np.nan
        t[g.random((B, W)) < 0.05] = np.inf
        t[g.random((B, W)) < 0.05] = -np.inf
        t[g.random((B, W)) < 0.05] = -np.finfo(np.float32).max
        t[g.random((B, W)) < 0.05] = 1e-42
    return t.astype(np.float32)


@pytest.mark.parametrize("kind", ["heavy", "ties", "equal", "zeros", "all"])
@pytest.mark.parametrize("W,lens,sinks,recent,budget", [
    (40, [40, 0, 1, 9, 10, 11], 2, 3, 10),
    (700, [700, 33, 699, 512], 0, 0, 33),
    (700, [700, 650], 16, 17, 33),        # sinks + recent = budget: none from between
    (5000, [5000, 4097, 4096, 100], 4, 64, 1000),
    (5000, [5000], 0, 0, 4999),
    (5000, [4999, 2], 1, 0, 1),
    (33000, [33000, 8192, 12345], 7, 101, 9000),
])
def test_select(nsa, kind, W, lens, sinks, recent, budget):
    t = _totals(kind, len(lens), W, W + budget)
    keep, new, code = _select(nsa, torch.from_numpy(t).cuda(), lens, sinks, recent, budget)
    want, n = select(t, lens, sinks, recent, budget)
    assert code == 0
    assert np.array_equal(new, n)
    assert np.array_equal(keep, want)


def test_select_rows_longer_than_shared_memory_holds(nsa):
    L = 8 * 48 * 1024 + 777
    t = _totals("heavy", 1, L, 5)
    keep, new, code = _select(nsa, torch.from_numpy(t).cuda(), [L], 3, 5, 70001)
    mid = t[0, 3:L - 5]
    best = np.sort(np.argsort(-mid, kind="stable")[:70001 - 8]) + 3
    want = np.concatenate([np.arange(3), best, np.arange(L - 5, L)])
    assert code == 0 and new[0] == 70001 and np.array_equal(keep[0], want)


def test_select_reads_no_further_than_the_length_and_writes_no_further_than_the_budget(nsa):
    t = _totals("heavy", 3, 600, 6)
    lens = [600, 90, 300]
    want, n = select(t, lens, 2, 8, 100)
    for b, l in enumerate(lens):
        t[b, l:] = np.nan if b % 2 else np.inf
    wide = torch.full((5, 120), -9, dtype=torch.int32, device="cuda")
    big = torch.zeros((3, 640), device="cuda")
    big[:, :600] = torch.from_numpy(t).cuda()
    _, new, code = _select(nsa, big[:, :600], lens, 2, 8, 100, keep=wide[1:4])
    assert code == 0 and np.array_equal(new, n)
    w = wide.cpu().numpy()
    assert np.array_equal(w[1:4, :100], want)
    assert (w[0] == -9).all() and (w[4] == -9).all() and (w[:, 100:] == -9).all()


def test_select_reports_bad_lengths(nsa):
    t = _totals("heavy", 3, 64, 7)
    keep, new, code = _select(nsa, torch.from_numpy(t).cuda(), [65, 64, -1], 1, 1, 8)
    assert code == nsa.ERR_BOUNDS
    assert new.tolist() == [0, 8, 0] and (keep[0] == -1).all() and (keep[2] == -1).all()
    assert np.array_equal(keep[1], select(t, [0, 64, 0], 1, 1, 8)[0][1])


# ------------------------------------------------------------------ compact

def _arrays(slots, g, kind):
    u8 = lambda n: torch.randint(0, 256, (slots, n), generator=g, dtype=torch.uint8)
    if kind == "serving":      # fp8 latent rows, indexer keys, their scales
        return [u8(656), u8(128), torch.rand(slots, generator=g)]
    if kind == "bf16":
        return [torch.randn((slots, 576), generator=g).to(torch.bfloat16), torch.rand(slots, generator=g)]
    if kind == "odd":          # rows of no whole words
        return [u8(37), u8(4), u8(2)]
    if kind == "wide":
        return [u8(12000), u8(9000)]
    return []


def _expect(arrays, total, table, ps, keep, new, old):
    arrays = [a.clone() for a in arrays]
    total = total.clone()
    for b, (n, o) in enumerate(zip(new, old)):
        if n == o:
            continue
        s = slots_of(table[b], max(int(o), 1), ps)
        src = torch.from_numpy(keep[b, :n].astype(np.int64))
        for a in arrays:
            a[s[:n]] = a[s[src]].clone()
        t = total[b].clone()
        total[b, :o] = 0
        total[b, :n] = t[src]
    return arrays, total


def _compact(nsa, arrays, total, table, ps, keep, new, old, max_len, ws=None):
    B = len(old)
    dev = [a.cuda() for a in arrays]
    tot = None if total is None else total.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = torch.full((nsa.nsa_evict_compact_workspace_bytes(B, max_len),), 0xAB, dtype=torch.uint8, device="cuda")
    i32 = lambda v: torch.as_tensor(np.asarray(v, dtype=np.int32)).cuda()
    nsa.nsa_evict_compact(i32(keep), i32(new), i32(old), max_len, table.cuda(), ps, dev, tot, ws, status)
    code = nsa.nsa_status_read(status)
    return [d.cpu() for d in dev], None if tot is None else tot.cpu(), code


def _same(got, want):
    return all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", ["serving", "bf16", "odd", "wide", "none"])
@pytest.mark.parametrize("ps,lens,budget,sinks,recent", [
    (64, [300, 64, 0, 1, 65], 64, 3, 9),
    (16, [1000, 999, 17], 500, 0, 0),
    (1, [50, 7], 11, 1, 2),
    (24, [2000], 1990, 4, 4),
    (64, [3000, 2900, 130, 2000], 10, 2, 2),
])
def test_compact(nsa, kind, ps, lens, budget, sinks, recent):
    g = torch.Generator().manual_seed(ps + budget)
    table, pages = page_table(lens, ps, g, fill=-5)
    W = max(lens)
    t = _totals("heavy", len(lens), W, budget)
    keep, new = select(t, lens, sinks, recent, budget)
    arrays = _arrays(pages * ps, g, kind)
    total = torch.from_numpy(t)
    got, gt, code = _compact(nsa, arrays, total, table, ps, keep, new, lens, W)
    want, wt = _expect(arrays, total, table, ps, keep, new, lens)
    assert code == 0
    assert _same(got, want)
    assert torch.equal(gt, wt)
    got, gt, code = _compact(nsa, arrays, None, table, ps, keep, new, lens, W)  # without totals
    assert code == 0 and gt is None
    assert _same(got, want)


@pytest.mark.parametrize("pattern", ["front", "back", "one_gap", "alternate", "random"])
def test_compact_long_chains_of_chunks(nsa, pattern):
    """Orders of kept rows that make every chunk wait for its predecessors, many requests at once."""
    lens, ps = [20000, 15001, 9999], 64
    g = torch.Generator().manual_seed(3)
    table, pages = page_table(lens, ps, g)
    keeps, new = [], []
    rng = np.random.default_rng(4)
    for L in lens:
        k = {"front": np.arange(L - 1), "back": np.arange(1, L), "one_gap": np.delete(np.arange(L), L // 3),
             "alternate": np.arange(0, L, 2), "random": np.sort(rng.permutation(L)[:L * 2 // 3])}[pattern]
        keeps.append(k)
        new.append(len(k))
    keep = np.full((3, max(new)), -1, np.int32)
    for b, k in enumerate(keeps):
        keep[b, :len(k)] = k
    arrays = _arrays(pages * ps, g, "serving")
    total = torch.rand((3, 20000), generator=g)
    want, wt = _expect(arrays, total, table, ps, keep, new, lens)
    ws = nsa.alloc_evict_workspace(3, 20000)
    for _ in range(3):
        got, gt, code = _compact(nsa, arrays, total, table, ps, keep, new, lens, 20000, ws)
        assert code == 0
        assert _same(got, want)
        assert torch.equal(gt, wt)


def test_compact_refuses_what_it_cannot_follow_row_by_row(nsa):
    lens, ps = [100, 100, 100], 16
    g = torch.Generator().manual_seed(5)
    table, pages = page_table(lens, ps, g)
    arrays, total = _arrays(pages * ps, g, "serving"), torch.rand((3, 100), generator=g)
    keep = np.tile(np.arange(50, dtype=np.int32) * 2, (3, 1))
    # a length beyond the budget, a new length beyond the old one: the requests stay as they are
    got, gt, code = _compact(nsa, arrays, total, table, ps, keep, [51, 50, 50], [100, 49, 100], 100)
    want, wt = _expect(arrays, total, table, ps, keep, [100, 49, 50], [100, 49, 100])
    assert code == nsa.ERR_BOUNDS
    assert _same(got, want)
    assert torch.equal(gt, wt)
    # a page outside the cache: the rows that need it stay
    bad = table.clone()
    bad[0, 5] = pages  # positions 80 .. 95 of request 0: sources of rows 40 .. 47
    got, gt, code = _compact(nsa, arrays, total, bad, ps, keep, [50] * 3, lens, 100)
    want, wt = _expect(arrays, total, table, ps, keep, [50] * 3, lens)
    assert code == nsa.ERR_BOUNDS
    s = slots_of(table[0], 100, ps)
    for b, o in zip(want, arrays):
        b[s[40:48]] = o[s[40:48]]
    assert _same(got, want)
    # a position past the length, and one out of order
    keep[0, 49], keep[1, 10] = 100, 18
    got, gt, code = _compact(nsa, arrays, total, table, ps, keep, [50] * 3, lens, 100)
    assert code == nsa.ERR_BOUNDS
    s2 = slots_of(table[2], 100, ps)
    assert _same([a[s2] for a in got], [b[s2] for b in want])


def test_compact_captured_and_replayed(nsa):
    lens, ps = [3000, 2000], 64
    g = torch.Generator().manual_seed(6)
    table, pages = page_table(lens, ps, g)
    t = _totals("heavy", 2, 3000, 6)
    keep, new = select(t, lens, 4, 64, 1000)
    arrays = _arrays(pages * ps, g, "serving")
    total = torch.from_numpy(t)
    want, wt = _expect(arrays, total, table, ps, keep, new, lens)
    dev, tot = [a.cuda() for a in arrays], total.cuda()
    args = [torch.from_numpy(keep).cuda(), torch.from_numpy(new).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
            3000, table.cuda(), ps, dev, tot, nsa.alloc_evict_workspace(2, 3000)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nsa.nsa_evict_compact(*args)
    for _ in range(2):
        for d, a in zip(dev, arrays):
            d.copy_(a)
        tot.copy_(total)
        graph.replay()
        torch.cuda.synchronize()
        assert _same([d.cpu() for d in dev], want)
        assert torch.equal(tot.cpu(), wt)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_decode_steps_that_evict_attend_to_the_kept_positions(nsa, kv):
    """Decode steps add their weights to the totals, a request over its budget is cut, and the
    next step on the compacted cache equals attention over the kept positions alone."""
    H, ps, budget, sinks, recent = 16, 64, 256, 4, 32
    p = Problem([700, 200, 391], H=H, kv=kv, ps=ps, seed=33)
    kvd, table = p.kv.cuda(), p.table.cuda()
    total = torch.zeros((p.B, 704), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = p.row_len.cuda()
    g = torch.Generator().manual_seed(34)
    out = torch.empty((p.B, H, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((p.B, H), device="cuda")
    ws = nsa.alloc_paged_mla_workspace(1, p.kv_dt, p.B, 1, H, 700)
    for _ in range(3):
        q = torch.randn((p.B, H, 576), generator=g).to(torch.bfloat16).cuda() * 2
        nsa.nsa_paged_mla(1, p.kv_dt, q[..., :512], q[..., 512:], kvd, ps, table, lens, 1, 700, SCALE, out, lse, ws, status)
        nsa.nsa_mla_key_weights(1, p.kv_dt, q[..., :512], q[..., 512:], kvd, ps, table, lens, 1, 700, SCALE, lse, total, status)
    keep = torch.empty((p.B, budget), dtype=torch.int32, device="cuda")
    new = torch.empty(p.B, dtype=torch.int32, device="cuda")
    t0 = total.cpu().numpy()
    nsa.nsa_evict_select(total, lens, 700, sinks, recent, budget, keep, new, status)
    nsa.nsa_evict_compact(keep, new, lens, 700, table, ps, [kvd], total, nsa.alloc_evict_workspace(p.B, 700), status)
    k_np, n_np = select(t0, p.lens, sinks, recent, budget)
    assert np.array_equal(keep.cpu().numpy(), k_np) and np.array_equal(new.cpu().numpy(), n_np)
    q = torch.randn((p.B, H, 576), generator=g).to(torch.bfloat16)
    qd = q.cuda()
    nsa.nsa_paged_mla(1, p.kv_dt, qd[..., :512], qd[..., 512:], kvd, ps, table, new, 1, 700, SCALE, out, lse, ws, status)
    assert nsa.nsa_status_read(status) == 0
    p.q = q
    o, l = out.double().cpu(), lse.double().cpu()
    for b in range(p.B):
        x, k = p.scores(b)  # the untouched CPU copy: the kept positions of the original cache
        kept = torch.from_numpy(k_np[b, :n_np[b]].astype(np.int64))
        x, k = x[:, kept], k[kept]
        want = torch.logsumexp(x, 1)
        pr = torch.exp(x - want[:, None])
        assert ((l[b] - want).abs() <= 1e-4 * (1 + want.abs())).all()
        spread = pr @ k[:, :512].abs()
        assert ((o[b] - pr @ k[:, :512]).abs() <= 2.0 ** -7 * spread + 2.0 ** -20).all()
    assert (total[0, 256:700] == 0).all() and (total[1].cpu().numpy() == t0[1]).all()
