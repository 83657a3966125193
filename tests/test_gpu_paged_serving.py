"""Dense paged attention, key weights and eviction as a serving loop uses them: fed by
nsa_metadata, beside the sparse attention, in captured graphs, on several streams, with
padded batches and workspaces that serve several shapes.  The tolerances are those of
test_gpu_paged_mla.py unless a test says otherwise."""
import numpy as np
import pytest
import torch

from tests._paged import SCALE, Problem, select, slots_of
from tests.test_gpu_paged_mla import _check, _check_weights, _run, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def nsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("n,H,ps", [(4, 128, 128), (4, 128, 8), (2, 128, 16), (1, 48, 64), (1, 33, 64), (1, 17, 256), (6, 128, 64),
                                    (1, 96, 40)])
def test_column_groups_and_page_sizes(nsa, kv, n, H, ps):
    p = Problem([5, 700, 0, 128, 333], n=n, H=H, kv=kv, ps=ps, seed=n * H + ps)
    out, lse, code = _run(nsa, p)
    assert code == 0
    _check(p, out, lse)
    total = torch.zeros((p.B, p.max_len), device="cuda")
    lse64 = p.attention()[1].float()
    assert _weights(nsa, p, lse64, total) == 0
    _check_weights(p, lse64, total)


@pytest.mark.parametrize("kv,n,H", [("bf16", 1, 128), ("fp8", 1, 128), ("fp8", 4, 128), ("bf16", 4, 16), ("fp8", 1, 64)])
def test_many_padded_requests_over_several_ctas_a_tile(nsa, kv, n, H):
    lens = [(i * 53) % 260 if i % 5 else 0 for i in range(90)]
    p = Problem(lens, n=n, H=H, kv=kv, seed=17)
    out, lse, code = _run(nsa, p)
    assert code == 0
    _check(p, out, lse)


@pytest.mark.parametrize("kv,n,H", [("bf16", 1, 128), ("bf16", 1, 16), ("fp8", 1, 128), ("fp8", 4, 128), ("fp8", 1, 16), ("fp8", 1, 64)])
def test_nan_behind_the_length_reaches_nothing(nsa, kv, n, H):
    """Stale rows behind each length, and queries of a padded row, are NaN."""
    p = Problem([70, 1, 130, 257, 40], n=n, H=H, kv=kv, seed=8, fill=2 ** 30)
    clean = _run(nsa, p)
    assert clean[2] == 0
    live = torch.cat([slots_of(p.table[b], l, p.ps) for b, l in enumerate(p.lens)])
    dead = torch.ones(p.pages * p.ps, dtype=torch.bool)
    dead[live] = False
    if kv == "bf16":
        p.kv[dead] = float("nan")
    else:
        p.kv[dead] = 0xFF
    for _ in range(2):  # twice: the second call's shared memory and workspace hold what the first left
        out, lse, code = _run(nsa, p)
        assert code == 0
        assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
    total = torch.zeros((p.B, p.max_len), device="cuda")
    lse64 = p.attention()[1].float()
    assert _weights(nsa, p, lse64, total) == 0
    _check_weights(p, lse64, total)
    # a padded request whose queries were never written
    last = p.row_len.view(p.B, n)
    last[-1] = 0
    p.q.view(p.B, n, H, 576)[-1] = float("nan")
    out, lse, code = _run(nsa, p)
    assert code == 0
    keep = (p.B - 1) * n
    assert torch.equal(out[:keep], clean[0][:keep]) and torch.equal(lse[:keep], clean[1][:keep])
    assert not out[keep:].any() and torch.isneginf(lse[keep:]).all()
    total.zero_()
    assert _weights(nsa, p, torch.where(torch.isinf(lse), lse, lse64.cuda()).cpu(), total) == 0
    assert torch.isfinite(total).all() and not total[-1].any()


def test_one_head_rows_of_a_wider_buffer(nsa):
    p = Problem([300, 40, 129], H=1, seed=19)
    wide = torch.zeros((p.R, 1, 640), dtype=torch.bfloat16, device="cuda")
    wide[..., :576] = p.q.cuda()
    out, lse, code = _run(nsa, p, q=wide[..., :576])
    assert code == 0
    _check(p, out, lse)


def test_a_workspace_serves_smaller_and_other_problems(nsa):
    probs = [Problem([3000, 500, 100], H=128, seed=1), Problem([700] * 9, H=16, n=4, seed=2), Problem([2500], H=16, kv="fp8", seed=3),
             Problem([600, 77], H=128, n=4, kv="fp8", seed=4)]
    need = max(nsa.nsa_paged_mla_workspace_bytes(p.q_dt, p.kv_dt, p.R, p.n, p.H, p.max_len) for p in probs)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN patterns: nothing in it is taken for a value
    for p in probs + probs[::-1]:
        out, lse, code = _run(nsa, p, ws=ws)
        assert code == 0
        _check(p, out, lse)


def test_dense_equals_sparse_where_the_top_k_holds_every_position(nsa):
    """Target-verify through nsa_metadata: rows no longer than the top-k select every position, so the
    sparse attention over the selected slots and the dense one over the page table agree to the
    rounding of their weights (2^-8 of sum p|v| each) and outputs (2^-8 each)."""
    lens, n, ps, H = [300, 90, 1500], 4, 64, 128
    p = Problem([l + n for l in lens], n=n, H=H, ps=ps, seed=23)
    B, R, W = p.B, p.R, p.max_len
    req_to_token = torch.zeros((B + 2, W), dtype=torch.int32)
    rows = torch.tensor([4, 0, 2], dtype=torch.int32)
    for b in range(B):
        req_to_token[rows[b], :p.lens[b]] = slots_of(p.table[b], p.lens[b], ps).to(torch.int32)
    md = nsa.alloc_metadata(nsa.MODE_TARGET_VERIFY, B, R, W, ps, "cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    nsa.nsa_metadata(nsa.MODE_TARGET_VERIFY, B, R, W, n, 2048, ps, torch.tensor(lens, dtype=torch.int32).cuda(), None,
                     req_to_token.cuda(), rows.cuda(), md, status)
    q, kv = p.q.cuda(), p.kv.cuda()
    out = torch.empty((R, H, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((R, H), device="cuda")
    ws = nsa.alloc_paged_mla_workspace(1, 1, R, n, H, W)
    nsa.nsa_paged_mla(1, 1, q[..., :512], q[..., 512:], kv, ps, md["real_page_table"], md["seqlens_expanded"], n, W, SCALE, out, lse,
                      ws, status)
    assert torch.equal(md["seqlens_expanded"].cpu(), torch.tensor([l + 1 + i for l in lens for i in range(n)], dtype=torch.int32))
    indices = torch.full((R, 2048), -1, dtype=torch.int32)
    for r in range(R):
        L = lens[r // n] + 1 + r % n
        indices[r, :L] = slots_of(p.table[r // n], L, ps).to(torch.int32)
    so, sl = torch.empty_like(out), torch.empty_like(lse)
    wsb = nsa.nsa_sparse_mla_workspace_bytes(1, 1, R, H, 512, 64, 2048)
    sws = torch.empty(max(wsb, 16), dtype=torch.uint8, device="cuda")
    nsa.nsa_sparse_mla(1, 1, q[..., :512], q[..., 512:], kv, indices.cuda(), SCALE, so, sl, sws, status, num_slots=p.pages * ps)
    assert nsa.nsa_status_read(status) == 0
    p.row_len = torch.tensor([l + 1 + i for l in lens for i in range(n)], dtype=torch.int32)
    _check(p, out, lse)
    assert ((lse - sl).abs() <= 2e-2 * (1 + lse.abs())).all()
    for r in range(R):
        x, k = p.scores(r)
        spread = torch.softmax(x, 1) @ k[:, :512].abs()
        o = out[r].double().cpu()
        assert ((o - so[r].double().cpu()).abs() <= 2.0 ** -7 * spread + 2.0 ** -7 * o.abs() + 1e-5).all()


def test_a_whole_eviction_step_in_one_graph_and_on_two_streams(nsa):
    """Attention, weights, selection and compaction captured once and replayed on fresh contents, while
    the same step of another batch runs on a second stream."""
    budget, sinks, recent, H, ps = 300, 4, 40, 16, 64

    class Step:
        def __init__(self, seed):
            self.p = Problem([900, 250, 411], H=H, ps=ps, kv="fp8", seed=seed)
            p = self.p
            self.q, self.kv, self.table, self.lens = p.q.cuda(), p.kv.cuda(), p.table.cuda(), p.row_len.cuda()
            self.total = torch.zeros((3, 900), device="cuda")
            self.out = torch.empty((3, H, 512), dtype=torch.bfloat16, device="cuda")
            self.lse = torch.empty((3, H), device="cuda")
            self.keep = torch.empty((3, budget), dtype=torch.int32, device="cuda")
            self.new = torch.empty(3, dtype=torch.int32, device="cuda")
            self.ws = nsa.alloc_paged_mla_workspace(1, 2, 3, 1, H, 900)
            self.ews = nsa.alloc_evict_workspace(3, 900)
            self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

        def run(self):
            a = (1, 2, self.q[..., :512], self.q[..., 512:], self.kv, ps, self.table, self.lens, 1, 900, SCALE)
            nsa.nsa_paged_mla(*a, self.out, self.lse, self.ws, self.status)
            nsa.nsa_mla_key_weights(*a, self.lse, self.total, self.status)
            nsa.nsa_evict_select(self.total, self.lens, 900, sinks, recent, budget, self.keep, self.new, self.status)
            nsa.nsa_evict_compact(self.keep, self.new, self.lens, 900, self.table, ps, [self.kv], self.total, self.ews, self.status)

        def reset(self):
            self.kv.copy_(self.p.kv)
            self.total.zero_()
            self.out.zero_()

        def check(self):
            p = self.p
            assert int(self.status) == 0
            _check(p, self.out, self.lse)
            w = torch.zeros((3, 900), device="cuda")
            assert _weights(nsa, p, self.lse.cpu(), w) == 0
            keep, new = select(w.cpu().numpy(), p.lens, sinks, recent, budget)
            assert np.array_equal(self.keep.cpu().numpy(), keep) and np.array_equal(self.new.cpu().numpy(), new)
            for b in range(3):
                s = slots_of(p.table[b], p.lens[b], ps)
                got = self.kv.cpu()[s[:new[b]]]
                assert torch.equal(got, p.kv[s[torch.from_numpy(keep[b, :new[b]].astype(np.int64))]])

    one, two = Step(41), Step(42)
    graph = torch.cuda.CUDAGraph()
    one.run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        one.run()
    side = torch.cuda.Stream()
    for _ in range(3):
        one.reset()
        two.reset()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            two.run()
        torch.cuda.synchronize()
        one.check()
        two.check()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_weights_give_equal_bits_and_follow_the_order_of_nothing(nsa, kv):
    p = Problem([1500, 3, 640], n=4, H=128, kv=kv, seed=51)
    lse = p.attention()[1].float()
    runs = []
    for _ in range(3):
        t = torch.full((3, 1500), 0.125, device="cuda")
        assert _weights(nsa, p, lse, t) == 0
        runs.append(t)
    assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])


def test_positions_beyond_32_bits_of_bytes(nsa):
    """A cache of more than 4 GiB, with the request's pages at its end."""
    ps, L, H = 64, 400, 16
    pages = (5 << 30) // (ps * 1152)
    kv = torch.empty((pages * ps, 576), dtype=torch.bfloat16, device="cuda")
    p = Problem([L], H=H, ps=ps, seed=61)
    table = torch.tensor([[pages - 1 - i for i in range(7)]], dtype=torch.int32)
    slots = slots_of(table[0], L, ps)
    rows = p.kv[slots_of(p.table[0], L, ps)]
    kv[slots.cuda()] = rows.cuda()
    out = torch.empty((1, H, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((1, H), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = p.q.cuda()
    a = (1, 1, q[..., :512], q[..., 512:], kv, ps, table.cuda(), p.row_len.cuda(), 1, L, SCALE)
    nsa.nsa_paged_mla(*a, out, lse, nsa.alloc_paged_mla_workspace(1, 1, 1, 1, H, L), status)
    total = torch.zeros((1, L), device="cuda")
    nsa.nsa_mla_key_weights(*a, lse, total, status)
    assert nsa.nsa_status_read(status) == 0
    _check(p, out, lse)
    _check_weights(p, lse.cpu(), total)
    keep, new = select(total.cpu().numpy(), [L], 2, 10, 100)
    nsa.nsa_evict_compact(torch.from_numpy(keep).cuda(), torch.from_numpy(new).cuda(), p.row_len.cuda(), L, table.cuda(), ps, [kv], total,
                          nsa.alloc_evict_workspace(1, L), status)
    assert nsa.nsa_status_read(status) == 0
    assert torch.equal(kv[slots[:100].cuda()].cpu(), rows[torch.from_numpy(keep[0].astype(np.int64))])
