"""nsa_paged_mla and nsa_mla_key_weights on the GPU against their formulas in 64 bits.

Tolerances, from the arithmetic:
  lse, weights  fp32 sums of exact products: a score x has an error of at most
        eps_s = 577 * 2^-24 * sum|q k| * sm_scale (576 fp32 additions, each off by at
        most half a step of a partial sum that sum|q k| bounds, doubled where an
        accumulator truncates), so lse, a weighted mean of scores, is off by at
        most 2 eps_s + 2^-22 * (2 + |lse|) and a weight relatively by as much as
        x and lse together.
  out   fp32 kernels: 2^-18 * (1 + |o|).  bf16: the weights are rounded to bf16 for the
        product with V (at most 2^-8 relative, so 2^-8 sum p|v|) and the result once
        more (2^-8 of it).
"""
import pytest
import torch

from tests._paged import SCALE, Problem, slots_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def nsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


def _run(nsa, p, stream=None, q=None, out=None, max_len=None, ws=None, table=None):
    """The attention call on device copies; returns (out, lse, status code)."""
    q = p.q.cuda() if q is None else q
    max_len = p.max_len if max_len is None else max_len
    out = torch.full((p.R, p.H, p.dl), float("nan"), dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full((p.R, p.H), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = nsa.alloc_paged_mla_workspace(p.q_dt, p.kv_dt, p.R, p.n, p.H, max_len, p.dl, p.dr)
    nsa.nsa_paged_mla(p.q_dt, p.kv_dt, q[..., :p.dl], q[..., p.dl:], p.kv.cuda(), p.ps,
                      (p.table if table is None else table).cuda(), p.row_len.cuda(), p.n, max_len, SCALE, out, lse, ws,
                      status, stream)
    return out, lse, nsa.nsa_status_read(status, stream)


def _score_err(p, r):
    """eps_s of the module's docstring, for row r."""
    if not int(p.row_len[r]):
        return 0.0
    return float((p.q[r].double().abs() @ p.values(r).abs().T).max()) * SCALE * 577 * 2.0 ** -24


def _check(p, out, lse):
    eo, el = p.attention()
    out, lse = out.double().cpu(), lse.double().cpu()
    for r in range(p.R):
        if int(p.row_len[r]) == 0:
            assert not out[r].any() and torch.isneginf(lse[r]).all()
            continue
        e = _score_err(p, r)
        assert torch.isfinite(lse[r]).all()
        assert ((lse[r] - el[r]).abs() <= 2 * e + 2.0 ** -22 * (2 + el[r].abs())).all(), (r, (lse[r] - el[r]).abs().max())
        if p.q_dt == 0:
            assert ((out[r] - eo[r]).abs() <= (2.0 ** -18 + 4 * e) * (1 + eo[r].abs())).all()
        else:
            x, k = p.scores(r)
            spread = torch.exp(x - el[r][:, None]) @ k[:, :p.dl].abs()  # sum p|v|
            assert ((out[r] - eo[r]).abs() <= (2.0 ** -8 + 4 * e) * spread + 2.0 ** -8 * eo[r].abs() + 2.0 ** -20).all(), r


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("n,H,ps,lens", [
    (1, 16, 64, [1, 0, 2, 63, 64, 65]),
    (1, 16, 64, [127, 128, 129, 1000]),
    (1, 128, 64, [300, 1, 2111, 257]),
    (1, 64, 128, [129, 640, 5]),
    (1, 100, 16, [77, 300]),
    (1, 20, 32, [31, 33, 95]),
    (4, 16, 64, [3, 200, 1025]),
    (4, 128, 64, [4, 515]),
    (3, 20, 8, [2, 9, 130]),
    (2, 7, 24, [50, 200]),
    (1, 1, 64, [700]),
    (1, 192, 64, [400, 70]),
])
def test_against_the_formula(nsa, kv, n, H, ps, lens):
    p = Problem(lens, n=n, H=H, kv=kv, ps=ps, seed=len(lens) * 100 + H)
    out, lse, code = _run(nsa, p)
    assert code == 0
    _check(p, out, lse)


@pytest.mark.parametrize("kv,ps,dl,dr,H", [("f32", 16, 64, 16, 4), ("f32", 5, 512, 64, 3), ("bf16", 3, 512, 64, 16),
                                           ("fp8", 1, 512, 64, 8), ("bf16", 64, 256, 32, 5), ("fp8", 7, 128, 2, 2),
                                           ("f32", 1, 33, 0, 1)])
def test_other_dims_and_page_sizes(nsa, kv, ps, dl, dr, H):
    p = Problem([40, 0, 1, 33], H=H, kv=kv, ps=ps, dl=dl, dr=dr, seed=5)
    out, lse, code = _run(nsa, p)
    assert code == 0
    _check(p, out, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_many_requests_of_mixed_length(nsa, kv):
    # more requests than thread blocks, empty ones among them (a padded batch)
    lens = [(i * 37) % 400 if i % 7 else 0 for i in range(333)]
    p = Problem(lens, H=16, kv=kv, seed=3)
    out, lse, code = _run(nsa, p)
    assert code == 0
    _check(p, out, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_one_long_request_is_split_and_joined(nsa, kv):
    p = Problem([20011], H=16, kv=kv, seed=4)
    out, lse, code = _run(nsa, p)
    assert code == 0
    _check(p, out, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_growing_scores_move_the_running_maximum(nsa, kv):
    p = Problem([1500, 400], H=64, kv=kv, seed=6)
    if kv == "bf16":  # keys grow along the positions, so later tiles exceed the maximum of earlier ones
        for b in range(2):
            s = slots_of(p.table[b], p.lens[b], 64)
            p.kv[s] = (p.kv[s].float() * torch.linspace(0.01, 8, p.lens[b])[:, None]).to(torch.bfloat16)
    else:
        p.q = (p.q.float() * 12).to(torch.bfloat16)
    out, lse, code = _run(nsa, p)
    assert code == 0
    _check(p, out, lse)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_positions_past_the_length_are_never_used(nsa, kv):
    """NaN and infinities behind each request's length (same page and later ones) change nothing."""
    p = Problem([70, 1, 130], H=32, kv=kv, seed=8, fill=2 ** 30)
    clean = _run(nsa, p)
    live = torch.cat([slots_of(p.table[b], l, p.ps) for b, l in enumerate(p.lens)])
    dead = torch.ones(p.pages * p.ps, dtype=torch.bool)
    dead[live] = False
    if kv == "bf16":
        p.kv[dead] = float("nan")
        p.kv[dead.nonzero()[::2, 0]] = float("inf")
    else:
        p.kv[dead] = 0xFF  # NaN codes, scales and rope values
    out, lse, code = _run(nsa, p)
    assert code == 0 and clean[2] == 0
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
    _check(p, out, lse)


def test_rows_of_one_request_with_their_own_lengths(nsa):
    p = Problem([200, 300], n=4, H=16, seed=9, row_len=[0, 7, 200, 64, 300, 1, 128, 129])
    out, lse, code = _run(nsa, p)
    assert code == 0
    _check(p, out, lse)


def test_bad_pages_and_lengths_are_reported_and_left_out(nsa):
    p = Problem([200, 300, 100], H=16, seed=10)
    full = _run(nsa, p)[:2]
    t = p.table.clone()
    t[1, 2] = p.pages            # positions 128 .. 191 of request 1
    t[1, 4] = -1                 # positions 256 .. 299
    out, lse, code = _run(nsa, p, table=t)
    assert code == nsa.ERR_BOUNDS
    assert torch.equal(out[0], full[0][0]) and torch.equal(lse[2], full[1][2])
    x, k = p.scores(1)
    ok = torch.ones(300, dtype=torch.bool)
    ok[128:192] = False
    ok[256:] = False
    want = torch.logsumexp(x[:, ok], 1)
    assert ((lse[1].double().cpu() - want).abs() <= 1e-4).all()
    exp = torch.exp(x[:, ok] - want[:, None]) @ k[ok, :512]
    assert ((out[1].double().cpu() - exp).abs() <= 0.02 * (1 + exp.abs())).all()
    p.row_len[1] = -3
    p.row_len[2] = p.max_len + 1
    out, lse, code = _run(nsa, p)
    assert code == nsa.ERR_BOUNDS
    assert not out[1:].any() and torch.isneginf(lse[1:]).all()
    assert torch.equal(out[0], full[0][0])


def test_strided_queries_and_a_wider_table(nsa):
    p = Problem([90, 400], H=16, seed=11)
    want = _run(nsa, p)
    wide = torch.zeros((p.R, 2 * p.H, 600), dtype=torch.bfloat16, device="cuda")
    wide[:, :p.H, 8:584] = p.q.cuda()
    q = wide[:, :p.H, 8:584]      # row stride 2 * H * 600: rows that are not packed
    got = _run(nsa, p, q=q)
    odd = torch.zeros((p.R, p.H, 577), dtype=torch.bfloat16, device="cuda")
    odd[..., 1:] = p.q.cuda()     # neither 16-byte aligned nor a stride of whole 16 bytes
    got2 = _run(nsa, p, q=odd[..., 1:])
    t = torch.zeros((p.B, p.table.shape[1] + 5), dtype=torch.int32, device="cuda")
    t[:, :p.table.shape[1]] = p.table.cuda()
    got3 = _run(nsa, p, table=t[:, :p.table.shape[1]])
    for g in (got, got2, got3):
        assert g[2] == 0
        _check(p, g[0], g[1])
    assert torch.equal(got3[0], want[0])


def test_equal_calls_give_equal_bits_and_write_only_their_rows(nsa):
    p = Problem([5000, 17, 900], H=128, seed=12)
    big = torch.full((p.R + 2, p.H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    a = _run(nsa, p, out=big[1:1 + p.R])
    b = _run(nsa, p)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert (big[0] == 7).all() and (big[-1] == 7).all()


def test_a_larger_bound_on_the_length_changes_only_the_plan(nsa):
    p = Problem([500, 3], H=16, seed=13)
    t = torch.zeros((2, 64), dtype=torch.int32)
    t[:, :p.table.shape[1]] = p.table
    out, lse, code = _run(nsa, p, max_len=4096, table=t)
    assert code == 0
    _check(p, out, lse)


def test_a_quantised_cache_equals_its_dequantised_copy(nsa):
    """fp8 rows give, to the accumulation's rounding, what nsa_dequantize_kv_paged's bf16 rows give."""
    p = Problem([300, 1100], H=128, kv="fp8", seed=14)
    out, lse, code = _run(nsa, p)
    slots = torch.arange(p.pages * p.ps, dtype=torch.int32, device="cuda")
    deq = torch.empty((p.pages * p.ps, 576), dtype=torch.bfloat16, device="cuda")
    nsa.nsa_dequantize_kv_paged(p.kv.cuda(), slots, deq)
    d = Problem([300, 1100], H=128, seed=14)
    d.table, d.kv, d.q = p.table, deq.cpu(), p.q
    out2, lse2, code2 = _run(nsa, d)
    assert code == 0 and code2 == 0
    assert ((lse - lse2).abs() <= 2.0 ** -20 * (2 + lse.abs())).all()
    _check(d, out, lse)


def test_captured_replayed_and_on_another_stream(nsa):
    p = Problem([900, 3000], H=128, seed=15)
    want = _run(nsa, p)
    q, kv, t, rl = p.q.cuda(), p.kv.cuda(), p.table.cuda(), p.row_len.cuda()
    outs = [torch.zeros((p.R, p.H, 512), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lses = [torch.zeros((p.R, p.H), device="cuda") for _ in range(2)]
    ws = [nsa.alloc_paged_mla_workspace(1, 1, p.R, 1, p.H, p.max_len) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        nsa.nsa_paged_mla(1, 1, q[..., :512], q[..., 512:], kv, 64, t, rl, 1, p.max_len, SCALE, outs[0], lses[0], ws[0])
    torch.cuda.synchronize()
    for _ in range(3):  # replayed on one stream while the same call runs on another
        outs[0].zero_()
        outs[1].zero_()
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            nsa.nsa_paged_mla(1, 1, q[..., :512], q[..., 512:], kv, 64, t, rl, 1, p.max_len, SCALE, outs[1], lses[1], ws[1])
        torch.cuda.synchronize()
        for o, l in zip(outs, lses):
            assert torch.equal(o, want[0]) and torch.equal(l, want[1])


# ------------------------------------------------------------------ key weights

def _weights(nsa, p, lse, total, table=None):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = p.q.cuda()
    nsa.nsa_mla_key_weights(p.q_dt, p.kv_dt, q[..., :p.dl], q[..., p.dl:], p.kv.cuda(), p.ps,
                            (p.table if table is None else table).cuda(), p.row_len.cuda(), p.n, p.max_len, SCALE,
                            lse.cuda(), total, status)
    return nsa.nsa_status_read(status)


def _check_weights(p, lse, got):
    w = p.weights(lse)
    e = max(_score_err(p, r) for r in range(p.R))
    # the weight of a row and head is off relatively by the error of x - lse, which fp32 holds to
    # 2^-23 of values up to 64, and the exponential's few steps; the sum over heads adds n*H steps
    rel = 2 * e + 64 * 2.0 ** -23 + (p.n * p.H + 8) * 2.0 ** -24
    assert ((got.double().cpu() - w).abs() <= rel * w + 1e-30).all(), ((got.double().cpu() - w).abs() / (w + 1e-30)).max()


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("n,H,ps,lens", [
    (1, 16, 64, [1, 0, 2, 63, 64, 65]),
    (1, 128, 64, [300, 1, 2111, 257]),
    (1, 100, 16, [77, 300]),
    (1, 20, 32, [31, 33, 129]),
    (4, 16, 64, [3, 200, 1025]),
    (4, 128, 64, [4, 515]),
    (3, 20, 8, [2, 9, 130]),
    (1, 192, 64, [400, 70]),
    (1, 1, 128, [700]),
])
def test_weights_against_the_formula(nsa, kv, n, H, ps, lens):
    p = Problem(lens, n=n, H=H, kv=kv, ps=ps, seed=len(lens) * 10 + H)
    _, lse = p.attention()
    lse = lse.float()
    total = torch.zeros((p.B, p.max_len), device="cuda")
    assert _weights(nsa, p, lse, total) == 0
    _check_weights(p, lse, total)
    # every head of every row hands out one unit of weight over its positions
    rows = (p.row_len > 0).view(p.B, n).sum(1) * H
    assert ((total.double().sum(1).cpu() - rows).abs() <= 1e-3 * (1 + rows)).all()


@pytest.mark.parametrize("kv,ps,dl,dr,H", [("f32", 16, 64, 16, 4), ("bf16", 3, 512, 64, 16), ("fp8", 1, 512, 64, 8),
                                           ("f32", 1, 33, 0, 1)])
def test_weights_other_dims_and_page_sizes(nsa, kv, ps, dl, dr, H):
    p = Problem([40, 0, 1, 33], H=H, kv=kv, ps=ps, dl=dl, dr=dr, seed=5)
    lse = p.attention()[1].float()
    total = torch.zeros((p.B, p.max_len), device="cuda")
    assert _weights(nsa, p, lse, total) == 0
    _check_weights(p, lse, total)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_weights_are_added_and_other_positions_stay(nsa, kv):
    p = Problem([200, 300], n=4, H=16, kv=kv, seed=21, row_len=[0, 7, 190, 64, 290, 1, 128, 129])
    lse = p.attention()[1].float()
    big = torch.full((p.B, 400), 0.5, device="cuda")
    assert _weights(nsa, p, lse, big[:, :310]) == 0
    assert (big[0, 190:] == 0.5).all() and (big[1, 290:] == 0.5).all()
    one = big.clone()
    assert _weights(nsa, p, lse, big[:, :310]) == 0
    w = p.weights(lse)
    assert ((one[:, :300].double().cpu() - 0.5 - w).abs() <= 1e-5 * (1 + w)).all()
    assert ((big[:, :300].double().cpu() - 0.5 - 2 * w).abs() <= 2e-5 * (1 + w)).all()
    again = torch.full((p.B, 400), 0.5, device="cuda")
    assert _weights(nsa, p, lse, again[:, :310]) == 0
    assert torch.equal(again, one)


def test_weights_bad_pages_and_lengths(nsa):
    p = Problem([200, 300, 100], H=16, seed=22)
    lse = p.attention()[1].float()
    t = p.table.clone()
    t[1, 2] = p.pages
    total = torch.zeros((3, 300), device="cuda")
    assert _weights(nsa, p, lse, total, table=t) == nsa.ERR_BOUNDS
    w = p.weights(lse)
    w[1, 128:192] = 0
    assert ((total.double().cpu() - w).abs() <= 1e-4 * (1e-6 + w)).all()
    p.row_len[1] = -1
    p.row_len[2] = 301
    total.zero_()
    assert _weights(nsa, p, lse, total) == nsa.ERR_BOUNDS
    assert not total[1:].any() and total[0].any()
