"""nsa_mla_prefill against the formula in 64 bits: lengths around the tiles' and blocks' edges, rows without a
key, strides, parts of long rows, values that are not finite where a row must not see them."""
import pytest
import torch

import deepseek_sparse_mla_indexer_gb300 as nsa
from tests import _forms as F

pytestmark = pytest.mark.gpu


def _run(q, kv, k_rope, nq, nk, causal, scale=F.SCALE, total_q=None, fill=None, ws=None, cu_q=None, cu_k=None):
    d = "cuda"
    q, kv, k_rope = q.to(d), kv.to(d), k_rope.to(d)
    out = torch.full((q.shape[0], q.shape[1], 128), 7.0 if fill is None else fill, dtype=F.BF, device=d)
    lse = torch.full(q.shape[:2], 7.0 if fill is None else fill, device=d)
    status = torch.zeros(1, dtype=torch.int32, device=d)
    nsa.nsa_mla_prefill(q[..., :128], q[..., 128:], kv[..., :128], k_rope, kv[..., 128:],
                        (F.starts(nq) if cu_q is None else cu_q).to(d), (F.starts(nk) if cu_k is None else cu_k).to(d), causal, scale,
                        out, lse, nsa.alloc_mla_prefill_workspace() if ws is None else ws, status)
    return out.cpu(), lse.cpu(), nsa.nsa_status_read(status)


def _inputs(nq, nk, H, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (F.rand(g, sum(nq), H, 192, scale=scale), F.rand(g, max(1, sum(nk)), H, 256)[:sum(nk)],
            F.rand(g, max(1, sum(nk)), 64)[:sum(nk)])


def _check(nq, nk, H, causal, seed=0, scale=1.0):
    q, kv, k_rope = _inputs(nq, nk, H, seed, scale)
    out, lse, status = _run(q, kv, k_rope, nq, nk, causal)
    assert status == 0
    o, l, to, tl = F.attention(q, kv, k_rope, nq, nk, causal)
    F.close(lse, l, tl, "lse")
    F.close(out, o, to, "out")


CAUSAL = {
    "one token": ([1], [1]), "one after a few": ([1], [77]), "a tile": ([128], [128]), "a tile and one": ([129], [129]),
    "a block": ([256], [256]), "a block and one": ([257], [257]), "below a tile": ([127], [127]), "prefix": ([37], [637]),
    "odd prefix": ([255], [402]), "blocks with prefix": ([513], [900]), "ragged": ([5, 300, 1, 128, 64], [5, 300, 40, 129, 700]),
    "no queries between": ([3, 0, 0, 7], [3, 50, 0, 7]), "no keys": ([4, 9], [0, 9]), "fewer keys than queries": ([300, 130], [41, 129]),
    "first tile sees none": ([256], [100]), "many requests": ([2, 1, 3] * 30, [2, 9, 140] * 30),
}


@pytest.mark.parametrize("H", [1, 3])
@pytest.mark.parametrize("name", CAUSAL)
def test_causal(name, H):
    _check(*CAUSAL[name], H, True, seed=H)


OTHER = {
    "one key": ([1], [1]), "one row": ([1], [513]), "a step": ([130], [128]), "a step and one": ([2], [129]),
    "ragged": ([100, 1, 290], [300, 1000, 3]), "no keys": ([200, 3], [0, 5]), "no queries": ([0, 3], [70, 5]),
}


@pytest.mark.parametrize("H", [1, 2])
@pytest.mark.parametrize("name", OTHER)
def test_all_keys(name, H):
    _check(*OTHER[name], H, False, seed=10 + H)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq,nk", [([1], [5000]), ([3, 2], [4000, 2500]), ([200], [3333]), ([1, 1], [9000, 0]), ([300], [2100])])
def test_rows_cut_into_parts(nq, nk, causal):
    _check(nq, nk, 2, causal, seed=3)


def test_a_head_for_every_part_of_the_grid():
    # more items than SMs, of lengths far apart: every item after the first of a CTA reuses its buffers
    _check([600, 1, 20, 257], [600, 900, 20, 2000], 70, True, seed=4)


@pytest.mark.parametrize("scale", [6.0, 40.0])
def test_peaked_rows(scale):
    # maxima that grow step by step ask for fresh ones
    nq, nk, H = [140], [900], 2
    q, kv, k_rope = _inputs(nq, nk, H, 5, scale)
    k_rope = k_rope * torch.linspace(0.2, 3.0, 900)[:, None].to(F.BF)
    out, lse, status = _run(q, kv, k_rope, nq, nk, True)
    o, l, to, tl = F.attention(q, kv, k_rope, nq, nk, True)
    assert status == 0
    F.close(lse, l, tl, "lse")
    F.close(out, o, to, "out")


@pytest.mark.parametrize("causal", [True, False])
def test_strides_and_order(causal):
    g = torch.Generator().manual_seed(6)
    nq, nk, H = [70, 131], [200, 131], 4
    d = "cuda"
    # heads before rows, wide rows, keys and values in arrays of their own
    qn = F.rand(g, H, 201, 136).to(d).transpose(0, 1)[..., :128]
    qr = F.rand(g, 201, H, 72).to(d)[..., 8:]
    kn = F.rand(g, 331, H + 1, 128).to(d)[:, 1:]
    v = F.rand(g, H, 340, 128).to(d).transpose(0, 1)[9:]
    kr = F.rand(g, 331, 576).to(d)[:, 512:]
    out, lse = torch.empty((201, H, 128), dtype=F.BF, device=d), torch.empty((201, H), device=d)
    nsa.nsa_mla_prefill(qn, qr, kn, kr, v, F.starts(nq).to(d), F.starts(nk).to(d), causal, 0.05, out, lse,
                        nsa.alloc_mla_prefill_workspace())
    o, l, to, tl = F.attention(torch.cat([qn, qr], -1).cpu(), torch.cat([kn, v], -1).cpu(), kr.cpu(), nq, nk, causal, 0.05)
    F.close(lse, l, tl, "lse")
    F.close(out, o, to, "out")


@pytest.mark.parametrize("parts", [False, True])
def test_rows_of_no_request_stay(parts):
    # 8 rows before the first request, 5 behind the last; with and without parts
    H, nq, nk = (2, [6], [3000]) if parts else (200, [6], [300])
    g = torch.Generator().manual_seed(7)
    q, kv, k_rope = F.rand(g, 8 + 6 + 5, H, 192), F.rand(g, nk[0] + 4, H, 256), F.rand(g, nk[0] + 4, 64)
    out, lse, status = _run(q, kv, k_rope, nq, nk, True, cu_q=F.starts(nq, 8), cu_k=F.starts(nk, 4))
    assert status == 0
    for a in (out, lse):
        assert (a[:8] == 7).all() and (a[14:] == 7).all()
    o, l, to, tl = F.attention(q[8:14], kv[4:], k_rope[4:], nq, nk, True)
    F.close(lse[8:14], l, tl, "lse")
    F.close(out[8:14], o, to, "out")


@pytest.mark.parametrize("what", ["k", "rope", "v"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("at", [0, 64, 127, 128, 200, 299])
def test_not_finite_reaches_only_rows_that_see_it(what, bad, at):
    nq, nk, H = [300, 50], [300, 60], 2
    q, kv, k_rope = _inputs(nq, nk, H, 8)
    clean_out, clean_lse, _ = _run(q, kv, k_rope, nq, nk, True)
    if what == "k":
        kv[at, 1, 5] = bad
    elif what == "rope":
        k_rope[at, 63] = bad
    else:
        kv[at, 1, 128 + 77] = bad
    out, lse, status = _run(q, kv, k_rope, nq, nk, True)
    assert status == 0
    assert torch.equal(out[:at], clean_out[:at]) and torch.equal(lse[:at], clean_lse[:at])
    assert torch.equal(out[300:], clean_out[300:]) and torch.equal(lse[300:], clean_lse[300:])
    if what == "v":
        # the value's own component alone: every weight is positive
        other = torch.ones(128, dtype=torch.bool)
        other[77] = False
        assert torch.equal(out[:, 1][:, other], clean_out[:, 1][:, other]) and torch.equal(out[:, 0], clean_out[:, 0])
        assert torch.equal(lse, clean_lse)
        got = out[at:300, 1, 77]
        assert torch.isnan(got).all() if bad != bad else (got == bad).all()
    elif bad != bad:
        heads = [0, 1] if what == "rope" else [1]
        assert torch.isnan(out[at:300, heads]).all() and torch.isnan(lse[at:300, heads]).all()


def test_not_finite_behind_a_request_and_in_padding():
    # keys behind the last request, and the next request's first ones, inside the same step
    nq, nk, H = [20, 30], [100, 130], 2
    g = torch.Generator().manual_seed(9)
    q, kv, k_rope = F.rand(g, 50, H, 192), F.rand(g, 260, H, 256), F.rand(g, 260, 64)
    o, l, to, tl = F.attention(q, kv[:230], k_rope[:230], nq, nk, False)
    kv[230:], k_rope[230:] = float("nan"), float("inf")
    for causal in (False,):
        out, lse, status = _run(q, kv, k_rope, nq, nk, causal)
        assert status == 0
        F.close(lse, l, tl, "lse")
        F.close(out, o, to, "out")
    kv2, r2 = kv.clone(), k_rope.clone()
    kv2[100:230], r2[100:230] = float("nan"), float("nan")
    out, lse, _ = _run(q, kv2, r2, nq, nk, False)
    F.close(lse[:20], l[:20], tl[:20], "lse")
    F.close(out[:20], o[:20], to[:20], "out")
    assert torch.isnan(out[20:]).all() and torch.isnan(lse[20:]).all()


@pytest.mark.parametrize("parts", [False, True])
def test_several_odd_values_in_parts(parts):
    H, nq, nk = (1, [130], [2600]) if parts else (1, [130], [131])
    q, kv, k_rope = _inputs(nq, nk, H, 11)
    n = nk[0]
    for j, val in ((n - 1, float("inf")), (n - 40, float("nan")), (n - 129, -float("inf")), (n - 100, float("inf"))):
        kv[j, 0, 128 + 3] = val
    out, lse, _ = _run(q, kv, k_rope, nq, nk, True)
    o, l, to, tl = F.attention(q, torch.nan_to_num(kv, posinf=0, neginf=0, nan=0), k_rope, nq, nk, True)
    keep = torch.arange(128) != 3
    F.close(lse, l, tl, "lse")
    F.close(out[..., keep], o[..., keep], to[..., keep], "out")
    row = torch.arange(130) + n - 130  # the last key that each row sees
    got = out[:, 0, 3]
    assert torch.isfinite(got[row < n - 129]).all()
    assert (got[(row >= n - 129) & (row < n - 100)] == -float("inf")).all()
    assert torch.isnan(got[row >= n - 100]).all()


def test_scores_of_minus_infinity():
    nq, nk, H = [3], [140], 1
    q, kv, k_rope = _inputs(nq, nk, H, 12)
    q[:] = q.abs() + 0.1
    kv[5, 0, :128] = -float("inf")     # weight 0
    out, lse, _ = _run(q, kv, k_rope, nq, nk, False)
    keep = torch.arange(140) != 5
    o, l, to, tl = F.attention(q, kv[keep], k_rope[keep], nq, [139], False)
    F.close(lse, l, tl, "lse")
    F.close(out, o, to, "out")
    kv[:, 0, :128] = -float("inf")     # nothing left
    out, lse, _ = _run(q, kv, k_rope, nq, nk, False)
    assert (out == 0).all() and (lse == -float("inf")).all()
    kv2 = kv.clone()
    kv2[7, 0, 128] = float("nan")
    out, lse, _ = _run(q, kv2, k_rope, nq, nk, False)
    assert (out == 0).all() and (lse == -float("inf")).all()


def test_far_apart_maxima_and_first_steps_of_minus_infinity():
    # the first 256 keys give -inf, the others follow
    nq, nk, H = [200], [700], 2
    q, kv, k_rope = _inputs(nq, nk, H, 13)
    q[..., 0] = q[..., 0].abs() + 0.5
    kv[:256, :, 0] = -float("inf")
    out, lse, _ = _run(q, kv, k_rope, nq, nk, False)
    o, l, to, tl = F.attention(q, kv[256:], k_rope[256:], nq, [444], False)
    F.close(lse, l, tl, "lse")
    F.close(out, o, to, "out")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("slope", [0.02, 0.2, 3.0, -0.2])
def test_scores_that_grow_along_the_keys(slope, causal):
    # the rows' maxima are refreshed again and again, in one half of a step or in both, by some rows only
    nq, nk, H = [300, 5], [900, 700], 2
    q, kv, k_rope = _inputs(nq, nk, H, 21)
    q[..., 0] = torch.arange(305)[:, None] % 7 / F.SCALE / 4
    kv[..., 0] = (torch.arange(1600) * slope)[:, None]
    out, lse, status = _run(q, kv, k_rope, nq, nk, causal)
    assert status == 0
    o, l, to, tl = F.attention(q, kv, k_rope, nq, nk, causal)
    F.close(lse, l, tl, "lse")
    F.close(out, o, to, "out")


def test_large_values_scale_the_result():
    # a power of two is exact everywhere, before a maximum is refreshed and behind it
    nq, nk, H = [300], [900], 2
    q, kv, k_rope = _inputs(nq, nk, H, 23)
    q[..., 0] = 40.0
    kv[..., 0] = (torch.arange(900) * 0.05)[:, None]
    want = _run(q, kv, k_rope, nq, nk, True)
    kv[..., 128:] *= 2.0 ** 100
    got = _run(q, kv, k_rope, nq, nk, True)
    assert torch.equal(got[0], want[0] * 2.0 ** 100) and torch.equal(got[1], want[1])


def test_a_row_does_not_depend_on_its_neighbours():
    # rows whose maxima are refreshed at other steps, or are not numbers, in the same block
    nq, nk, H = [256], [1000], 1
    q, kv, k_rope = _inputs(nq, nk, H, 22)
    kv[..., 0] = (torch.arange(1000) * 0.1)[:, None]
    q[..., 0] = 0.0
    want = _run(q, kv, k_rope, nq, nk, False)
    q[::2, :, 0] = 40.0
    q[::16, :, 1] = float("nan")
    got = _run(q, kv, k_rope, nq, nk, False)
    assert torch.equal(got[0][1::2], want[0][1::2]) and torch.equal(got[1][1::2], want[1][1::2])
    assert not torch.equal(got[0][2::16], want[0][2::16]) and torch.isnan(got[0][::16]).all()


def test_bad_starts_are_reported_and_left_out():
    nq, nk, H = [4, 5, 6], [4, 5, 6], 2
    q, kv, k_rope = _inputs(nq, nk, H, 14)
    cu = F.starts(nk)
    for bad in ([0, 9, 4, 15], [0, 4, 99, 15], [0, -3, 9, 15]):
        out, lse, status = _run(q, kv, k_rope, nq, nk, True, cu_k=torch.tensor(bad, dtype=torch.int32))
        assert status == nsa.ERR_BOUNDS
    out, lse, status = _run(q, kv, k_rope, nq, nk, True, cu_k=torch.tensor([0, 4, 99, 15], dtype=torch.int32))
    o, l, to, tl = F.attention(q, kv, k_rope, nq, nk, True)
    F.close(out[:4], o[:4], to[:4], "out")
    assert (out[4:] == 7).all()
    assert cu[-1] == 15


def test_equal_calls_give_equal_bits_and_graphs_replay():
    nq, nk, H = [100, 3], [1500, 900], 2
    q, kv, k_rope = _inputs(nq, nk, H, 15)
    a = _run(q, kv, k_rope, nq, nk, True)
    b = _run(q, kv, k_rope, nq, nk, True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    d = "cuda"
    qd, kvd, rd, cq, ck = q.to(d), kv.to(d), k_rope.to(d), F.starts(nq).to(d), F.starts(nk).to(d)
    out, lse = torch.zeros((103, H, 128), dtype=F.BF, device=d), torch.zeros((103, H), device=d)
    ws = nsa.alloc_mla_prefill_workspace()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            nsa.nsa_mla_prefill(qd[..., :128], qd[..., 128:], kvd[..., :128], rd, kvd[..., 128:], cq, ck, True, F.SCALE, out, lse, ws)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), a[0]) and torch.equal(lse.cpu(), a[1])
    # other lengths of the same total in the same graph
    cq.copy_(F.starts([50, 53]))
    g.replay()
    torch.cuda.synchronize()
    o, l, to, tl = F.attention(q, kv, k_rope, [50, 53], nk, True)
    F.close(lse, l, tl, "lse")
    F.close(out, o, to, "out")


def test_on_another_stream_beside_another_call():
    nq, nk, H = [40], [2000], 3
    ins = [_inputs(nq, nk, H, 20 + i) for i in range(2)]
    want = [_run(*x, nq, nk, True)[:2] for x in ins]
    d = "cuda"
    cq, ck = F.starts(nq).to(d), F.starts(nk).to(d)
    dev = [tuple(t.to(d) for t in x) for x in ins]
    ws = [nsa.alloc_mla_prefill_workspace() for _ in range(2)]
    outs = [torch.empty((40, H, 128), dtype=F.BF, device=d) for _ in range(2)]
    lses = [torch.empty((40, H), device=d) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            q, kv, r = dev[i]
            nsa.nsa_mla_prefill(q[..., :128], q[..., 128:], kv[..., :128], r, kv[..., 128:], cq, ck, True, F.SCALE, outs[i],
                                lses[i], ws[i], stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i].cpu(), want[i][0]) and torch.equal(lses[i].cpu(), want[i][1])


def test_nothing_to_do():
    d = "cuda"
    z = lambda *s: torch.zeros(s, dtype=F.BF, device=d)
    ws, cu = nsa.alloc_mla_prefill_workspace(), torch.zeros(1, dtype=torch.int32, device=d)
    out, lse = torch.full((2, 2, 128), 7.0, dtype=F.BF, device=d), torch.full((2, 2), 7.0, device=d)
    nsa.nsa_mla_prefill(z(2, 2, 128), z(2, 2, 64), z(0, 2, 128), z(0, 64), z(0, 2, 128), cu, cu, True, 0.1, out, lse, ws)
    assert (out == 7).all() and (lse == 7).all()  # no request
    cq, ck = torch.tensor([0, 2], dtype=torch.int32, device=d), torch.tensor([0, 0], dtype=torch.int32, device=d)
    for causal in (True, False):
        nsa.nsa_mla_prefill(z(2, 2, 128), z(2, 2, 64), z(0, 2, 128), z(0, 64), z(0, 2, 128), cq, ck, causal, 0.1, out, lse, ws)
        assert (out == 0).all() and (lse == -float("inf")).all()  # no keys
        out.fill_(7), lse.fill_(7)
    nsa.nsa_mla_prefill(z(0, 2, 128), z(0, 2, 64), z(3, 2, 128), z(3, 64), z(3, 2, 128), ck, cq, True, 0.1, out[:0], lse[:0], ws)
