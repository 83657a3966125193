"""Host-side checks of the dense paged attention and the eviction calls, on a machine
without a GPU: the addresses are never dereferenced, every refusal comes before a launch."""
import ctypes as C

import pytest
import torch


@pytest.fixture(scope="module")
def nsa():
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


P = lambda x: C.c_void_p(x) if x else None


def _paged(nsa, weights=False, **kw):
    a = dict(qdt=1, kdt=1, qn=0x10000, nr=16 * 576, nh=576, qr=0x20000, rr=16 * 576, rh=576, kv=0x30000, pages=9, ps=64,
             pt=0x40000, pt_ld=4, rl=0x50000, R=4, n=2, H=16, dl=512, dr=64, ml=256, scale=0.1, out=0x60000, lse=0x70000,
             total=0x80000, total_ld=256, ws=0, wsb=0, status=0)
    a.update(kw)
    lib = nsa.load()
    head = [a["qdt"], a["kdt"], P(a["qn"]), a["nr"], a["nh"], P(a["qr"]), a["rr"], a["rh"], P(a["kv"]), a["pages"], a["ps"],
            P(a["pt"]), a["pt_ld"], P(a["rl"]), a["R"], a["n"], a["H"], a["dl"], a["dr"], a["ml"], C.c_float(a["scale"])]
    if weights:
        return lib.nsa_mla_key_weights(*head, P(a["lse"]), P(a["total"]), a["total_ld"], P(a["status"]), None)
    return lib.nsa_paged_mla(*head, P(a["out"]), P(a["lse"]), P(a["ws"]), a["wsb"], P(a["status"]), None)


@pytest.mark.parametrize("weights", [False, True])
def test_paged_attention_host_checks(nsa, weights):
    inval, unsup = nsa.ERR_INVALID_ARG, nsa.ERR_UNSUPPORTED
    call = lambda **kw: _paged(nsa, weights, **kw)
    assert call(R=0) == 0                          # nothing to do
    assert call(R=-2) == inval
    assert call(R=3) == inval                      # no whole requests
    assert call(n=0) == inval
    assert call(H=0) == inval
    assert call(ps=0) == inval
    assert call(pt_ld=3) == inval                  # 256 positions need 4 pages of 64
    assert call(ml=-1) == inval
    assert call(scale=0.0) == inval
    assert call(scale=float("nan")) == inval
    assert call(scale=float("inf")) == inval
    assert call(qdt=1, kdt=0) == unsup             # bf16 queries over an fp32 cache
    assert call(qdt=0, kdt=1) == unsup
    assert call(qdt=2, kdt=2) == unsup
    assert call(kdt=2, dl=500) == unsup            # no whole scale blocks
    assert call(kdt=2, dr=63) == unsup
    assert call(pages=2 ** 40) == unsup            # slots beyond 32 bits
    assert call(ml=2 ** 30 + 64, pt_ld=2 ** 25) == unsup
    assert call(pages=0) == inval
    for name in ("qn", "qr", "kv", "pt", "rl", "lse"):
        assert call(**{name: 0}) == inval, name    # NULL
    assert call(qn=0x10001) == inval               # misaligned
    assert call(kv=0x30001) == inval
    assert call(pt=0x40002) == inval
    assert call(lse=0x70002) == inval
    assert call(status=0x90001) == inval
    if weights:
        assert call(total=0) == inval
        assert call(total_ld=255) == inval
        assert call(ml=0, pt=0) == 0               # no positions: nothing to add
    else:
        assert call(out=0) == inval
        assert call(out=0x60001) == inval


def test_paged_attention_workspace(nsa):
    need = nsa.nsa_paged_mla_workspace_bytes(1, 1, 4, 2, 16, 256)
    if need:
        assert _paged(nsa, ws=0, wsb=0) == nsa.ERR_INVALID_ARG
        assert _paged(nsa, ws=0x100000, wsb=need - 1) == nsa.ERR_INVALID_ARG
        assert _paged(nsa, ws=0x100008, wsb=need) == nsa.ERR_INVALID_ARG  # not 16-byte aligned
    assert nsa.nsa_paged_mla_workspace_bytes(1, 1, 0, 1, 16, 256) == 0
    assert nsa.nsa_paged_mla_workspace_bytes(0, 0, 4, 1, 16, 256) == 0    # the fp32 kernel joins nothing


def test_evict_select_host_checks(nsa):
    lib, inval = nsa.load(), nsa.ERR_INVALID_ARG

    def call(**kw):
        a = dict(t=0x10000, ld=100, lens=0x20000, B=2, ml=100, sinks=2, recent=3, budget=10, keep=0x30000, kld=10, new=0x40000)
        a.update(kw)
        return lib.nsa_evict_select(P(a["t"]), a["ld"], P(a["lens"]), a["B"], a["ml"], a["sinks"], a["recent"], a["budget"],
                                    P(a["keep"]), a["kld"], P(a["new"]), None, None)

    assert call(B=0) == 0
    assert call(B=-1) == inval
    assert call(ld=99) == inval
    assert call(kld=9) == inval
    assert call(budget=0) == inval
    assert call(sinks=8) == inval            # sinks + recent beyond the budget
    assert call(sinks=2 ** 30, recent=2 ** 30, budget=2 ** 30, kld=2 ** 30) == inval
    assert call(sinks=-1) == inval
    assert call(recent=-1) == inval
    assert call(ml=2 ** 30 + 1, ld=2 ** 31) == nsa.ERR_UNSUPPORTED
    for name in ("t", "lens", "keep", "new"):
        assert call(**{name: 0}) == inval
        assert call(**{name: 0x10002}) == inval


def test_evict_compact_host_checks(nsa):
    lib, inval, unsup = nsa.load(), nsa.ERR_INVALID_ARG, nsa.ERR_UNSUPPORTED

    def call(arrays=(0x100000,), rows=(656,), **kw):
        a = dict(B=2, keep=0x10000, kld=10, budget=10, new=0x20000, old=0x30000, ml=100, pt=0x40000, pt_ld=7, ps=16, pages=20,
                 total=0x50000, tld=100, ws=0x60000, wsb=1 << 20)
        a.update(kw)
        n = len(arrays)
        ptrs = (C.c_void_p * max(1, n))(*arrays)
        nb = (C.c_int64 * max(1, n))(*rows)
        return lib.nsa_evict_compact(a["B"], P(a["keep"]), a["kld"], a["budget"], P(a["new"]), P(a["old"]), a["ml"], P(a["pt"]),
                                     a["pt_ld"], a["ps"], a["pages"], n, ptrs, nb, P(a["total"]), a["tld"], P(a["ws"]), a["wsb"],
                                     None, None)

    assert call(B=0) == 0
    assert call(ml=0) == 0
    assert call(arrays=(), rows=(), total=0) == 0     # nothing to move
    assert call(B=-1) == inval
    assert call(kld=9) == inval                       # rows shorter than the budget
    assert call(pt_ld=6) == inval                     # 100 positions need 7 pages of 16
    assert call(ps=0) == inval
    assert call(tld=99) == inval
    assert call(rows=(0,)) == inval
    assert call(arrays=(None,)) == inval
    assert call(arrays=(0x100000,) * 9, rows=(16,) * 9) == inval
    assert call(rows=(24 * 1024 + 16,)) == unsup
    assert call(arrays=(0x100000, 0x900000), rows=(13 * 1024, 12 * 1024)) == unsup
    assert call(pages=2 ** 40) == unsup
    assert call(pages=0) == inval
    assert call(wsb=15) == inval
    assert call(ws=0) == inval
    assert call(ws=0x60008) == inval
    for name in ("keep", "new", "old", "pt"):
        assert call(**{name: 0}) == inval
        assert call(**{name: 0x10002}) == inval


def test_binding_refuses_what_the_library_would_misread(nsa):
    """Shapes, types and devices, before any call into the library."""
    bf, i32 = torch.bfloat16, torch.int32
    q = torch.zeros((4, 16, 576), dtype=bf)
    kv = torch.zeros((4 * 64, 576), dtype=bf)
    pt, rl = torch.zeros((2, 2), dtype=i32), torch.zeros(4, dtype=i32)
    out, lse = torch.zeros((4, 16, 512), dtype=bf), torch.zeros((4, 16))
    total = torch.zeros((2, 128))

    def attn(q=q, kv=kv, ps=64, pt=pt, rl=rl, n=2, ml=128, out=out, lse=lse, kdt=1):
        nsa.nsa_paged_mla(1, kdt, q[..., :512], q[..., 512:], kv, ps, pt, rl, n, ml, 0.1, out, lse)

    for kw in (dict(), dict(n=3), dict(kv=kv[:, :500]), dict(kv=kv[:250]), dict(pt=pt.long()), dict(pt=pt[:1]), dict(ml=129),
               dict(rl=rl[:3]), dict(rl=rl.long()), dict(out=out.float()), dict(out=out[:, :, ::2]), dict(lse=lse.double()),
               dict(q=q.half()), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), dict(kdt=2), dict(ps=0)):
        with pytest.raises(ValueError):  # the first one for its tensors being on the CPU
            attn(**kw)
    with pytest.raises(ValueError):
        nsa.nsa_mla_key_weights(1, 1, q[..., :512], q[..., 512:], kv, 64, pt, rl, 2, 128, 0.1, lse, total[:, :100])
    with pytest.raises(ValueError):
        nsa.nsa_evict_select(total, rl[:2], 128, 0, 0, 10, torch.zeros((2, 9), dtype=i32), rl[:2])
    for arrays in ([kv], [kv[:250]], [kv[:, :64]], [kv, torch.zeros(255)]):
        with pytest.raises(ValueError):
            nsa.nsa_evict_compact(torch.zeros((2, 10), dtype=i32), rl[:2], rl[:2], 128, pt, 64, arrays, total,
                                  torch.zeros(1 << 16, dtype=torch.uint8))
