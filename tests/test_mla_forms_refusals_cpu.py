"""What the calls of latent attention's two forms refuse: the binding by its message (every check of shapes, types and
strides comes before the one of devices), the library by its status, before anything is launched."""
import ctypes as C

import pytest
import torch

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
ON_CPU = "expected CUDA tensors on the current device"
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def nsa():
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


z = lambda *s, d=BF: torch.zeros(s, dtype=d)


def _prefill(**kw):
    q, kv = z(6, 4, 192), z(9, 4, 256)
    a = dict(qn=q[..., :128], qr=q[..., 128:], kn=kv[..., :128], kr=z(9, 64), v=kv[..., 128:], cq=z(3, d=I32), ck=z(3, d=I32),
             out=z(6, 4, 128), lse=z(6, 4, d=F32), ws=z(64, d=torch.uint8), status=None)
    a.update(kw)
    return a


PREFILL = {
    "nothing wrong": (dict(), ON_CPU),
    "half queries": (dict(qn=z(6, 4, 128, d=torch.float16)), "q_nope must be bf16"),
    "narrow queries": (dict(qn=z(6, 4, 64)), r"q_nope must be bf16 \[any, any, 128\]"),
    "flat queries": (dict(qn=z(6, 512)), "q_nope must be bf16"),
    "rope of other rows": (dict(qr=z(5, 4, 64)), r"q_rope must be bf16 \[6, 4, 64\]"),
    "rope of other heads": (dict(qr=z(6, 1, 64)), r"q_rope must be bf16 \[6, 4, 64\]"),
    "spread queries": (dict(qn=z(6, 4, 256)[..., ::2]), "last dimension adjacent"),
    "keys of other heads": (dict(kn=z(9, 2, 128)), r"k_nope must be bf16 \[9, 4, 128\]"),
    "keys of other rows": (dict(kn=z(8, 4, 128)), r"k_nope must be bf16 \[9, 4, 128\]"),
    "rope keys a head": (dict(kr=z(9, 4, 64)), r"k_rope must be bf16 \[any, 64\]"),
    "wide values": (dict(v=z(9, 4, 256)), r"v must be bf16 \[9, 4, 128\]"),
    "fp32 values": (dict(v=z(9, 4, 128, d=F32)), "v must be bf16"),
    "64-bit starts": (dict(cq=z(3, d=torch.int64)), "cu_seqlens_q must be 3 contiguous int32"),
    "starts of another batch": (dict(ck=z(4, d=I32)), "cu_seqlens_k must be 3 contiguous int32"),
    "no starts": (dict(cq=z(0, d=I32)), "cu_seqlens_q must be 1 contiguous int32"),
    "fp32 out": (dict(out=z(6, 4, 128, d=F32)), "out must be bf16"),
    "strided out": (dict(out=z(6, 4, 256)[..., :128]), "out must be bf16"),
    "short lse": (dict(lse=z(6, 3, d=F32)), r"lse must be contiguous float32 \[6, 4\]"),
    "bf16 lse": (dict(lse=z(6, 4)), r"lse must be contiguous float32 \[6, 4\]"),
    "spread workspace": (dict(ws=z(64, d=torch.uint8)[::2]), "the workspace must be contiguous"),
    "64-bit status": (dict(status=z(1, d=torch.int64)), "status must be an int32 word"),
}


@pytest.mark.parametrize("name", PREFILL)
def test_prefill(nsa, name):
    kw, msg = PREFILL[name]
    a = _prefill(**kw)
    with pytest.raises(ValueError, match=msg):
        nsa.nsa_mla_prefill(a["qn"], a["qr"], a["kn"], a["kr"], a["v"], a["cq"], a["ck"], True, 0.1, a["out"], a["lse"], a["ws"], a["status"])


EXPAND = {
    "nothing wrong": (dict(), ON_CPU),
    "weight of no whole heads": (dict(w=z(300, 512)), r"w must be bf16 \[heads \* 256, 512\]"),
    "no heads": (dict(w=z(0, 512)), r"w must be bf16 \[heads \* 256, 512\]"),
    "narrow weight": (dict(w=z(512, 500)), r"w must be bf16 \[any, 512\]"),
    "strided weight": (dict(w=z(512, 1024)[:, :512]), "w must be bf16"),
    "fp32 weight": (dict(w=z(512, 512, d=F32)), "w must be bf16"),
    "64-bit slots": (dict(slots=z(7, d=torch.int64)), "slots must be 7 contiguous int32"),
    "table of slots": (dict(slots=z(7, 1, d=I32)), "slots must be 7 contiguous int32"),
    "other rows out": (dict(out=z(6, 2, 256)), r"kv_out must be bf16 \[7, 2, 256\]"),
    "other heads out": (dict(out=z(7, 1, 256)), r"kv_out must be bf16 \[7, 2, 256\]"),
    "spread rope out": (dict(rope=z(7, 128)[:, :64]), r"k_rope_out must be bf16 \[7, 64\]"),
    "narrow cache rows": (dict(kv=z(50, 575)), "contiguous rows of 1152 bytes"),
    "bf16 rows as fp8": (dict(dt=2), "the cache must be torch.float8_e4m3fn"),
    "64-bit status": (dict(status=z(1, d=torch.int64)), "status must be an int32 word"),
}


@pytest.mark.parametrize("name", EXPAND)
def test_expand(nsa, name):
    a = dict(dt=1, kv=z(50, 576), slots=z(7, d=I32), w=z(512, 512), out=z(7, 2, 256), rope=z(7, 64), ws=z(16, d=torch.uint8), status=None)
    kw, msg = EXPAND[name]
    a.update(kw)
    with pytest.raises(ValueError, match=msg):
        nsa.nsa_mla_expand_kv(a["dt"], a["kv"], a["slots"], a["w"], a["out"], a["rope"], a["ws"], a["status"])


HEADS = {
    "nothing wrong": (dict(), ON_CPU),
    "other heads": (dict(x=lambda K: z(5, 3, K)), r"must be bf16 \[any, 2, "),
    "other width": (dict(x=lambda K: z(5, 2, K - 8)), r"must be bf16 \[any, 2, "),
    "spread": (dict(x=lambda K: z(5, 2, 2 * K)[..., ::2]), "last dimension adjacent"),
    "fp32": (dict(x=lambda K: z(5, 2, K, d=F32)), "must be bf16"),
    "no rows' dimension": (dict(x=lambda K: z(2, K)), "must be bf16"),
    "strided out": (dict(out=lambda F: z(5, 2, 2 * F)[..., :F]), "out must be bf16"),
    "out of other rows": (dict(out=lambda F: z(4, 2, F)), "out must be bf16"),
    "weight of no whole heads": (dict(w=z(257, 512)), "heads"),
}


@pytest.mark.parametrize("name", HEADS)
@pytest.mark.parametrize("op", ["absorb", "project"])
def test_head_products(nsa, op, name):
    K, F = (128, 512) if op == "absorb" else (512, 128)
    a = dict(x=lambda K: z(5, 2, K), w=z(512, 512), out=lambda F: z(5, 2, F))
    kw, msg = HEADS[name]
    a.update(kw)
    call = nsa.nsa_mla_absorb_q if op == "absorb" else nsa.nsa_mla_project_v
    with pytest.raises(ValueError, match=msg):
        call(a["x"](K), a["w"], a["out"](F))


def test_merge(nsa):
    p, l = z(4, 16), z(4, d=F32)

    def refused(msg, parts, lses, out, lse):
        with pytest.raises(ValueError, match=msg):
            nsa.nsa_merge_attention(parts, lses, out, lse)

    refused(ON_CPU, [p, p], [l, l], z(4, 16), z(4, d=F32))
    refused("at least one", [], [], p, l)
    refused("as many lse as parts", [p, p], [l], p, l)
    refused("float32 or bf16", [p.half()], [l], p, l)
    refused("float32 or bf16", [p], [l], p.half(), l)
    refused("parts must be contiguous", [p, p.float()], [l, l], p, l)
    refused("parts must be contiguous", [p, z(4, 8)], [l, l], p, l)
    refused("parts must be contiguous", [p], [l], z(5, 16), l)
    refused("parts must be contiguous", [p], [z(5, d=F32)], p, l)
    refused("parts must be contiguous", [p], [l.double()], p, l)
    refused("parts must be contiguous", [p], [l], z(4, 32)[:, :16], l)
    refused("parts must be contiguous", [p], [l], p, z(8, d=F32)[::2])


# ------------------------------------------------------------------ the library's own checks: pointers that are never followed

A = 1 << 20  # a 16-byte aligned address


def _status(nsa, fn, args):
    return getattr(nsa.load(), fn)(*args)


def test_prefill_abi(nsa):
    names = ["qn", "qn_r", "qn_h", "qr", "qr_r", "qr_h", "kn", "kn_r", "kn_h", "kr", "kr_r", "v", "v_r", "v_h", "cq", "ck", "B", "tq",
             "tk", "H", "dn", "dr", "dv", "causal", "scale", "out", "lse", "ws", "wsb", "status", "stream"]
    good = dict(qn=A, qn_r=768, qn_h=192, qr=A, qr_r=768, qr_h=192, kn=A, kn_r=1024, kn_h=256, kr=A, kr_r=64, v=A, v_r=1024, v_h=256,
                cq=A, ck=A, B=2, tq=6, tk=9, H=4, dn=128, dr=64, dv=128, causal=1, scale=0.1, out=A, lse=A, ws=A, wsb=0, status=0, stream=0)

    def call(**kw):
        a = dict(good, **kw)
        return _status(nsa, "nsa_mla_prefill", [a[n] for n in names])

    for kw in (dict(B=-1), dict(tq=-1), dict(tk=-1), dict(H=0), dict(causal=2), dict(causal=-1), dict(scale=0.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(scale=-1.0), dict(qn=0), dict(qr=0), dict(kn=0), dict(kr=0), dict(v=0), dict(cq=0), dict(ck=0),
               dict(out=0), dict(lse=0), dict(ws=0), dict(qn=A + 2), dict(kr=A + 8), dict(v=A + 8), dict(out=A + 4), dict(ws=A + 8),
               dict(cq=A + 2), dict(lse=A + 2), dict(status=A + 1), dict(qn_h=120), dict(qn_h=132), dict(kn_r=1020), dict(kr_r=56),
               dict(v_h=0), dict(qr_r=-768), dict(kn_h=0)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dn=64), dict(dr=32), dict(dv=256), dict(H=65536), dict(tk=(1 << 30) + 1), dict(tq=(1 << 30) + 1), dict(kn_r=1 << 39)):
        assert call(**kw) == UNSUPPORTED, kw
    # nothing to do
    assert call(B=0) == 0 and call(tq=0) == 0


def test_expand_abi(nsa):
    names = ["dt", "kv", "slots_n", "slots", "m", "w", "H", "dl", "dr", "dn", "dv", "out", "rope", "ws", "wsb", "status", "stream"]
    good = dict(dt=1, kv=A, slots_n=64, slots=A, m=7, w=A, H=2, dl=512, dr=64, dn=128, dv=128, out=A, rope=A, ws=A, wsb=7 * 1024, status=0, stream=0)

    def call(**kw):
        a = dict(good, **kw)
        return _status(nsa, "nsa_mla_expand_kv", [a[n] for n in names])

    for kw in (dict(m=-1), dict(H=0), dict(slots_n=-1), dict(slots_n=0), dict(kv=0), dict(slots=0), dict(w=0), dict(out=0), dict(rope=0),
               dict(ws=0), dict(wsb=7 * 1024 - 1), dict(kv=A + 8), dict(w=A + 2), dict(out=A + 8), dict(rope=A + 8), dict(ws=A + 8),
               dict(slots=A + 2), dict(status=A + 2)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dt=0), dict(dt=3), dict(dl=256), dict(dr=32), dict(dn=64), dict(dv=64), dict(H=65536)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(m=0) == 0
    size = nsa.nsa_mla_expand_kv_workspace_bytes
    assert size(0) == 0 and size(7) <= 7 * 1024 and size(8) >= size(7)


@pytest.mark.parametrize("fn,ld", [("nsa_mla_absorb_q", 128), ("nsa_mla_project_v", 512)])
def test_head_products_abi(nsa, fn, ld):
    names = ["x", "ld_r", "ld_h", "w", "R", "H", "dn", "dv", "dl", "out", "status", "stream"]
    good = dict(x=A, ld_r=2 * ld, ld_h=ld, w=A, R=5, H=2, dn=128, dv=128, dl=512, out=A, status=0, stream=0)

    def call(**kw):
        a = dict(good, **kw)
        return _status(nsa, fn, [a[n] for n in names])

    for kw in (dict(R=-1), dict(H=0), dict(x=0), dict(w=0), dict(out=0), dict(x=A + 8), dict(w=A + 8), dict(out=A + 8), dict(status=A + 2),
               dict(ld_h=ld - 8), dict(ld_h=ld + 4), dict(ld_r=ld - 8), dict(ld_r=2 * ld + 2), dict(ld_h=0), dict(ld_r=-ld)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dn=64), dict(dv=64), dict(dl=256), dict(H=65536), dict(ld_r=1 << 39)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(R=0) == 0


def test_merge_abi(nsa):
    two = (C.c_void_p * 9)(*[A] * 9)

    def call(dt=1, odt=1, n=2, parts=two, lses=two, rows=4, D=16, out=A, lse=A):
        return _status(nsa, "nsa_merge_attention", [dt, odt, n, parts, lses, rows, D, out, lse, 0])

    for kw in (dict(n=0), dict(rows=-1), dict(D=0), dict(parts=None), dict(lses=None), dict(out=0), dict(lse=0), dict(out=A + 8),
               dict(lse=A + 2), dict(parts=(C.c_void_p * 2)(A, 0)), dict(lses=(C.c_void_p * 2)(A, A + 2)), dict(parts=(C.c_void_p * 2)(A, A + 4))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dt=2), dict(dt=1, odt=0), dict(dt=0, odt=2), dict(n=9), dict(D=12), dict(D=2056)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(rows=0) == 0


def test_rows_past_32_bit_coordinates(nsa):
    big = (1 << 30) + 1
    expand = [1, A, 64, A, big, A, 2, 512, 64, 128, 128, A, A, A, big * 1024, 0, 0]
    assert _status(nsa, "nsa_mla_expand_kv", expand) == UNSUPPORTED
    for fn, ld in ("nsa_mla_absorb_q", 128), ("nsa_mla_project_v", 512):
        assert _status(nsa, fn, [A, 2 * ld, ld, A, big, 2, 128, 128, 512, A, 0, 0]) == UNSUPPORTED


def test_merge_of_a_part_of_another_type_that_is_the_result(nsa):
    a, b, l = z(4, 16, d=F32), z(4, 16), z(4, d=F32)
    with pytest.raises(ValueError, match="parts must be contiguous"):
        nsa.nsa_merge_attention([a, b], [l, l], b, l)
    with pytest.raises(ValueError, match="parts must be contiguous"):
        nsa.nsa_merge_attention([z(d=F32)], [l], z(d=F32), l)


@pytest.mark.parametrize("fn,ld", [("nsa_mla_absorb_q", 128), ("nsa_mla_project_v", 512)])
def test_the_stride_of_a_single_row_or_head_is_not_looked_at(nsa, fn, ld):
    if torch.cuda.is_available():
        pytest.skip("the addresses are none; without a GPU a call that nothing refuses ends where it asks for the device")
    for far in (1 << 39, 1 << 62, -8, 0, 3):
        for R, H, ld_r, ld_h in ((5, 1, ld, far), (1, 2, far, ld), (1, 1, far, far)):
            got = _status(nsa, fn, [A, ld_r, ld_h, A, R, H, 128, 128, 512, A, 0, 0])
            assert got not in (0, INVALID, UNSUPPORTED), (R, H, far)


def test_the_version_tells_a_library_with_these_calls(nsa):
    assert nsa.nsa_abi_version() >= 104
