"""What the binding of the paged operators refuses, by the message it gives: every check of shapes, types and
strides comes before the one of devices, so tensors on the CPU reach it (no GPU, no launch)."""
import pytest
import torch

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def nsa():
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


z = lambda *s, d=F32: torch.zeros(s, dtype=d)
ON_CPU = "expected CUDA tensors on the current device"


def _args(**kw):
    q = z(4, 16, 576, d=BF)
    a = dict(q_dt=1, kv_dt=1, qn=q[..., :512], qr=q[..., 512:], kv=z(256, 576, d=BF), ps=64, pt=z(2, 2, d=I32), rl=z(4, d=I32), n=2,
             ml=128, scale=0.1, out=z(4, 16, 512, d=BF), lse=z(4, 16), ws=None, status=None, total=z(2, 128))
    a.update(kw)
    return a


def _attend(nsa, a):
    nsa.nsa_paged_mla(a["q_dt"], a["kv_dt"], a["qn"], a["qr"], a["kv"], a["ps"], a["pt"], a["rl"], a["n"], a["ml"], a["scale"],
                      a["out"], a["lse"], a["ws"], a["status"])


def _weigh(nsa, a):
    nsa.nsa_mla_key_weights(a["q_dt"], a["kv_dt"], a["qn"], a["qr"], a["kv"], a["ps"], a["pt"], a["rl"], a["n"], a["ml"], a["scale"],
                            a["lse"], a["total"], a["status"])


BOTH = {
    "nothing wrong": (dict(), ON_CPU),
    "rows of no whole requests": (dict(n=3), "4 rows are no whole requests of 3"),
    "no rows a request": (dict(n=0), "4 rows are no whole requests of 0"),
    "rope of other rows": (dict(qr=z(2, 16, 64, d=BF)), r"q_rope \(2, 16, 64\) does not match"),
    "rope of other heads": (dict(qr=z(4, 8, 64, d=BF)), r"q_rope \(4, 8, 64\) does not match"),
    "spread query elements": (dict(qn=z(4, 16, 1024, d=BF)[..., ::2]), "elements of each query head must be adjacent"),
    "spread rope elements": (dict(qr=z(4, 16, 128, d=BF)[..., ::2]), "elements of each query head must be adjacent"),
    "half rope": (dict(qr=z(4, 16, 64, d=torch.float16)), "q must be torch.bfloat16"),
    "narrow cache rows": (dict(kv=z(256, 500, d=BF)), "contiguous rows of 1152 bytes"),
    "cache rows of 4 dims": (dict(kv=z(2, 2, 64, 576, d=BF)), "contiguous rows of 1152 bytes"),
    "spread cache rows": (dict(kv=z(256, 1152, d=BF)[:, :576]), "contiguous rows of 1152 bytes"),
    "bf16 rows as fp8": (dict(kv_dt=2), "the cache must be torch.float8_e4m3fn"),
    "half cache": (dict(kv=z(256, 576, d=torch.float16)), "the cache must be torch.bfloat16"),
    "fp32 cache of as many bytes": (dict(kv=z(256, 288)), "the cache must be torch.bfloat16"),
    "e5m2 cache": (dict(kv_dt=2, kv=z(256, 656, d=torch.uint8).view(torch.float8_e5m2)), "the cache must be torch.float8_e4m3fn"),
    "part of a page": (dict(kv=z(250, 576, d=BF)), "250 slots are no whole pages of 64"),
    "no page size": (dict(ps=0), "256 slots are no whole pages of 0"),
    "64-bit table": (dict(pt=z(2, 2, d=torch.int64)), r"page_table must be int32 \[2, pages\]"),
    "table of another batch": (dict(pt=z(1, 2, d=I32)), r"page_table must be int32 \[2, pages\]"),
    "short table": (dict(ml=129), "a page-table row of 2 pages of 64 does not hold 129 positions"),
    "spread table": (dict(pt=z(2, 4, d=I32)[:, ::2]), "elements of each row must be adjacent"),
    "lengths of other rows": (dict(rl=z(3, d=I32)), "row_len must be 4 contiguous int32 values"),
    "64-bit lengths": (dict(rl=z(4, d=torch.int64)), "row_len must be 4 contiguous int32 values"),
    "spread lengths": (dict(rl=z(8, d=I32)[::2]), "row_len must be 4 contiguous int32 values"),
    "lengths in two dims": (dict(rl=z(4, 1, d=I32)), "row_len must be 4 contiguous int32 values"),
    "64-bit lse": (dict(lse=z(4, 16, d=torch.float64)), "lse"),
    "byte status": (dict(status=z(4, d=torch.uint8)), "status must be an int32 word"),
    "empty status": (dict(status=z(0, d=I32)), "status must be an int32 word"),
}
ATTEND = {
    "fp32 out": (dict(out=z(4, 16, 512)), "out must be"),
    "spread out": (dict(out=z(4, 16, 1024, d=BF)[..., ::2]), "out must be"),
    "out of other heads": (dict(out=z(4, 8, 512, d=BF)), "out must be"),
    "half q and out": (dict(qn=z(4, 16, 512, d=torch.float16), out=z(4, 16, 512, d=torch.float16)), "q must be torch.bfloat16"),
    "spread workspace": (dict(ws=z(64, d=torch.uint8)[::2]), "the workspace must be contiguous"),
    "broadcast workspace": (dict(ws=z(1, d=torch.uint8).expand(1 << 20)), "the workspace must be contiguous"),
}
WEIGH = {
    "short totals": (dict(total=z(2, 127)), r"total must be float32 \[2, >= 128\]"),
    "totals of another batch": (dict(total=z(3, 128)), r"total must be float32 \[2, >= 128\]"),
    "64-bit totals": (dict(total=z(2, 128, d=torch.float64)), r"total must be float32 \[2, >= 128\]"),
    "spread totals": (dict(total=z(2, 256)[:, ::2]), "elements of each row must be adjacent"),
    "half q": (dict(qn=z(4, 16, 512, d=torch.float16)), "q must be torch.bfloat16"),
}


@pytest.mark.parametrize("name", [*BOTH, *ATTEND])
def test_attention(nsa, name):
    change, message = {**BOTH, **ATTEND}[name]
    with pytest.raises(ValueError, match=message):
        _attend(nsa, _args(**change))


@pytest.mark.parametrize("name", [*BOTH, *WEIGH])
def test_weights(nsa, name):
    change, message = {**BOTH, **WEIGH}[name]
    with pytest.raises(ValueError, match=message):
        _weigh(nsa, _args(**change))


@pytest.mark.parametrize("kv_dt,kv", [(1, z(256, 1152, d=torch.uint8)), (1, z(256, 576, d=torch.int16)), (2, z(256, 656, d=torch.uint8)),
                                      (2, z(256, 656, d=torch.int8)), (2, z(4, 64, 656, d=torch.uint8)),
                                      (2, z(256, 656, d=torch.uint8).view(torch.float8_e4m3fn))])
def test_a_cache_of_bytes_is_taken(nsa, kv_dt, kv):
    for call in (_attend, _weigh):
        with pytest.raises(ValueError, match=ON_CPU):  # nothing but the device is wrong
            call(nsa, _args(kv_dt=kv_dt, kv=kv))


@pytest.mark.parametrize("change,message", [
    (dict(), ON_CPU),
    (dict(keep=z(2, 9, d=I32)), r"keep must be int32 \[2, >= 10\]"),
    (dict(keep=z(3, 10, d=I32)), r"keep must be int32 \[2, >= 10\]"),
    (dict(keep=z(2, 10, d=torch.int64)), r"keep must be int32 \[2, >= 10\]"),
    (dict(keep=z(2, 20, d=I32)[:, ::2]), "elements of each row must be adjacent"),
    (dict(total=z(2, 127)), r"total must be float32 \[2, >= 128\]"),
    (dict(total=z(2, 128, d=BF)), r"total must be float32 \[2, >= 128\]"),
    (dict(lens=z(2, d=torch.int64)), "lens must be 2 contiguous int32 values"),
    (dict(lens=z(4, d=I32)[::2]), "lens must be 2 contiguous int32 values"),
    (dict(new=z(3, d=I32)), "new_len must be 2 contiguous int32 values"),
    (dict(status=z(1)), "status must be an int32 word"),
])
def test_select(nsa, change, message):
    a = dict(total=z(2, 128), lens=z(2, d=I32), keep=z(2, 10, d=I32), new=z(2, d=I32), status=None)
    a.update(change)
    with pytest.raises(ValueError, match=message):
        nsa.nsa_evict_select(a["total"], a["lens"], 128, 0, 0, 10, a["keep"], a["new"], a["status"])


@pytest.mark.parametrize("change,message", [
    (dict(), ON_CPU),
    (dict(total=None), ON_CPU),
    (dict(arrays=[]), ON_CPU),
    (dict(keep=z(3, 10, d=I32)), r"keep must be int32 \[2, budget\]"),
    (dict(keep=z(2, 10, d=torch.int64)), r"keep must be int32 \[2, budget\]"),
    (dict(keep=z(2, 20, d=I32)[:, ::2]), "elements of each row must be adjacent"),
    (dict(new=z(3, d=I32)), "new_len must be 2 contiguous int32 values"),
    (dict(new=z(2, d=torch.int64)), "new_len must be 2 contiguous int32 values"),
    (dict(old=z(4, d=I32)[::2]), "old_len must be 2 contiguous int32 values"),
    (dict(pt=z(1, 2, d=I32)), r"page_table must be int32 \[2, pages\]"),
    (dict(pt=z(2, 1, d=I32)), "a page-table row of 1 pages of 64 does not hold 128 positions"),
    (dict(ps=0), "page_size must be positive, got 0"),
    (dict(ps=-64), "page_size must be positive, got -64"),
    (dict(ps=48), "one first dimension of whole pages of 48"),
    (dict(arrays=[z(250, 4)]), "one first dimension of whole pages of 64"),
    (dict(arrays=[z(256, 8)[:, :4]]), "the arrays must be contiguous"),
    (dict(arrays=[z(256, 4), z(192)]), "one first dimension of whole pages of 64"),
    (dict(arrays=[z(0, 4)]), "one first dimension of whole pages of 64"),
    (dict(total=z(2, 127)), r"total must be float32 \[2, >= 128\]"),
    (dict(ws=z(1, d=torch.uint8).expand(4096)), "the workspace must be contiguous"),
    (dict(status=z(1, d=torch.int64)), "status must be an int32 word"),
])
def test_compact(nsa, change, message):
    a = dict(keep=z(2, 10, d=I32), new=z(2, d=I32), old=z(2, d=I32), pt=z(2, 2, d=I32), ps=64, arrays=[z(256, 4)], total=z(2, 128),
             ws=z(4096, d=torch.uint8), status=None)
    a.update(change)
    with pytest.raises(ValueError, match=message):
        nsa.nsa_evict_compact(a["keep"], a["new"], a["old"], 128, a["pt"], a["ps"], a["arrays"], a["total"], a["ws"], a["status"])
