"""nsa_paged_mla and nsa_mla_key_weights at the widest cache rows that they take, where few heads fit in shared
memory at a time.  Both calls take the same dims.

Tolerances: fp32 sums of dq products, each addition off by at most half a step (2^-24) of a partial sum that
sum|q k| bounds, as in test_gpu_paged_mla with dq + 1 in the place of 577."""
import pytest
import torch

from tests._paged import SCALE, Problem
from tests.test_gpu_paged_mla import _run, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def nsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


DIMS = [("f32", 1687, 64, 17), ("f32", 1751, 0, 1), ("f32", 1, 1750, 2), ("f32", 1100, 36, 20), ("bf16", 1536, 64, 16),
        ("bf16", 1200, 551, 5), ("fp8", 1664, 64, 16), ("fp8", 1152, 64, 3), ("f32", 1, 0, 1)]


def _err(p, r):
    if not int(p.row_len[r]):
        return 0.0
    return float((p.q[r].double().abs() @ p.values(r).abs().T).max()) * SCALE * (p.dl + p.dr + 1) * 2.0 ** -24


@pytest.mark.parametrize("kv,dl,dr,H", DIMS)
def test_attention(nsa, kv, dl, dr, H):
    p = Problem([40, 0, 1, 33], H=H, kv=kv, ps=4, dl=dl, dr=dr, seed=5)
    out, lse, code = _run(nsa, p)
    assert code == 0
    eo, el = p.attention()
    out, lse = out.double().cpu(), lse.double().cpu()
    for r in range(p.R):
        if int(p.row_len[r]) == 0:
            assert not out[r].any() and torch.isneginf(lse[r]).all()
            continue
        e = _err(p, r)
        x, k = p.scores(r)
        spread = torch.exp(x - el[r][:, None]) @ k[:, :dl].abs()
        assert ((lse[r] - el[r]).abs() <= 2 * e + 2.0 ** -22 * (2 + el[r].abs())).all()
        half = 2.0 ** -8 * eo[r].abs() if p.q_dt else 0.0  # the result's rounding to bf16
        assert ((out[r] - eo[r]).abs() <= (2.0 ** -18 + 4 * e) * spread + half + 2.0 ** -20).all()


@pytest.mark.parametrize("kv,dl,dr,H", DIMS)
def test_weights(nsa, kv, dl, dr, H):
    p = Problem([40, 0, 1, 33], H=H, kv=kv, ps=4, dl=dl, dr=dr, seed=5)
    lse = p.attention()[1].float()
    total = torch.zeros((p.B, p.max_len), device="cuda")
    assert _weights(nsa, p, lse, total) == 0
    w = p.weights(lse)
    rel = 2 * max(_err(p, r) for r in range(p.R)) + 64 * 2.0 ** -23 + (p.n * p.H + 8) * 2.0 ** -24
    assert ((total.double().cpu() - w).abs() <= rel * w + 1e-30).all()


@pytest.mark.parametrize("kv,dl,dr", [("f32", 1688, 64), ("bf16", 8192, 64), ("fp8", 1792, 64), ("f32", 2 ** 20, 1)])
def test_wider_rows_are_refused_by_both(nsa, kv, dl, dr):
    dt, kdt = (0, 0) if kv == "f32" else (1, 1 if kv == "bf16" else 2)
    t = torch.float32 if kv == "f32" else torch.bfloat16
    z = lambda *s, d=t: torch.zeros(s, dtype=d, device="cuda")
    kvt = z(4, dl + 4 * (dl // 128) + 2 * dr, d=torch.uint8) if kv == "fp8" else z(4, dl + dr)
    i32 = dict(dtype=torch.int32, device="cuda")
    args = (dt, kdt, z(1, 1, dl), z(1, 1, dr), kvt, 4, torch.zeros((1, 1), **i32), torch.ones(1, **i32), 1, 4, SCALE)
    for call in (lambda: nsa.nsa_paged_mla(*args, z(1, 1, dl), z(1, 1, d=torch.float32)),
                 lambda: nsa.nsa_mla_key_weights(*args, z(1, 1, d=torch.float32), z(1, 4, d=torch.float32))):
        with pytest.raises(nsa.NsaError) as e:
            call()
        assert e.value.code == nsa.ERR_UNSUPPORTED
