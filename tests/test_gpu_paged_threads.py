"""The CUDA-core forms called by two host threads at once, with shapes that need different amounts of shared
memory: every call launches and gives what it gives alone."""
import ctypes as C
import functools
import threading

import pytest
import torch

from tests._paged import SCALE, Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def nsa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deepseek_sparse_mla_indexer_gb300 as m
    m.load()
    return m


CALLS = 4000


@pytest.mark.parametrize("op", ["attention", "weights"])
def test_two_host_threads(nsa, op):
    jobs = []
    for i, shape in enumerate((dict(dl=512, dr=64, H=16), dict(dl=33, dr=0, H=2))):
        p = Problem([5, 9], kv="f32", ps=4, seed=i, **shape)
        out, lse = p.attention()
        d = dict(p=p, want=(out, lse), q=p.q.cuda(), kv=p.kv.cuda(), t=p.table.cuda(), rl=p.row_len.cuda(),
                 out=torch.zeros((p.R, p.H, p.dl), device="cuda"), lse=lse.float().cuda(),
                 total=torch.zeros((p.B, p.max_len), device="cuda"), stream=torch.cuda.Stream())
        jobs.append(d)
    torch.cuda.synchronize()

    # the C calls alone, with their arguments at hand, so that the threads are mostly inside them
    lib, P = nsa.load(), lambda t: C.c_void_p(t.data_ptr())
    for d in jobs:
        p, q = d["p"], d["q"]
        head = (0, 0, P(q), p.H * (p.dl + p.dr), p.dl + p.dr, P(q[..., p.dl:]), p.H * (p.dl + p.dr), p.dl + p.dr, P(d["kv"]),
                p.pages, p.ps, P(d["t"]), p.table.shape[1], P(d["rl"]), p.R, 1, p.H, p.dl, p.dr, p.max_len, C.c_float(SCALE))
        stream = C.c_void_p(d["stream"].cuda_stream)
        if op == "attention":
            d["call"] = functools.partial(lib.nsa_paged_mla, *head, P(d["out"]), P(d["lse"]), None, 0, None, stream)
        else:
            d["call"] = functools.partial(lib.nsa_mla_key_weights, *head, P(d["lse"]), P(d["total"]), p.max_len, None, stream)

    failed = []

    def loop(d):
        for _ in range(CALLS):
            rc = d["call"]()
            if rc != 0:
                failed.append(rc)
                return

    threads = [threading.Thread(target=loop, args=(d,)) for d in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for d in jobs:
        out, lse = d["want"]
        if op == "attention":
            # fp32 sums of at most 576 products: far below this
            assert ((d["out"].double().cpu() - out).abs() <= 1e-4 * (1 + out.abs())).all()
            assert ((d["lse"].double().cpu() - lse).abs() <= 1e-4 * (1 + lse.abs())).all()
        else:
            # CALLS additions in fp32, each off by at most half a step of the sum
            w = CALLS * d["p"].weights(lse)
            assert ((d["total"].double().cpu() - w).abs() <= (CALLS * 2.0 ** -24 + 1e-4) * w).all()
