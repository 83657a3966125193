"""Inputs and 64-bit definitions for the tests of dense paged MLA attention and
cache eviction.  The definitions walk positions one request and row at a time,
from the formulas alone."""
from __future__ import annotations

import math

import numpy as np
import torch

SCALE = 192 ** -0.5


def page_table(lens, ps, gen, slack=3, fill=0):
    """Whole pages in random order; `fill` past each request's last page.  (table, pages)"""
    per = [-(-int(l) // ps) for l in lens]
    pages = sum(per) + slack
    perm = torch.randperm(pages, generator=gen).to(torch.int32)
    t = torch.full((len(lens), max(1, max(per, default=1))), fill, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, pages


def fp8_rows(x, d_latent, d_rope):
    """fp32 [slots, d] -> the e4m3 row layout (codes | fp32 scale per 128 | bf16 rope)."""
    slots, nb = x.shape[0], d_latent // 128
    lat = x[:, :d_latent].reshape(slots, nb, 128)
    scale = lat.abs().amax(-1) / 448.0
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    codes = (lat / scale[..., None]).reshape(slots, d_latent).to(torch.float8_e4m3fn)
    return torch.cat([codes.view(torch.uint8), scale.contiguous().view(torch.uint8).reshape(slots, 4 * nb),
                      x[:, d_latent:].to(torch.bfloat16).contiguous().view(torch.uint8).reshape(slots, 2 * d_rope)], 1)


def row_values(kv, kv_dt, d_latent, d_rope):
    """Cache rows [.., row] -> float64 [.., d_latent + d_rope]; an e4m3 row stands for
    code x scale rounded to fp32, then to bf16."""
    if kv_dt != 2:
        return kv.double()
    n, nb = kv.shape[0], d_latent // 128
    codes = kv[:, :d_latent].contiguous().view(torch.float8_e4m3fn).float().view(n, nb, 128)
    scale = kv[:, d_latent:d_latent + 4 * nb].contiguous().view(torch.float32)
    lat = (codes * scale[..., None]).to(torch.bfloat16).view(n, d_latent)
    rope = kv[:, d_latent + 4 * nb:].contiguous().view(torch.bfloat16)
    return torch.cat([lat, rope], 1).double()


def slots_of(table_row, n, ps):
    pos = torch.arange(n)
    return table_row.long()[pos // ps] * ps + pos % ps


class Problem:
    """One attention problem on the CPU: rows, cache, table."""

    def __init__(self, lens, n=1, H=16, kv="bf16", ps=64, seed=0, dl=512, dr=64, row_len=None, q_scale=1.0, fill=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.n, self.H, self.ps, self.dl, self.dr = list(lens), n, H, ps, dl, dr
        self.kv_dt = {"f32": 0, "bf16": 1, "fp8": 2}[kv]
        self.q_dt = 0 if kv == "f32" else 1
        self.B, self.R = len(lens), len(lens) * n
        self.table, self.pages = page_table(lens, ps, g, fill=fill)
        x = torch.randn((self.pages * ps, dl + dr), generator=g)
        self.kv = x if kv == "f32" else x.to(torch.bfloat16) if kv == "bf16" else fp8_rows(x, dl, dr)
        q = torch.randn((self.R, H, dl + dr), generator=g) * q_scale
        self.q = q if kv == "f32" else q.to(torch.bfloat16)
        if row_len is None:
            row_len = [max(0, l - (n - 1 - i)) for l in self.lens for i in range(n)]
        self.row_len = torch.tensor(row_len, dtype=torch.int32)
        self.max_len = max(self.lens, default=0)

    def values(self, r):
        """float64 values of the positions that row r sees."""
        L = int(self.row_len[r])
        rows = self.kv[slots_of(self.table[r // self.n], L, self.ps)]
        return row_values(rows, self.kv_dt, self.dl, self.dr)

    def scores(self, r):
        """float64 scores [H, row_len] of row r and its values."""
        k = self.values(r)
        return (self.q[r].double() @ k.T) * SCALE, k

    def attention(self):
        out = torch.zeros((self.R, self.H, self.dl), dtype=torch.float64)
        lse = torch.full((self.R, self.H), -math.inf, dtype=torch.float64)
        for r in range(self.R):
            x, k = self.scores(r)
            if x.shape[1]:
                lse[r] = torch.logsumexp(x, 1)
                out[r] = torch.exp(x - lse[r][:, None]) @ k[:, :self.dl]
        return out, lse

    def weights(self, lse):
        w = torch.zeros((self.B, max(1, self.max_len)), dtype=torch.float64)
        for r in range(self.R):
            x, _ = self.scores(r)
            if x.shape[1]:
                w[r // self.n, :x.shape[1]] += torch.exp(x - lse[r].double()[:, None]).sum(0)
        return w


def select(total, lens, sinks, recent, budget):
    """Kept positions by sorting each request's middle range in plain Python."""
    keep = np.full((len(lens), budget), -1, np.int32)
    new = np.zeros(len(lens), np.int32)
    for b, L in enumerate(lens):
        L = int(L)
        if L <= budget:
            k = list(range(L))
        else:
            mid = range(sinks, L - recent)
            w = total[b]
            key = lambda i: (1, 0.0) if math.isnan(w[i]) else (0, -float(w[i]))
            best = sorted(mid, key=lambda i: (*key(i), i))[:budget - sinks - recent]
            k = sorted(list(range(sinks)) + best + list(range(L - recent, L)))
        keep[b, :len(k)] = k
        new[b] = len(k)
    return keep, new
