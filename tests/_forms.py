"""Inputs, 64-bit definitions and error bounds for the tests of latent attention's two forms.

Bounds, from the formats alone (half a step of bf16 is 2^-8 of the value, of fp32 2^-24).  A sum of n
products kept in fp32 is off by at most n 2^-23 of the sum of their magnitudes (2^-23: also where a
tensor core cuts an addend off instead of rounding it)."""
from __future__ import annotations

import torch

SCALE = 192 ** -0.5
BF, F32 = torch.bfloat16, torch.float32
EPS_BF = 2.0 ** -8


def rand(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def starts(lens, first=0):
    return torch.tensor([first] + list(lens), dtype=torch.int32).cumsum(0).to(torch.int32)


def weight(g, H):
    return rand(g, H * 256, 512, scale=512 ** -0.5)


def product_tol(x, w, exact):
    """x [.., K] and w [F, K] in 64 bits: the bound of x w^T summed in fp32 and rounded to bf16."""
    size = x.abs() @ w.abs().transpose(-1, -2)
    return EPS_BF * exact.abs() + (1 + EPS_BF) * x.shape[-1] * 2.0 ** -23 * size + 1e-30


def attention(q, kv, k_rope, nq, nk, causal, scale=SCALE):
    """(out, lse, tol_out, tol_lse) of ragged attention in 64 bits.  q [Tq, H, 192], kv [Tk, H, 256], k_rope [Tk, 64]."""
    q, kv, k_rope = q.double(), kv.double(), k_rope.double()
    Tq, H = q.shape[:2]
    out, lse = torch.zeros((Tq, H, 128), dtype=torch.float64), torch.full((Tq, H), -torch.inf, dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    q0 = k0 = 0
    for a, b in zip(nq, nk):
        for h in range(H if a and b else 0):
            k = torch.cat([kv[k0:k0 + b, h, :128], k_rope[k0:k0 + b]], 1)
            v = kv[k0:k0 + b, h, 128:]
            x = (q[q0:q0 + a, h] @ k.T) * scale
            # a score's error: 192 products, the product with the scale, the exponent's argument in fp32
            dx = (q[q0:q0 + a, h].abs() @ k.abs().T) * scale * (192 * 2.0 ** -23 + 2.0 ** -21)
            if causal:
                hide = torch.arange(b)[None, :] > torch.arange(b - a, b)[:, None]
                x, dx = x.masked_fill(hide, -torch.inf), dx.masked_fill(hide, 0.0)
            d = dx.amax(-1, keepdim=True) + 2.0 ** -20  # and 2^x and the sum of weights
            l = torch.logsumexp(x, -1, keepdim=True)
            p = torch.where(l == -torch.inf, torch.zeros_like(x), torch.exp(x - l))
            o = p @ v
            mag = p @ v.abs()
            out[q0:q0 + a, h], lse[q0:q0 + a, h] = o, l[:, 0]
            # weights rounded to bf16, every weight and the sum off by d, the sum of products in fp32, the result rounded
            tol_o[q0:q0 + a, h] = (EPS_BF + 2 * d + b * 2.0 ** -23) * mag * (1 + EPS_BF) + EPS_BF * o.abs()
            tol_l[q0:q0 + a, h] = d[:, 0] + torch.nan_to_num(l[:, 0].abs(), posinf=0, neginf=0) * 2.0 ** -22
        q0, k0 = q0 + a, k0 + b
    return out, lse, tol_o, tol_l


def merge(parts, lses):
    """(out, lse, size) in 64 bits: rows without a key are 0 and -inf; size: the sum of the addends' magnitudes."""
    l = torch.stack([x.double() for x in lses])
    total = torch.logsumexp(l, 0)
    w = torch.exp(l - torch.where(total == -torch.inf, torch.zeros_like(total), total))
    o = sum(torch.where(wi[..., None] > 0, p.double() * wi[..., None], 0.0) for p, wi in zip(parts, w))
    size = sum(torch.where(wi[..., None] > 0, p.double().abs() * wi[..., None], 0.0) for p, wi in zip(parts, w))
    return o, total, size


def close(got, want, tol, what=""):
    got, want = got.double().cpu(), want.double()
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    bad = ~(same | ((got - want).abs() <= tol))
    if bad.any():
        i = tuple(torch.nonzero(bad)[0].tolist())
        worst = ((got - want).abs() / tol.clamp_min(1e-300)).nan_to_num(posinf=1e30, nan=1e30).masked_fill(same, 0).max()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values out of bounds, first at {i}: got {float(got[i])}, "
                             f"want {float(want[i])} +- {float(tol[i])}; worst {float(worst):.3g} bounds")
