"""Measured cases of the dense paged MLA attention and the cache-eviction operators.

Four operators, as a serving loop runs them over one layer's paged latent cache:

  attn     nsa_paged_mla        attention of each request's newest token(s) over its whole paged cache
  weights  nsa_mla_key_weights  the attention weight each cached position received, summed over heads
                                and rows, added to a running total per position
  select   nsa_evict_select     the positions a request keeps: first ones, last ones, heaviest between
  compact  nsa_evict_compact    the kept rows of every paged array moved to the front, in place

Where `own` is false, `run` computes them from elementary torch operations in 32 bits; where it is
true, it makes the library's calls.
"""
import math

import torch

own = False

D_LATENT, D_ROPE = 512, 64
ROW_FP8 = D_LATENT + 16 + 2 * D_ROPE  # e4m3 codes | four fp32 scales | bf16 rope values
SCALE = 192 ** -0.5

# Lengths are min_len .. max_len, uniform in their logarithm; the first request has max_len.


def listed():
    return [
        # one request just past its prompt on a rank that holds 16 heads: latency
        dict(name="attn_one_short_h16", op="attn", kv="bf16", B=1, n=1, H=16, ps=64, min_len=501, max_len=501),
        # 32 requests decoding, all 128 heads: the repository's benchmark batch, attended densely
        dict(name="attn_batch_h128", op="attn", kv="bf16", B=32, n=1, H=128, ps=64, min_len=4096, max_len=32768),
        # 128 requests on a rank of 16 heads, fp8 cache
        dict(name="attn_batch_fp8_h16", op="attn", kv="fp8", B=128, n=1, H=16, ps=64, min_len=1024, max_len=16384),
        # speculative verify of four draft tokens over long contexts, fp8 cache, all heads
        dict(name="attn_verify_fp8_h128", op="attn", kv="fp8", B=8, n=4, H=128, ps=64, min_len=16384, max_len=131072),
        # the weights that the same kinds of step leave on the cache
        dict(name="weights_small_h16", op="weights", kv="bf16", B=2, n=1, H=16, ps=64, min_len=700, max_len=2111),
        dict(name="weights_batch_h128", op="weights", kv="bf16", B=32, n=1, H=128, ps=64, min_len=4096, max_len=32768),
        dict(name="weights_verify_fp8_h16", op="weights", kv="fp8", B=16, n=4, H=16, ps=64, min_len=16384, max_len=65536),
        # one request over its budget: latency
        dict(name="select_one", op="select", B=1, min_len=4099, max_len=4099, keep=2048, sinks=4, recent=64),
        # a long-context batch cut to 32 K positions a request
        dict(name="select_batch_long", op="select", B=16, min_len=50000, max_len=131072, keep=32768, sinks=64, recent=1024),
        # the rows that one short request keeps: bf16 latent rows and indexer keys with their scales
        dict(name="compact_one", op="compact", kv="bf16", B=1, ps=64, min_len=4099, max_len=4099, keep=2048, sinks=4, recent=64),
        # a decoding batch, fp8 rows, odd budget
        dict(name="compact_batch_fp8", op="compact", kv="fp8", B=32, ps=64, min_len=4096, max_len=32768, keep=5001, sinks=4, recent=512),
        # long contexts cut in half
        dict(name="compact_long", op="compact", kv="bf16", B=4, ps=64, min_len=65536, max_len=131072, keep=50000, sinks=16, recent=4096),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "weights", "select", "compact"])
    B = _log_int(rng, 1, 64)
    # so many positions over the batch that no draw outgrows the listed cases
    longest = min(131072, 400000 // B)
    hi = _log_int(rng, 16, longest)
    lo = max(1, int(hi * rng.uniform(0.1, 1.0)))
    case = dict(op=op, B=B, min_len=lo, max_len=hi)
    if op in ("attn", "weights"):
        case.update(kv=rng.choice(["bf16", "fp8"]), n=rng.choice([1, 1, 1, 2, 4]), ps=rng.choice([16, 32, 64, 128]),
                    H=rng.choice([16, 32, 64, 128, rng.randint(1, 128)]))
    else:
        keep = _log_int(rng, 8, hi)
        sinks = rng.randint(0, min(64, keep // 4))
        case.update(keep=keep, sinks=sinks, recent=rng.randint(0, keep // 4))
        if op == "compact":
            case.update(kv=rng.choice(["bf16", "fp8"]), ps=rng.choice([16, 64, 128]))
    return case


# ------------------------------------------------------------------ inputs

def _lengths(case):
    """Lengths by the case alone, so that its work does not depend on the seed."""
    B, lo, hi = case["B"], case["min_len"], case["max_len"]
    # the fractional parts of i * golden ratio spread evenly over [0, 1)
    u = [(i * 0.6180339887498949) % 1.0 for i in range(B)]
    return [hi if i == 0 else int(round(math.exp(math.log(lo) + u[i] * (math.log(hi) - math.log(lo))))) for i in range(B)]


def _page_table(lens, ps, g, dev):
    """Whole pages in random order over the pool; entries past a request's length are 0."""
    per = torch.tensor([-(-l // ps) for l in lens])
    used = int(per.sum())
    pages = used + 3
    perm = torch.randperm(pages, generator=g, device=dev)[:used].to(torch.int32)
    width = int(per.max())
    live = torch.arange(width)[None, :] < per[:, None]
    table = torch.zeros((len(lens), width), dtype=torch.int32, device=dev)
    table[live.to(dev)] = perm
    return table, pages


def _kv_cache(kv, slots, g, dev):
    x = torch.randn((slots, D_LATENT + D_ROPE), generator=g, device=dev, dtype=torch.bfloat16)
    if kv == "bf16":
        return x
    rows = torch.empty((slots, ROW_FP8), dtype=torch.uint8, device=dev)
    lat = x[:, :D_LATENT].view(slots, 4, 128).float()
    scale = lat.abs().amax(-1) / 448.0
    rows[:, :D_LATENT] = (lat / scale[..., None]).view(slots, D_LATENT).to(torch.float8_e4m3fn).view(torch.uint8)
    rows[:, D_LATENT:D_LATENT + 16] = scale.contiguous().view(torch.uint8)
    rows[:, D_LATENT + 16:] = x[:, D_LATENT:].contiguous().view(torch.uint8)
    return rows


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    lens = _lengths(case)
    B = case["B"]
    s = dict(case=case, op=case["op"], max_len=max(lens), status=torch.zeros(1, dtype=torch.int32, device=dev))
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if case["op"] in ("attn", "weights"):
        n, H, ps = case["n"], case["H"], case["ps"]
        # row i of a request's n newest tokens sees all but the n - 1 - i tokens after its own
        rows = [max(0, l - (n - 1 - i)) for l in lens for i in range(n)]
        s["row_len"] = torch.tensor(rows, dtype=torch.int32, device=dev)
        s["table"], s["pages"] = _page_table(lens, ps, g, dev)
        s["cache"] = _kv_cache(case["kv"], s["pages"] * ps, g, dev)
        q = torch.randn((B * n, H, D_LATENT + D_ROPE), generator=g, device=dev, dtype=torch.bfloat16)
        s["q_nope"], s["q_rope"] = q[..., :D_LATENT], q[..., D_LATENT:]
        if case["op"] == "weights":
            s["lse"] = _plain_attention(s, want_out=False)[1]
            s["total"] = torch.rand((B, s["max_len"]), generator=g, device=dev)
    else:
        # weights that a few positions dominate, as attention leaves them; equal values among the small ones
        w = torch.randn((B, s["max_len"]), generator=g, device=dev).mul_(2.0).exp_()
        s["total"] = (w * 256).round_() / 256
        if case["op"] == "compact":
            ps = case["ps"]
            s["table"], s["pages"] = _page_table(lens, ps, g, dev)
            s["cache"] = _kv_cache(case["kv"], s["pages"] * ps, g, dev)
            s["index_k"] = torch.randn((s["pages"] * ps, 128), generator=g, device=dev).to(torch.float8_e4m3fn)
            s["index_scale"] = torch.rand((s["pages"] * ps,), generator=g, device=dev)
            s["keep"], s["new_len"] = _plain_select(s)
    return s


# ------------------------------------------------------------------ plain forms

def _values(cache, page_size, table, dtype=torch.float32):
    """The cached rows of each request in order, [B, positions, 576].  An e4m3 row stands for
    what the library's dequantiser gives: code x scale in fp32, then bf16."""
    if cache.dtype == torch.uint8:
        codes = cache[:, :D_LATENT].view(torch.float8_e4m3fn).float().view(-1, 4, 128)
        scale = cache[:, D_LATENT:D_LATENT + 16].contiguous().view(torch.float32)
        lat = (codes * scale[..., None]).to(torch.bfloat16).view(-1, D_LATENT)
        cache = torch.cat([lat, cache[:, D_LATENT + 16:].contiguous().view(torch.bfloat16)], 1)
    pages = cache.view(-1, page_size, D_LATENT + D_ROPE)
    return pages[table.long()].view(table.shape[0], -1, D_LATENT + D_ROPE).to(dtype)


def _scores(s, dtype=torch.float32):
    """Scaled scores [B, n, H, positions], -inf at and past each row's length, and the values."""
    c = s["case"]
    k = _values(s["cache"], c["ps"], s["table"], dtype)
    q = torch.cat([s["q_nope"], s["q_rope"]], -1).to(dtype).view(c["B"], c["n"] * c["H"], -1)
    x = torch.matmul(q, k.transpose(1, 2)).view(c["B"], c["n"], c["H"], -1).mul_(SCALE)
    masked = torch.arange(k.shape[1], device=k.device) >= s["row_len"].view(c["B"], c["n"], 1, 1)
    return x.masked_fill_(masked, -math.inf), k


def _plain_attention(s, want_out=True):
    c = s["case"]
    x, k = _scores(s)
    m = x.amax(-1, keepdim=True)
    p = torch.exp_(x.sub_(torch.where(torch.isinf(m), torch.zeros_like(m), m)))
    l = p.sum(-1, keepdim=True)
    lse = (m + torch.log(l)).view(c["B"] * c["n"], c["H"])
    if not want_out:
        return None, lse
    o = torch.matmul(p.view(c["B"], c["n"] * c["H"], -1), k[..., :D_LATENT])
    o = o / torch.where(l > 0, l, torch.ones_like(l)).view(c["B"], -1, 1)
    return o.view(c["B"] * c["n"], c["H"], D_LATENT).to(torch.bfloat16), lse


def _plain_weights(s):
    c = s["case"]
    x, _ = _scores(s)
    lse = s["lse"].view(c["B"], c["n"], c["H"], 1)
    p = torch.where(torch.isinf(lse), torch.zeros_like(x), torch.exp(x - lse))
    w = p.sum((1, 2))[:, :s["max_len"]]
    # in place, as the running total of a user's program; positions past the rows' lengths get zeros
    return s["total"].add_(w)


def _plain_select(s):
    c = s["case"]
    w, lens, keep = s["total"], s["lens"].long()[:, None], c["keep"]
    pos = torch.arange(w.shape[1], device=w.device)[None, :]
    held = (pos < c["sinks"]) | (pos >= lens - c["recent"])
    rank = torch.where(held, torch.full_like(w, math.inf), w)
    rank = torch.where(pos < lens, rank, torch.full_like(w, -math.inf))
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices  # ties: the lower position first
    place = torch.empty_like(order)
    place.scatter_(1, order, pos.expand_as(order).contiguous())
    kept = (pos < lens) & (place < keep)
    new_len = kept.sum(1)
    at = kept.cumsum(1) - 1
    out = torch.full((w.shape[0], keep + 1), -1, dtype=torch.int32, device=w.device)
    # what is not kept goes to a column of its own, which is cut off
    out.scatter_(1, torch.where(kept, at, torch.full_like(at, keep)), pos.expand_as(at).to(torch.int32))
    return out[:, :keep].contiguous(), new_len.to(torch.int32)


def _plain_compact(s):
    c = s["case"]
    ps, table = c["ps"], s["table"].long()
    i = torch.arange(s["keep"].shape[1], device=table.device)[None, :]
    live = i < s["new_len"].long()[:, None]
    b, to = torch.nonzero(live, as_tuple=True)
    src = s["keep"].long()[live]
    from_slot = table[b, src // ps] * ps + src % ps
    to_slot = table[b, to // ps] * ps + to % ps
    for a in (s["cache"], s["index_k"].view(torch.uint8), s["index_scale"]):
        a[to_slot] = a[from_slot]
    t = s["total"]
    moved = torch.zeros_like(t)
    moved[b, to] = t[b, src]
    inside = torch.arange(t.shape[1], device=t.device)[None, :] < s["lens"].long()[:, None]
    t.copy_(torch.where(inside, moved, t))
    return _compacted(s)


def _compacted(s):
    cache = s["cache"]
    if cache.dtype == torch.uint8:  # codes, scales and rope values, as what they stand for
        parts = [cache[:, :D_LATENT].view(torch.float8_e4m3fn), cache[:, D_LATENT:D_LATENT + 16].view(torch.float32),
                 cache[:, D_LATENT + 16:].view(torch.bfloat16)]
    else:
        parts = [cache]
    return parts + [s["index_k"], s["index_scale"], s["total"]]


# ------------------------------------------------------------------ one pass

def run(state):
    s, op = state, state["op"]
    if own:
        return _OWN[op](s)
    if op == "attn":
        return _plain_attention(s)
    if op == "weights":
        return _plain_weights(s)
    if op == "select":
        return _plain_select(s)
    return _plain_compact(s)


def _own_attn(s):
    import deepseek_sparse_mla_indexer_gb300 as nsa
    c = s["case"]
    kv_dt = nsa.DT_E4M3 if c["kv"] == "fp8" else nsa.DT_BF16
    R, H = s["q_nope"].shape[:2]
    if "ws" not in s:
        s["ws"] = nsa.alloc_paged_mla_workspace(nsa.DT_BF16, kv_dt, R, c["n"], H, s["max_len"])
    out = torch.empty((R, H, D_LATENT), dtype=torch.bfloat16, device=s["cache"].device)
    lse = torch.empty((R, H), dtype=torch.float32, device=s["cache"].device)
    nsa.nsa_paged_mla(nsa.DT_BF16, kv_dt, s["q_nope"], s["q_rope"], s["cache"], c["ps"], s["table"], s["row_len"], c["n"],
                      s["max_len"], SCALE, out, lse, s["ws"], s["status"])
    return out, lse


def _own_weights(s):
    import deepseek_sparse_mla_indexer_gb300 as nsa
    c = s["case"]
    kv_dt = nsa.DT_E4M3 if c["kv"] == "fp8" else nsa.DT_BF16
    nsa.nsa_mla_key_weights(nsa.DT_BF16, kv_dt, s["q_nope"], s["q_rope"], s["cache"], c["ps"], s["table"], s["row_len"],
                            c["n"], s["max_len"], SCALE, s["lse"], s["total"], s["status"])
    return s["total"]


def _own_select(s):
    import deepseek_sparse_mla_indexer_gb300 as nsa
    c = s["case"]
    keep = torch.empty((c["B"], c["keep"]), dtype=torch.int32, device=s["total"].device)
    new_len = torch.empty(c["B"], dtype=torch.int32, device=s["total"].device)
    nsa.nsa_evict_select(s["total"], s["lens"], s["max_len"], c["sinks"], c["recent"], c["keep"], keep, new_len, s["status"])
    return keep, new_len


def _own_compact(s):
    import deepseek_sparse_mla_indexer_gb300 as nsa
    c = s["case"]
    if "ws" not in s:
        s["ws"] = nsa.alloc_evict_workspace(c["B"], s["max_len"])
    nsa.nsa_evict_compact(s["keep"], s["new_len"], s["lens"], s["max_len"], s["table"], c["ps"],
                          [s["cache"], s["index_k"], s["index_scale"]], s["total"], s["ws"], s["status"])
    return _compacted(s)


_OWN = {"attn": _own_attn, "weights": _own_weights, "select": _own_select, "compact": _own_compact}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    lens = _lengths(case)
    B, keys = case["B"], sum(lens)
    row = {"bf16": 2 * (D_LATENT + D_ROPE), "fp8": ROW_FP8}.get(case.get("kv"), 0)
    if case["op"] in ("attn", "weights"):
        n, H = case["n"], case["H"]
        seen = sum(max(0, l - (n - 1 - i)) for l in lens for i in range(n))
        table = 4 * sum(-(-l // case["ps"]) for l in lens)
        q = B * n * H * 2 * (D_LATENT + D_ROPE)
        if case["op"] == "attn":
            return {"bytes": keys * row + q + B * n * H * (2 * D_LATENT + 4) + table + 4 * B * n,
                    "flops": 2.0 * seen * H * (2 * D_LATENT + D_ROPE)}
        return {"bytes": keys * (row + 8) + q + B * n * H * 4 + table + 4 * B * n, "flops": 2.0 * seen * H * (D_LATENT + D_ROPE)}
    if case["op"] == "select":
        return {"bytes": 4 * keys + 4 * B * case["keep"] + 8 * B, "flops": 0}
    # of a request over its budget the first ones stay; the other kept rows move, and its totals are rewritten
    over = [l for l in lens if l > case["keep"]]
    moved = len(over) * (case["keep"] - case["sinks"])
    return {"bytes": moved * 2 * (row + 128 + 4) + 8 * len(over) * case["keep"] + 4 * sum(over) + 8 * B, "flops": 0}


# ------------------------------------------------------------------ the definition in 64 bits

def _rows64(s, b, length):
    """The first `length` cached rows of request b, one 128-value block after the other."""
    ps = s["case"]["ps"]
    pos = torch.arange(length, device=s["cache"].device)
    rows = s["cache"][s["table"][b].long()[pos // ps] * ps + pos % ps]
    if rows.dtype != torch.uint8:
        return rows.double()
    parts = []
    for j in range(4):
        codes = rows[:, 128 * j:128 * (j + 1)].contiguous().view(torch.float8_e4m3fn).double()
        scale = rows[:, D_LATENT + 4 * j:D_LATENT + 4 * j + 4].contiguous().view(torch.float32).double()
        # a code has 4 significant bits, a scale 24: their product is exact in 64 bits; then the
        # two roundings that define the row's value
        parts.append((codes * scale).float().bfloat16().double())
    parts.append(rows[:, D_LATENT + 16:].contiguous().view(torch.bfloat16).double())
    return torch.cat(parts, 1)


def exact(case, seed):
    if case["op"] == "select":
        return None  # whole numbers
    s = prepare(case, seed)
    c = s["case"]
    if s["op"] == "compact":
        # request by request, on copies: position i of the front is position keep[i] of before
        outs = [t.double() for t in _compacted(s)]
        paged, total = outs[:-1], outs[-1]
        olds = [t.clone() for t in paged]
        was = total.clone()
        for b, (n, l) in enumerate(zip(s["new_len"].tolist(), s["lens"].tolist())):
            slots = (s["table"][b].long()[:, None] * c["ps"] + torch.arange(c["ps"], device=total.device)).flatten()
            src = s["keep"][b, :n].long()
            for t, old in zip(paged, olds):
                t[slots[:n]] = old[slots[src]]
            total[b, :l] = 0
            total[b, :n] = was[b, src]
        return outs
    if sum(_lengths(case)) * case["n"] * case["H"] > 6e8:
        return None  # too long in 64 bits
    outs, lses, totals = [], [], []
    for b in range(c["B"]):
        k = _rows64(s, b, int(s["lens"][b]))
        for i in range(c["n"]):
            r = b * c["n"] + i
            L = int(s["row_len"][r])
            q = torch.cat([s["q_nope"][r], s["q_rope"][r]], -1).double()
            x = (q @ k[:L].T) * SCALE
            if s["op"] == "attn":
                outs.append(torch.softmax(x, -1) @ k[:L, :D_LATENT])
                lses.append(torch.logsumexp(x, -1))
            else:
                if i == 0:
                    totals.append(s["total"][b].double())
                totals[b][:L] += torch.exp(x - s["lse"][r].double()[:, None]).sum(0)
    return (torch.stack(outs), torch.stack(lses)) if s["op"] == "attn" else torch.stack(totals)
