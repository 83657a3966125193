"""Measured cases of the two forms of latent attention: expanded for prompts, absorbed for tokens.

A cached row holds one latent vector of 512 values and 64 rope values for all heads.  The weight of
the key/value up-projection, w [H * 256, 512], holds for each head 128 rows W_k that expand a latent
into the head's keys and 128 rows W_v that expand it into the head's values.  Five operators:

  expand   nsa_mla_expand_kv    rows of the paged cache gathered and expanded: keys and values of every head
  prefill  nsa_mla_prefill      attention of ragged prompts over expanded keys and values (192 / 128 wide)
  merge    nsa_merge_attention  attention over parts of the keys joined by the parts' lse
  absorb   nsa_mla_absorb_q     a head's query through W_k into the latent space, where the cache is attended
  project  nsa_mla_project_v    a head's attended latent through W_v

Where `own` is false, `run` computes them from elementary torch operations in 32 bits; where it is
true, it makes the library's calls.
"""
import math

import torch

own = False

D_LATENT, D_ROPE, D_NOPE, D_V = 512, 64, 128, 128
ROW_FP8 = D_LATENT + 16 + 2 * D_ROPE  # e4m3 codes | four fp32 scales | bf16 rope values
SCALE = (D_NOPE + D_ROPE) ** -0.5

# Query lengths are q_lo .. q_hi and prefixes p_lo .. p_hi, uniform in their logarithm; the first
# request has the longest of both.  A causal request attends its prefix and itself, another one the
# prefix alone.


def listed():
    return [
        # a short turn's cached rows on a rank of 16 heads, fp8 cache
        dict(name="expand_turn_fp8_h16", op="expand", kv="fp8", m=1037, H=16, ps=64),
        # one chunk of a long prefix for all heads
        dict(name="expand_chunk_h128", op="expand", kv="bf16", m=8192, H=128, ps=64),
        # one short turn after a few hundred tokens: latency
        dict(name="prefill_turn_h16", op="prefill", B=1, H=16, q_lo=37, q_hi=37, p_lo=600, p_hi=600, causal=True),
        # new prompts of mixed lengths in one batch, all heads
        dict(name="prefill_batch_h128", op="prefill", B=8, H=128, q_lo=150, q_hi=2000, p_lo=0, p_hi=0, causal=True),
        # one long prompt, all heads
        dict(name="prefill_long_h128", op="prefill", B=1, H=128, q_lo=8192, q_hi=8192, p_lo=0, p_hi=0, causal=True),
        # chunks of two prompts over their long prefixes, on a rank of 16 heads
        dict(name="prefill_prefix_h16", op="prefill", B=2, H=16, q_lo=500, q_hi=1001, p_lo=20000, p_hi=40000, causal=False),
        # the two parts of a short turn; and the three of a long chunk for all heads
        dict(name="merge_turn_h16", op="merge", n=2, rows=37, H=16, D=128, dtype="bf16"),
        dict(name="merge_chunk_h128", op="merge", n=3, rows=8192, H=128, D=128, dtype="bf16"),
        # a decoding batch with all heads: queries in, attended latents out
        dict(name="absorb_batch_h128", op="absorb", R=32, H=128),
        dict(name="project_batch_h128", op="project", R=32, H=128),
        # a prompt's chunk that attends selected positions, on a rank of 16 heads
        dict(name="absorb_chunk_h16", op="absorb", R=4001, H=16),
        dict(name="project_chunk_h16", op="project", R=4001, H=16),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    return rng.choice([16, 32, 64, 128, rng.randint(1, 128)])


def draw(rng):
    op = rng.choice(["expand", "prefill", "prefill", "merge", "absorb", "project"])
    H = _heads(rng)
    if op == "expand":
        # no more output than the largest listed case has
        return dict(op=op, kv=rng.choice(["bf16", "fp8"]), m=_log_int(rng, 1, min(65536, 8192 * 128 // H)), H=H, ps=rng.choice([16, 32, 64, 128]))
    if op == "merge":
        D = rng.choice([64, 128, 512])
        n = rng.choice([2, 2, 3, 5])
        return dict(op=op, n=n, rows=_log_int(rng, 1, 8192 * 128 * 3 * 128 // (H * n * D)), H=H, D=D, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op in ("absorb", "project"):
        return dict(op=op, R=_log_int(rng, 1, 8192 * 128 // (2 * H)), H=H)
    B = _log_int(rng, 1, 16)
    causal = rng.random() < 0.6
    q_hi = _log_int(rng, 1, 8192)
    p_hi = rng.choice([0, _log_int(rng, 1, 65536)]) if causal else _log_int(rng, 1, 65536)
    # no more pairs of a query and a key, nor more keys, than the largest listed cases have
    while B * H * q_hi * (p_hi + q_hi * causal) > 64 * 8192 * 8192 or B * H * (p_hi + q_hi * causal) > 2 * 128 * 8192:
        q_hi, p_hi = max(1, q_hi * 2 // 3), p_hi * 2 // 3 if causal else max(1, p_hi * 2 // 3)
    return dict(op=op, B=B, H=H, q_lo=max(1, int(q_hi * rng.uniform(0.1, 1.0))), q_hi=q_hi,
                p_lo=int(p_hi * rng.uniform(0.1, 1.0)), p_hi=p_hi, causal=causal)


# ------------------------------------------------------------------ inputs

def _spread(B, lo, hi, step):
    """B lengths by the case alone, so that its work does not depend on the seed; the first is `hi`."""
    # the fractional parts of i * step spread evenly over [0, 1)
    u = [(i * step) % 1.0 for i in range(B)]
    a = max(lo, 0.5)
    return [hi if i == 0 or hi == 0 else min(hi, max(lo, int(round(math.exp(math.log(a) + u[i] * (math.log(hi) - math.log(a)))))))
            for i in range(B)]


def _lengths(case):
    """Queries and keys of each request of a prefill case."""
    nq = _spread(case["B"], case["q_lo"], case["q_hi"], 0.6180339887498949)
    p = _spread(case["B"], case["p_lo"], case["p_hi"], 0.4142135623730951)
    return nq, [a + b if case["causal"] else b for a, b in zip(nq, p)]


def _starts(lens, dev):
    return torch.tensor([0] + lens, device=dev).cumsum(0).to(torch.int32)


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


def _weight(H, g, dev):
    """[H * 256, 512]: the product with latents of unit variance has unit variance."""
    w = torch.randn((H * (D_NOPE + D_V), D_LATENT), generator=g, device=dev)
    return (w * D_LATENT ** -0.5).to(torch.bfloat16)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, H = case["op"], case["H"]
    bf16 = dict(generator=g, device=dev, dtype=torch.bfloat16)
    s = dict(case=case, op=op, status=torch.zeros(1, dtype=torch.int32, device=dev))
    if op == "expand":
        # the slots of the rows, whole pages in random order over the pool, as the flattened page table gives them
        m, ps = case["m"], case["ps"]
        used = -(-m // ps)
        pages = torch.randperm(used + 3, generator=g, device=dev)[:used]
        slots = (pages[:, None] * ps + torch.arange(ps, device=dev)[None, :]).flatten()[:m]
        s.update(cache=_kv_cache(case["kv"], (used + 3) * ps, g, dev), slots=slots.to(torch.int32), w=_weight(H, g, dev))
    elif op == "prefill":
        nq, nk = _lengths(case)
        # the queries as their projection leaves them; keys and values of a head next to each other
        s["q"] = torch.randn((sum(nq), H, D_NOPE + D_ROPE), **bf16)
        s["kv"] = torch.randn((sum(nk), H, D_NOPE + D_V), **bf16)
        s["k_rope"] = torch.randn((sum(nk), D_ROPE), **bf16)
        s["nq"], s["nk"], s["cu_q"], s["cu_k"] = nq, nk, _starts(nq, dev), _starts(nk, dev)
    elif op == "merge":
        shape = (case["rows"], H, case["D"])
        dt = {"bf16": torch.bfloat16, "f32": torch.float32}[case["dtype"]]
        s["parts"] = [torch.randn(shape, generator=g, device=dev, dtype=dt) for _ in range(case["n"])]
        s["lses"] = [torch.randn(shape[:2], generator=g, device=dev) * 2 + 6 for _ in range(case["n"])]
        # rows that see no key of the last part
        none = torch.rand(shape[0], generator=g, device=dev) < 0.1
        s["parts"][-1][none] = 0
        s["lses"][-1][none] = -math.inf
    else:
        s["w"] = _weight(H, g, dev)
        if op == "absorb":
            s["x"] = torch.randn((case["R"], H, D_NOPE + D_ROPE), **bf16)[..., :D_NOPE]
        else:
            s["x"] = torch.randn((case["R"], H, D_LATENT), **bf16)
    return s


# ------------------------------------------------------------------ plain forms

def _plain_expand(s):
    rows = s["cache"][s["slots"].long()]
    if rows.dtype == torch.uint8:
        # an e4m3 row stands for what the library's dequantiser gives: code x scale in fp32, then bf16
        codes = rows[:, :D_LATENT].view(torch.float8_e4m3fn).float().view(-1, 4, 128)
        scale = rows[:, D_LATENT:D_LATENT + 16].contiguous().view(torch.float32)
        lat = (codes * scale[..., None]).to(torch.bfloat16).view(-1, D_LATENT)
        rope = rows[:, D_LATENT + 16:].contiguous().view(torch.bfloat16)
    else:
        lat, rope = rows[:, :D_LATENT], rows[:, D_LATENT:].contiguous()
    kv = torch.matmul(lat.float(), s["w"].float().t())
    return kv.to(torch.bfloat16).view(-1, s["case"]["H"], D_NOPE + D_V), rope


def _plain_prefill(s):
    H, causal = s["case"]["H"], s["case"]["causal"]
    dev = s["q"].device
    out = torch.empty((s["q"].shape[0], H, D_V), dtype=torch.bfloat16, device=dev)
    lse = torch.empty((s["q"].shape[0], H), device=dev)
    q0 = k0 = 0
    for nq, nk in zip(s["nq"], s["nk"]):
        k_rope = s["k_rope"][k0:k0 + nk].float()
        hidden = None
        if causal:
            hidden = torch.arange(nk, device=dev)[None, :] > torch.arange(nk - nq, nk, device=dev)[:, None]
        # heads at a time: scores of up to 4 GB
        step = max(1, min(H, 2 ** 30 // max(1, nq * nk)))
        for h in range(0, H, step):
            q = s["q"][q0:q0 + nq, h:h + step].float().transpose(0, 1)
            kv = s["kv"][k0:k0 + nk, h:h + step].float().transpose(0, 1)
            x = torch.matmul(q[..., :D_NOPE], kv[..., :D_NOPE].transpose(1, 2))
            x.add_(torch.matmul(q[..., D_NOPE:], k_rope.t())).mul_(SCALE)
            if hidden is not None:
                x.masked_fill_(hidden, -math.inf)
            m = x.amax(-1, keepdim=True)
            p = x.sub_(m).exp_()
            l = p.sum(-1, keepdim=True)
            o = torch.matmul(p, kv[..., D_NOPE:]) / l
            out[q0:q0 + nq, h:h + step] = o.transpose(0, 1).to(torch.bfloat16)
            lse[q0:q0 + nq, h:h + step] = (m + torch.log(l)).squeeze(-1).t()
        q0, k0 = q0 + nq, k0 + nk
    return out, lse


def _plain_merge(s):
    lses = torch.stack(s["lses"])
    m = lses.amax(0)
    w = torch.exp(lses - m)
    total = w.sum(0)
    o = torch.zeros(s["parts"][0].shape, device=m.device)
    for part, wi in zip(s["parts"], w):
        o += part.float() * (wi / total)[..., None]
    return o.to(s["parts"][0].dtype), m + torch.log(total)


def _plain_head_product(s):
    w = s["w"].float().view(s["case"]["H"], D_NOPE + D_V, D_LATENT)
    x = s["x"].float().transpose(0, 1)
    w = w[:, :D_NOPE] if s["op"] == "absorb" else w[:, D_NOPE:].transpose(1, 2)
    return torch.matmul(x, w).transpose(0, 1).to(torch.bfloat16).contiguous()


# ------------------------------------------------------------------ one pass

def run(state):
    s, op = state, state["op"]
    if own:
        return _OWN[op](s)
    if op == "expand":
        return _plain_expand(s)
    if op == "prefill":
        return _plain_prefill(s)
    if op == "merge":
        return _plain_merge(s)
    return _plain_head_product(s)


def _own_expand(s):
    import deepseek_sparse_mla_indexer_gb300 as nsa
    c = s["case"]
    dev = s["cache"].device
    if "ws" not in s:
        s["ws"] = nsa.alloc_mla_expand_workspace(c["m"])
    kv = torch.empty((c["m"], c["H"], D_NOPE + D_V), dtype=torch.bfloat16, device=dev)
    k_rope = torch.empty((c["m"], D_ROPE), dtype=torch.bfloat16, device=dev)
    nsa.nsa_mla_expand_kv(nsa.DT_E4M3 if c["kv"] == "fp8" else nsa.DT_BF16, s["cache"], s["slots"], s["w"], kv, k_rope, s["ws"], s["status"])
    return kv, k_rope


def _own_prefill(s):
    import deepseek_sparse_mla_indexer_gb300 as nsa
    c = s["case"]
    q, kv = s["q"], s["kv"]
    if "ws" not in s:
        s["ws"] = nsa.alloc_mla_prefill_workspace()
    out = torch.empty((q.shape[0], c["H"], D_V), dtype=torch.bfloat16, device=q.device)
    lse = torch.empty((q.shape[0], c["H"]), dtype=torch.float32, device=q.device)
    nsa.nsa_mla_prefill(q[..., :D_NOPE], q[..., D_NOPE:], kv[..., :D_NOPE], s["k_rope"], kv[..., D_NOPE:], s["cu_q"], s["cu_k"],
                        c["causal"], SCALE, out, lse, s["ws"], s["status"])
    return out, lse


def _own_merge(s):
    import deepseek_sparse_mla_indexer_gb300 as nsa
    out, lse = torch.empty_like(s["parts"][0]), torch.empty_like(s["lses"][0])
    nsa.nsa_merge_attention(s["parts"], s["lses"], out, lse)
    return out, lse


def _own_absorb(s):
    import deepseek_sparse_mla_indexer_gb300 as nsa
    out = torch.empty((s["case"]["R"], s["case"]["H"], D_LATENT), dtype=torch.bfloat16, device=s["w"].device)
    nsa.nsa_mla_absorb_q(s["x"], s["w"], out)
    return out


def _own_project(s):
    import deepseek_sparse_mla_indexer_gb300 as nsa
    out = torch.empty((s["case"]["R"], s["case"]["H"], D_V), dtype=torch.bfloat16, device=s["w"].device)
    nsa.nsa_mla_project_v(s["x"], s["w"], out)
    return out


_OWN = {"expand": _own_expand, "prefill": _own_prefill, "merge": _own_merge, "absorb": _own_absorb, "project": _own_project}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, H = case["op"], case["H"]
    if op == "expand":
        m, cols = case["m"], H * (D_NOPE + D_V)
        row = ROW_FP8 if case["kv"] == "fp8" else 2 * (D_LATENT + D_ROPE)
        return {"bytes": m * (row + 4 + 2 * D_ROPE + 2 * cols) + 2 * cols * D_LATENT, "flops": 2.0 * m * cols * D_LATENT}
    if op == "merge":
        values, each = case["rows"] * H * case["D"], {"bf16": 2, "f32": 4}[case["dtype"]]
        return {"bytes": (case["n"] + 1) * (values * each + 4 * case["rows"] * H), "flops": 2.0 * case["n"] * values}
    if op in ("absorb", "project"):
        R = case["R"]
        return {"bytes": 2 * R * H * (D_NOPE + D_LATENT) + 2 * H * D_NOPE * D_LATENT, "flops": 2.0 * R * H * D_NOPE * D_LATENT}
    nq, nk = _lengths(case)
    pairs = 0
    for a, b in zip(nq, nk):
        pairs += a * (b - a) + a * (a + 1) // 2 if case["causal"] else a * b
    rows = sum(nq) * H * (2 * (D_NOPE + D_ROPE + D_V) + 4)
    keys = sum(nk) * 2 * (H * (D_NOPE + D_V) + D_ROPE)
    return {"bytes": rows + keys + 8 * (case["B"] + 1), "flops": 2.0 * pairs * H * (D_NOPE + D_ROPE + D_V)}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    op, H = case["op"], case["H"]
    if op == "prefill":
        nq, nk = _lengths(case)
        if sum(a * b for a, b in zip(nq, nk)) * H > 2e10:
            return None  # too long in 64 bits
    s = prepare(case, seed)
    if op == "expand":
        rows = s["cache"].index_select(0, s["slots"].long())
        if case["kv"] == "fp8":
            lat, rope = [], rows[:, ROW_FP8 - 2 * D_ROPE:].contiguous().view(torch.bfloat16).double()
            for j in range(4):
                codes = rows[:, 128 * j:128 * (j + 1)].contiguous().view(torch.float8_e4m3fn).double()
                scale = rows[:, D_LATENT + 4 * j:D_LATENT + 4 * j + 4].contiguous().view(torch.float32).double()
                # a code has 4 significant bits, a scale 24: their product is exact in 64 bits; then the
                # two roundings that define the row's value
                lat.append((codes * scale).float().bfloat16().double())
            lat = torch.cat(lat, 1)
        else:
            lat, rope = rows.double().split([D_LATENT, D_ROPE], 1)
        return torch.einsum("tl,hfl->thf", lat, s["w"].double().view(H, D_NOPE + D_V, D_LATENT)), rope.contiguous()
    if op == "merge":
        weights = torch.softmax(torch.stack(s["lses"], -1).double(), -1)
        return (torch.einsum("rhdn,rhn->rhd", torch.stack([p.double() for p in s["parts"]], -1), weights),
                torch.logsumexp(torch.stack(s["lses"], -1).double(), -1))
    if op in ("absorb", "project"):
        outs = []
        for h in range(H):
            block = s["w"][h * (D_NOPE + D_V):(h + 1) * (D_NOPE + D_V)].double()
            outs.append(s["x"][:, h].double() @ (block[:D_NOPE] if op == "absorb" else block[D_NOPE:].t()))
        return torch.stack(outs, 1)
    outs, lses, q0, k0 = [], [], 0, 0
    for a, b in zip(nq, nk):
        q_all, kv_all, k_rope = s["q"][q0:q0 + a], s["kv"][k0:k0 + b], s["k_rope"][k0:k0 + b].double()
        o = torch.empty((a, H, D_V), dtype=torch.float64, device=q_all.device)
        lse = torch.empty((a, H), dtype=torch.float64, device=q_all.device)
        for h in range(H):
            k = torch.cat([kv_all[:, h, :D_NOPE].double(), k_rope], 1)
            x = (q_all[:, h].double() @ k.t()) * SCALE
            if case["causal"]:
                x += torch.full_like(x, -math.inf).triu_(b - a + 1)
            o[:, h] = torch.softmax(x, -1) @ kv_all[:, h, D_NOPE:].double()
            lse[:, h] = torch.logsumexp(x, -1)
        outs.append(o)
        lses.append(lse)
        q0, k0 = q0 + a, k0 + b
    return torch.cat(outs), torch.cat(lses)
