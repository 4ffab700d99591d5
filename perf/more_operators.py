"""Workloads of the full-attention layer that hybrid stacks put beside delta-rule layers: keys and values
rotated and appended to a paged cache, attention over whole prompts, and paged decode with shared prefixes.
Inputs, the operators in plain torch, the library's calls, and the definition in 64 bits.

A case is a dict with an ``op``:

  append   rotary positions (one axis or several) applied to q and k, k and v written into the cache's pages
  prefill  causal attention of packed prompts with grouped heads
  decode   1..12 tokens of each sequence against the paged cache; sequences of a group share a prefix

``heads`` are query heads, ``kv_heads`` key/value heads.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
def listed():
    return [
        # one decode step of a full serving batch: 256 sequences, a token each, a tenth of the batch padded
        {"name": "append_batch", "op": "append", "io": "bf16", "seqs": 256, "tokens": 256, "heads": 32, "kv_heads": 4,
         "dim": 128, "rotary": 128, "axes": 1, "interleaved": False, "page": 64, "context": 511, "padded": 25},
        # the prefill batch of 8 ragged prompts, 32 query heads
        {"name": "append_prompt", "op": "append", "io": "bf16", "seqs": 8, "tokens": 32768, "heads": 32, "kv_heads": 8,
         "dim": 128, "rotary": 128, "axes": 1, "interleaved": False, "page": 64, "context": 0, "padded": 0},
        # prompts with images in full precision: positions in time, height and width, half of the channels rotated
        {"name": "append_axes", "op": "append", "io": "f32", "seqs": 5, "tokens": 5003, "heads": 16, "kv_heads": 2,
         "dim": 64, "rotary": 32, "axes": 3, "interleaved": True, "page": 16, "context": 70, "padded": 0},
        # one short prompt of a single user: latency counts
        {"name": "prefill_short", "op": "prefill", "io": "bf16", "seqs": 1, "tokens": 333, "heads": 16, "kv_heads": 4,
         "dim": 64},
        # the prefill batch of 8 ragged prompts
        {"name": "prefill_ragged", "op": "prefill", "io": "bf16", "seqs": 8, "tokens": 32768, "heads": 32,
         "kv_heads": 8, "dim": 128},
        # one long document
        {"name": "prefill_long", "op": "prefill", "io": "bf16", "seqs": 1, "tokens": 16384, "heads": 32, "kv_heads": 4,
         "dim": 128},
        # odd lengths in full precision, a key head per query head
        {"name": "prefill_odd", "op": "prefill", "io": "f32", "seqs": 3, "tokens": 3001, "heads": 8, "kv_heads": 8,
         "dim": 64},
        # one user's next token
        {"name": "decode_single", "op": "decode", "io": "bf16", "seqs": 1, "q_len": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "context": 4097, "groups": 0, "prefix": 0, "padded": 0},
        # a ragged serving batch that shares nothing
        {"name": "decode_batch", "op": "decode", "io": "bf16", "seqs": 64, "q_len": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "context": 8191, "groups": 0, "prefix": 0, "padded": 6},
        # accepting the drafted tokens of 64 sequences, up to 12 each
        {"name": "decode_verify", "op": "decode", "io": "bf16", "seqs": 64, "q_len": 12, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "context": 4095, "groups": 0, "prefix": 0, "padded": 0},
        # 64 samples of one long prompt
        {"name": "decode_shared", "op": "decode", "io": "bf16", "seqs": 64, "q_len": 1, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 64, "context": 511, "groups": 1, "prefix": 16384, "padded": 0},
        # 32 searches of 8 beams in full precision, each over its own prompt
        {"name": "decode_beams", "op": "decode", "io": "f32", "seqs": 256, "q_len": 1, "heads": 16, "kv_heads": 4,
         "dim": 64, "page": 32, "context": 127, "groups": 32, "prefix": 1000, "padded": 0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "prefill", "decode"])
    kv_heads, per, dim, io = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8]), rng.choice([64, 128]), rng.choice(["bf16", "f32"])
    c = {"op": op, "io": io, "heads": kv_heads * per, "kv_heads": kv_heads, "dim": dim}
    if op == "append":
        tokens = _log_int(rng, 1, max(1, int(8e7 / ((c["heads"] + 2 * kv_heads) * dim))))
        seqs = min(tokens, _log_int(rng, 1, 256))
        return {**c, "seqs": seqs, "tokens": tokens, "rotary": rng.choice([dim, dim, dim // 2, dim // 4 + 2, 0]),
                "axes": rng.choice([1, 1, 2, 3]), "interleaved": rng.random() < 0.5, "page": rng.choice([16, 32, 64, 128]),
                "context": _log_int(rng, 1, 512) - 1, "padded": rng.choice([0, 0, seqs // 10])}
    if op == "prefill":
        seqs = _log_int(rng, 1, 32)
        most = 3e11 if io == "bf16" else 3e10   # multiply-adds of a square of tokens
        tokens = _log_int(rng, 1, int(min(32768, math.sqrt(most * seqs / (c["heads"] * dim)))))
        return {**c, "seqs": min(seqs, tokens), "tokens": tokens}
    groups, q_len = rng.choice([0, 0, 1, 2, 7]), rng.choice([1, 1, 1, 2, 5, 12])
    seqs = max(groups, _log_int(rng, 1, 256))
    room = 2.5e8 / (kv_heads * dim)
    prefix = _log_int(rng, 16, max(17, int(min(32768, room / 2 / groups)))) if groups else 0
    return {**c, "seqs": seqs, "q_len": q_len, "page": rng.choice([16, 32, 64, 128, 256]),
            "context": _log_int(rng, 1, max(2, int(min(32768, room / seqs)))), "groups": groups, "prefix": prefix,
            "padded": rng.choice([0, 0, seqs // 10])}


# ---------------------------------------------------------------------------
# inputs
def _prompts(c):
    """Lengths that sum to ``tokens``, the longest about seven times the shortest, in order of length."""
    n = c["seqs"]
    weight = np.linspace(0.25, 1.75, n) if n > 1 else np.ones(1)
    ends = np.round(np.cumsum(weight) / weight.sum() * (c["tokens"] - n)).astype(np.int64)
    return np.diff(np.concatenate([[0], ends])) + 1


def _contexts(c):
    """Tokens before the step, spread evenly over 0..context (behind the prefix where there is one)."""
    n = c["seqs"]
    return c["prefix"] + np.round(np.linspace(c["context"] / n, c["context"], n)).astype(np.int64)


def _drafts(c):
    return 1 + np.arange(c["seqs"]) % c["q_len"]


def _groups(c):
    """Sequences of each group: the batch cut into near-equal parts."""
    return np.diff(np.round(np.linspace(0, c["seqs"], c["groups"] + 1)).astype(np.int64))


def _offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def _table(rs, need, page, shared=None):
    """Pages of each sequence in random order: (table [N, most], pages in all). ``shared``: for each sequence
    the group whose prefix pages it starts with and their count."""
    count = -(-need // page)
    own_pages = count - (shared[1] if shared is not None else 0)
    first = shared[2] if shared is not None else 0
    # as many for every order of the same lengths
    order = rs.permutation(first + int(need.sum() - page * (count - own_pages).sum()) // page + len(need) + 3)
    table = np.zeros((len(need), max(1, int(count.max()))), np.int32)
    at = first
    for n in range(len(need)):
        s = count[n] - own_pages[n]
        if s:
            g = shared[0][n]
            table[n, :s] = order[shared[3][g]: shared[3][g] + s]
        table[n, s: count[n]] = order[at: at + own_pages[n]]
        at += own_pages[n]
    return table, len(order)


def _frequencies(c):
    """f[a, i] of a base of 10000; with several axes the pairs are dealt out to them in turn."""
    half = c["rotary"] // 2
    f = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(1, half))
    out = torch.zeros(c["axes"], half, dtype=torch.float32)
    for i in range(half):
        out[i % c["axes"], i] = f[i]
    return out.cuda()


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    c, io = case, DTYPES[case["io"]]
    hq, hk, d = c["heads"], c["kv_heads"], c["dim"]
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=gen)  # noqa: E731
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    # heads attend over a few tokens or over many
    sharp = torch.exp(torch.empty(hq, 1, device="cuda").uniform_(math.log(0.5), math.log(4.0), generator=gen))
    s = {"case": dict(case)}
    if c["op"] == "decode":
        order = rs.permutation(c["seqs"])
        ctx, lens = _contexts(c)[order], rs.permutation(_drafts(c))
        shared = None
        if c["groups"]:
            sizes = _groups(c)
            of = np.repeat(np.arange(c["groups"]), sizes)
            whole = c["prefix"] // c["page"]   # the page in which the prefix ends is each sequence's own
            shared = (of, whole, c["groups"] * whole, np.arange(c["groups"]) * whole)
            s["group_offsets"] = dev(_offsets(sizes))
            s["prefix_lens"] = torch.full((c["groups"],), c["prefix"], dtype=torch.int32, device="cuda")
        table, pages = _table(rs, ctx + lens, c["page"], shared)
        if c["padded"]:
            ctx[rs.permutation(c["seqs"])[: c["padded"]]] = -1
        s["k_pages"] = rand(pages, hk, c["page"], d).to(io)
        s["v_pages"] = rand(pages, hk, c["page"], d).to(io)
        if c["groups"]:   # ... and holds the same last tokens of the prefix for all of a group
            rest = c["prefix"] % c["page"]
            for g in range(c["groups"] if rest else 0):
                rows = np.nonzero(of == g)[0]
                ids = dev(table[rows, whole].astype(np.int64))
                for p in (s["k_pages"], s["v_pages"]):
                    p[ids, :, :rest] = p[ids[:1], :, :rest].clone()
        cu = _offsets(lens)
        s["q"] = (rand(int(cu[-1]), hq, d) * sharp).to(io)
        s["cu"] = dev(cu) if c["q_len"] > 1 else None
        s["table"], s["context"] = dev(table), dev(ctx.astype(np.int32))
        s["host"] = (ctx.tolist(), cu.tolist())
        s["o"] = torch.zeros(int(cu[-1]), hq, d, dtype=io, device="cuda")
        return s
    lens = rs.permutation(_prompts(c))
    cu = _offsets(lens)
    s["cu"], s["host"] = dev(cu), cu.tolist()
    # one projection's output: q, k and v are views of its rows
    qkv = torch.cat([rand(c["tokens"], hq, d) * sharp, rand(c["tokens"], 2 * hk, d)], 1).to(io)
    s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq: hq + hk], qkv[:, hq + hk:]
    if c["op"] == "prefill":
        s["q"], s["k"] = s["q"].contiguous(), s["k"].contiguous()   # as the rotation leaves them
        return s
    ctx = np.round(np.linspace(0, c["context"], c["seqs"])).astype(np.int64)[rs.permutation(c["seqs"])]
    table, pages = _table(rs, ctx + lens, c["page"])
    if c["padded"]:
        ctx[rs.permutation(c["seqs"])[: c["padded"]]] = -1
    s["k_pages"] = torch.zeros(pages, hk, c["page"], d, dtype=io, device="cuda")
    s["v_pages"] = torch.zeros_like(s["k_pages"])
    s["table"], s["context"], s["freq"] = dev(table), dev(ctx.astype(np.int32)), _frequencies(c)
    s["positions"] = None
    if c["axes"] > 1:   # far into a video: frames on the first axis, patches on the others
        far = np.stack([np.arange(c["tokens"]) // (16 if a == 0 else 1) % (200000 if a == 0 else 4 + 60 * a)
                        for a in range(c["axes"])])
        s["positions"] = dev((far + rs.randint(0, 100000, (c["axes"], 1)) * (np.arange(c["axes"])[:, None] == 0)).astype(np.int32))
    s["q_out"] = torch.zeros(c["tokens"], hq, d, dtype=io, device="cuda")
    s["k_out"] = torch.zeros(c["tokens"], hk, d, dtype=io, device="cuda")
    return s


def work(case):
    c = case
    size = 2 if c["io"] == "bf16" else 4
    hq, hk, d = c["heads"], c["kv_heads"], c["dim"]
    if c["op"] == "append":   # k is written twice: into its page and for the prompt's own attention
        live = c["tokens"] * (c["seqs"] - c["padded"]) / c["seqs"]
        return {"bytes": live * (2 * hq + 5 * hk) * d * size, "flops": 3 * live * (hq + hk) * c["rotary"]}
    if c["op"] == "prefill":
        n = _prompts(c).astype(np.float64)
        return {"bytes": c["tokens"] * (2 * hq + 2 * hk) * d * size, "flops": float(4 * d * hq * (n * (n + 1) / 2).sum())}
    live = (c["seqs"] - c["padded"]) / c["seqs"]
    ctx, new = _contexts(c).astype(np.float64), _drafts(c).mean()
    tokens = c["groups"] * c["prefix"] + live * (ctx - c["prefix"] + new).sum()
    return {"bytes": (2 * tokens * hk + 2 * live * c["seqs"] * new * hq) * d * size,
            "flops": float(4 * d * hq * live * (new * (ctx + (new + 1) / 2)).sum())}


# ---------------------------------------------------------------------------
# plain forms
def _rotate(s, x):
    c = s["case"]
    half = c["rotary"] // 2
    if half == 0:
        return x
    cos, sin = s["cos"][:, None], s["sin"][:, None]
    y = x.float().clone()
    a, b = (y[..., 0: 2 * half: 2], y[..., 1: 2 * half: 2]) if c["interleaved"] else (y[..., :half], y[..., half: 2 * half])
    na, nb = a * cos - b * sin, b * cos + a * sin
    a.copy_(na)
    b.copy_(nb)
    return y.to(x.dtype)


def _plain_append(s):
    c, t = s["case"], torch.arange(s["case"]["tokens"], device="cuda")
    n = torch.searchsorted(s["cu"].long(), t, right=True) - 1
    context = s["context"].long()[n]
    live = context >= 0
    at = context + t - s["cu"].long()[n]
    pos = at[None] if s["positions"] is None else s["positions"]
    angle = (pos.double()[:, :, None] * s["freq"].double()[:, None]).sum(0)
    rotated = {**s, "cos": angle.cos().float(), "sin": angle.sin().float()}
    q, k = _rotate(rotated, s["q"]), _rotate(rotated, s["k"])
    s["q_out"].copy_(torch.where(live[:, None, None], q, s["q_out"]))
    s["k_out"].copy_(torch.where(live[:, None, None], k, s["k_out"]))
    kept = live.nonzero()[:, 0]
    n, at = n[kept], at[kept]
    page, row = s["table"].long()[n, at // c["page"]], at % c["page"]
    s["k_pages"][page, :, row] = k[kept]
    s["v_pages"][page, :, row] = s["v"][kept]
    return {"q": s["q_out"], "k": s["k_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _attend(q, k, v, first, scale):
    """q [t, HQ, D] against k, v [HKV, L, D], fp32; row i sees the tokens 0..first + i."""
    t, hq, d = q.shape
    hk, length = k.shape[:2]
    q = q.reshape(t, hk, hq // hk, d).permute(1, 2, 0, 3).reshape(hk, -1, d)
    x = torch.bmm(q, k.transpose(1, 2).contiguous()).mul_(scale).view(hk, hq // hk, t, length)
    seen = torch.arange(length, device="cuda") <= first + torch.arange(t, device="cuda")[:, None]
    x = x.masked_fill_(~seen, -math.inf)
    x = x.sub_(x.amax(3, keepdim=True)).exp_()
    total = x.sum(3, keepdim=True)
    o = torch.bmm(x.view(hk, -1, length), v).view(hk, hq // hk, t, d) / total
    return o.permute(2, 0, 1, 3).reshape(t, hq, d)


def _plain_prefill(s):
    c = s["case"]
    scale, out = 1.0 / math.sqrt(c["dim"]), torch.empty_like(s["q"])
    for t0, t1 in zip(s["host"][:-1], s["host"][1:]):
        k, v = (s[x][t0:t1].float().transpose(0, 1).contiguous() for x in ("k", "v"))
        rows = max(16, int(2e8) // (c["heads"] * (t1 - t0)))
        for a in range(t0, t1, rows):
            b = min(t1, a + rows)
            out[a:b] = _attend(s["q"][a:b].float(), k[:, : b - t0].contiguous(), v[:, : b - t0].contiguous(), a - t0, scale).to(out.dtype)
    return {"o": out}


def _plain_decode(s):
    c, (ctx, cu) = s["case"], s["host"]
    scale, d = 1.0 / math.sqrt(c["dim"]), c["dim"]
    for n, have in enumerate(ctx):
        if have < 0:
            continue
        t0, t1 = cu[n], cu[n + 1]
        pages = s["table"][n, : -(-(have + t1 - t0) // c["page"])].long()
        k, v = (s[x][pages].transpose(0, 1).reshape(c["kv_heads"], -1, d)[:, : have + t1 - t0].float() for x in ("k_pages", "v_pages"))
        s["o"][t0:t1] = _attend(s["q"][t0:t1].float(), k, v, have, scale).to(s["o"].dtype)
    return {"o": s["o"]}


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"append": _plain_append, "prefill": _plain_prefill, "decode": _plain_decode}[c["op"]](s)
    from gated_delta_rule_63_amd import gdr
    if c["op"] == "append":
        q, k = gdr.gdr_rope_append_paged(s["q"], s["k"], s["v"], s["freq"], k_pages=s["k_pages"], v_pages=s["v_pages"],
                                         page_table=s["table"], context_lens=s["context"], cu_seqlens=s["cu"],
                                         positions=s["positions"], interleaved=c["interleaved"], q_out=s["q_out"],
                                         k_out=s["k_out"])
        return {"q": q, "k": k, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if c["op"] == "prefill":
        return {"o": gdr.gdr_attn_prefill_fwd(s["q"], s["k"], s["v"], cu_seqlens=s["cu"])}
    shared = {"group_offsets": s["group_offsets"], "prefix_lens": s["prefix_lens"]} if c["groups"] else {}
    return {"o": gdr.gdr_attn_decode_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["context"],
                                           cu_seqlens=s["cu"], max_q_len=c["q_len"], o=s["o"], **shared)}


# ---------------------------------------------------------------------------
# the definition in 64 bits, a sequence and a head at a time
def _exact_append(s):
    c, cu = s["case"], s["host"]
    half, freq = c["rotary"] // 2, s["freq"].double().cpu().numpy()
    ctx, table = s["context"].cpu().numpy(), s["table"].cpu().numpy()
    pos = None if s["positions"] is None else s["positions"].cpu().numpy().astype(np.float64)
    wide = {x: s[x].double().cpu().numpy() for x in ("q", "k", "v", "q_out", "k_out", "k_pages", "v_pages")}
    for n in range(c["seqs"]):
        if ctx[n] < 0:
            continue
        a, b = cu[n], cu[n + 1]
        at = ctx[n] + np.arange(b - a)
        angle = np.zeros((b - a, half))
        for axis in range(c["axes"]):
            angle += np.outer(at if pos is None else pos[axis, a:b], freq[axis])
        turn = np.exp(1j * angle)[:, None, :]
        for x in ("q", "k"):
            y = wide[x][a:b].copy()
            even, odd = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c["interleaved"] else (slice(0, half), slice(half, 2 * half))
            z = (y[..., even] + 1j * y[..., odd]) * turn
            y[..., even], y[..., odd] = z.real, z.imag
            wide[x + "_out"][a:b] = y
        for i, j in enumerate(at):
            page, row = table[n, j // c["page"]], j % c["page"]
            wide["k_pages"][page, :, row] = wide["k_out"][a + i]
            wide["v_pages"][page, :, row] = wide["v"][a + i]
    return {"q": wide["q_out"], "k": wide["k_out"], "k_pages": wide["k_pages"], "v_pages": wide["v_pages"]}


def _exact_rows(q, k, v, first):
    """One head, 64 bits: q [t, D] against k, v [L, D]."""
    x = (q @ k.T) / math.sqrt(q.shape[1])
    t, length = x.shape
    future = torch.ones(t, length, dtype=torch.bool, device=x.device).triu(first + 1)
    x = torch.where(future, torch.full((), -math.inf, dtype=x.dtype, device=x.device), x)
    return torch.exp(x - torch.logsumexp(x, 1, keepdim=True)) @ v


def _exact_prefill(s):
    c = s["case"]
    out, per = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda"), c["heads"] // c["kv_heads"]
    for n in range(c["seqs"]):
        t0, t1 = s["host"][n], s["host"][n + 1]
        for h in range(c["heads"]):
            k, v = s["k"][t0:t1, h // per].double(), s["v"][t0:t1, h // per].double()
            for a in range(t0, t1, 4096):
                b = min(a + 4096, t1)
                out[a:b, h] = _exact_rows(s["q"][a:b, h].double(), k[: b - t0], v[: b - t0], a - t0)
    return {"o": out}


def _exact_decode(s):
    c, out = s["case"], s["o"].double()
    context, table, per = s["context"].cpu().numpy(), s["table"].cpu().numpy(), c["heads"] // c["kv_heads"]
    t1 = 0
    for n in range(c["seqs"]):
        t0, t1 = t1, t1 + 1 if s["cu"] is None else int(s["cu"][n + 1])
        if context[n] < 0:
            continue
        at = np.arange(context[n] + t1 - t0)
        page, row = torch.from_numpy(table[n, at // c["page"]]).long().cuda(), torch.from_numpy(at % c["page"]).cuda()
        for g in range(c["kv_heads"]):
            k, v = s["k_pages"][page, g, row].double(), s["v_pages"][page, g, row].double()
            for h in range(g * per, (g + 1) * per):
                out[t0:t1, h] = _exact_rows(s["q"][t0:t1, h].double(), k, v, int(context[n]))
    return {"o": out}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "prefill": _exact_prefill, "decode": _exact_decode}[case["op"]](s)
