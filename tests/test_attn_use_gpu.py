"""Full attention of serving as programs use it: the operators together, captured, on other streams, at the ends of
their ranges.  Tolerances: _attn.py."""
import numpy as np
import pytest
import torch

from _attn import TORCH, check_attention, normal
from _dev import f64, to_dev, to_host
from gated_delta_rule_63_amd import gdr
from oracle import attn, beam
from test_attn_gpu import _decode_call, _decode_inputs, _freq, _rotated_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io,D,interleaved", [("f32", 64, True), ("bf16", 128, False)])
def test_a_layer_from_prompts_to_forked_samples(io, D, interleaved):
    """Three prompts with positions on two axes are rotated, stored and attended to; each goes on as four samples that
    share its whole pages (the page in which it ends is copied), for five steps of one to three tokens.  Every output is
    checked against the oracle on the whole sequence."""
    r = np.random.default_rng(51)
    HQ, HK, page, width = 8, 2, 16, 12
    lens, R = [70, 33, 100], D
    freq = _freq(2, R // 2)
    num = 120
    kp = torch.full((num, HK, page, D), float("nan"), dtype=TORCH[io], device="cuda")
    vp = kp.clone()
    free = list(r.permutation(num))

    def project(T):
        t, w = normal(r, (T, HQ + 2 * HK, D), io)
        return (t[:, :HQ], t[:, HQ:HQ + HK], t[:, HQ + HK:]), (w[:, :HQ], w[:, HQ:HQ + HK], w[:, HQ + HK:])

    def positions(n):
        return r.integers(0, 100000, (2, n)).astype(np.int32)

    # prompts
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    table = np.full((3, width), -1, np.int32)
    for n, L in enumerate(lens):
        for i in range(-(-L // page)):
            table[n, i] = free.pop()
    (q, k, v), (qw, kw, vw) = project(int(cu[-1]))
    pos = positions(int(cu[-1]))
    qr, kr = gdr.gdr_rope_append_paged(q, k, v, to_dev(freq), k_pages=kp, v_pages=vp, page_table=to_dev(table), cu_seqlens=to_dev(cu),
                                       positions=to_dev(pos), interleaved=interleaved)
    theta = attn.angles(pos, freq)
    _rotated_close(f64(qr), qw, theta, interleaved, io, "q")
    _rotated_close(f64(kr), kw, theta, interleaved, io, "k")
    o, lse = gdr.gdr_attn_prefill_fwd(qr, kr, v, cu_seqlens=to_dev(cu), output_lse=True)
    ref = attn.prefill(f64(qr), f64(kr), vw, cu, 1 / np.sqrt(D))
    check_attention(f64(o), f64(lse), ref, io, np.arange(int(cu[-1])), "prompts")
    # the prompts' last rows come out of the cache as well
    last = to_dev(np.array(lens, np.int32) - 1)
    o1 = gdr.gdr_attn_decode_paged(qr[to_dev(cu[1:] - 1).long()].contiguous(), kp, vp, to_dev(table), last)
    check_attention(f64(o1), None, {x: ref[x][cu[1:] - 1] for x in ref}, io, np.arange(3), "last rows")

    # four samples each
    keys = [f64(kr)[cu[n]:cu[n + 1]] for n in range(3) for _ in range(4)]
    values = [vw[cu[n]:cu[n + 1]] for n in range(3) for _ in range(4)]
    forks = np.full((12, width), -1, np.int32)
    for s in range(12):
        n, whole = s // 4, lens[s // 4] // page
        forks[s, :whole] = table[n, :whole]
        if lens[n] % page:
            forks[s, whole] = table[n, whole] if s % 4 == 0 else free.pop()
            if s % 4:
                for p in (kp, vp):
                    p[int(forks[s, whole])] = p[int(table[n, whole])]
    ctx = np.repeat(lens, 4).astype(np.int32)
    offsets, prefix = to_dev(np.array([0, 4, 8, 12], np.int32)), to_dev(np.array(lens, np.int32))
    for step in range(5):
        m = 1 + r.integers(0, 3, 12)
        m[:] = m if step else 1
        cu = np.concatenate([[0], np.cumsum(m)]).astype(np.int32)
        for s in range(12):
            for i in range(-(-int(ctx[s] + m[s]) // page)):
                if forks[s, i] < 0:
                    forks[s, i] = free.pop()
        (q, k, v), (qw, kw, vw) = project(int(cu[-1]))
        pos = positions(int(cu[-1]))
        cu_arg = to_dev(cu) if step else None      # one token each
        qr, kr = gdr.gdr_rope_append_paged(q, k, v, to_dev(freq), k_pages=kp, v_pages=vp, page_table=to_dev(forks),
                                           context_lens=to_dev(ctx), cu_seqlens=cu_arg, positions=to_dev(pos), interleaved=interleaved)
        o, lse = gdr.gdr_attn_decode_paged(qr, kp, vp, to_dev(forks), to_dev(ctx), cu_seqlens=cu_arg, max_q_len=3 if step else 1,
                                           group_offsets=offsets, prefix_lens=prefix, output_lse=True)
        alone = gdr.gdr_attn_decode_paged(qr, kp, vp, to_dev(forks), to_dev(ctx), cu_seqlens=cu_arg, max_q_len=3 if step else 1)
        o, lse, alone, qf, kf = f64(o), f64(lse), f64(alone), f64(qr), f64(kr)
        for s in range(12):
            a, b = cu[s], cu[s + 1]
            keys[s], values[s] = np.concatenate([keys[s], kf[a:b]]), np.concatenate([values[s], vw[a:b]])
            L = len(keys[s])
            whole_q = np.zeros((L, HQ, D))
            whole_q[L - m[s]:] = qf[a:b]
            ref = attn.prefill(whole_q, keys[s], values[s], [0, L], 1 / np.sqrt(D))
            ref = {x: ref[x][L - m[s]:] for x in ref}
            check_attention(o[a:b], lse[a:b], ref, io, np.arange(m[s]), f"step {step} sample {s}")
            check_attention(alone[a:b], None, ref, io, np.arange(m[s]), f"step {step} sample {s} alone")
        ctx = ctx + m.astype(np.int32)


def test_beams_share_their_prompt():
    """A step of beam search over the cache: attention of the beams, the best candidates, and the parents' own pages
    copied to their children's (slots of pages, as gdr_beam_reorder moves any pool)."""
    B, W, D, HQ, HK, page, prompt = 2, 4, 64, 4, 1, 16, 48
    r = np.random.default_rng(52)
    own, shared = 2, prompt // page                         # pages of a beam, of a prompt
    num = B * shared + B * W * own
    (kp, kw), (vp, vw) = normal(r, (num, HK, page, D), "f32"), normal(r, (num, HK, page, D), "f32")
    slots = (np.arange(B * W).reshape(B, W)).astype(np.int32)
    ctx = np.full(B * W, prompt + 9, np.int32)

    def table(slots):
        t = np.empty((B * W, shared + own), np.int32)
        for b in range(B):
            for w in range(W):
                t[b * W + w, :shared] = b * shared + np.arange(shared)
                t[b * W + w, shared:] = B * shared + slots[b, w] * own + np.arange(own)
        return t

    args = dict(group_offsets=to_dev(np.arange(0, B * W + 1, W, dtype=np.int32)), prefix_lens=to_dev(np.full(B, prompt, np.int32)))
    q, qw = normal(r, (B * W, HQ, D), "f32")
    o = gdr.gdr_attn_decode_paged(q, kp, vp, to_dev(table(slots)), to_dev(ctx), **args)
    ref = attn.decode(qw, np.arange(B * W + 1), ctx, kw, vw, table(slots), 1 / np.sqrt(D))
    check_attention(f64(o), None, ref, "f32", np.arange(B * W))
    logits, lw = normal(r, (B, W, 500), "f32")
    scores, sw = normal(r, (B, W), "f32")
    _, parents, tokens = gdr.gdr_beam_select(logits, scores, W)
    want = beam.select(lw, sw, W)
    assert np.array_equal(to_host(parents), want[1]) and np.array_equal(to_host(tokens), want[2])
    new = None
    for p, w in ((kp, kw), (vp, vw)):
        pool = p[B * shared:].view(B * W, own, HK, page, D)
        new = gdr.gdr_beam_reorder(pool, to_dev(slots), parents)
        _, moves = beam.reorder(slots, want[1], B * W)
        before = w.copy()
        for a, b in moves:
            w[B * shared + b * own: B * shared + (b + 1) * own] = before[B * shared + a * own: B * shared + (a + 1) * own]
    new = to_host(new)
    o = gdr.gdr_attn_decode_paged(q, kp, vp, to_dev(table(new)), to_dev(ctx), **args)
    ref = attn.decode(qw, np.arange(B * W + 1), ctx, kw, vw, table(new), 1 / np.sqrt(D))
    check_attention(f64(o), None, ref, "f32", np.arange(B * W))


# ---------------------------------------------------------------------------
def _step(io="bf16", groups=True):
    """Everything that one decode step of a layer reads and writes, with a call that fills it in."""
    d = _decode_inputs(61, io, 128, 8, 2, [2, 1, 3, 2, 1, 2], [130, 140, 135, 300, 5, -1], 16, groups=[(3, 128), (1, 0)] if groups else None)
    T = int(d["cu"][-1])
    r = np.random.default_rng(62)
    q, k, v = normal(r, (T, 8, 128), io)[0], normal(r, (T, 2, 128), io)[0], normal(r, (T, 2, 128), io)[0]
    t = dict(cu=to_dev(d["cu"]), ctx=to_dev(d["ctx"]), table=to_dev(d["table"]), freq=to_dev(_freq(1, 64)), q=q, k=k, v=v,
             kp=d["k"].clone(), vp=d["v"].clone(), qo=torch.zeros_like(q), ko=torch.zeros_like(k), o=torch.zeros_like(q),
             lse=torch.zeros(T, 8, device="cuda"), po=torch.zeros_like(q))
    more = dict(group_offsets=to_dev(d["offsets"]), prefix_lens=to_dev(d["prefix"])) if groups else {}
    need = gdr.gdr_attn_workspace_size(q, t["kp"], 6, 3, 2 if groups else 0)
    t["ws"] = torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda")

    def call(t, stream=None):
        gdr.gdr_rope_append_paged(t["q"], t["k"], t["v"], t["freq"], k_pages=t["kp"], v_pages=t["vp"], page_table=t["table"],
                                  context_lens=t["ctx"], cu_seqlens=t["cu"], q_out=t["qo"], k_out=t["ko"], stream=stream)
        gdr.gdr_attn_decode_paged(t["qo"], t["kp"], t["vp"], t["table"], t["ctx"], cu_seqlens=t["cu"], max_q_len=3, o=t["o"],
                                  lse=t["lse"], workspace=t["ws"], stream=stream, **more)
        gdr.gdr_attn_prefill_fwd(t["qo"], t["ko"], t["v"], cu_seqlens=t["cu"], o=t["po"], stream=stream)

    return t, call


OUTS = ("kp", "vp", "qo", "ko", "o", "lse", "po")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("groups", [False, True])
def test_calls_are_repeatable_and_captured(groups, io):
    t, call = _step(io, groups)
    call(t)
    torch.cuda.synchronize()
    want = {n: t[n].clone() for n in OUTS}
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call(t)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call(t)
    for i in range(4):
        for n in ("o", "lse", "po"):
            t[n].fill_(3.0)
        t["ws"].fill_(17 * i)                       # its contents need not be kept
        if i == 2:                                  # other inputs, the same graph; an eager call between the replays
            t["q"].mul_(0.5)
            t["ctx"][0] = 100
            call(t)
            torch.cuda.synchronize()
            want = {n: t[n].clone() for n in OUTS}
            t["o"].zero_()
        g.replay()
        torch.cuda.synchronize()
        for n in OUTS:
            live = t[n]
            ref = want[n]
            if n in ("o", "lse", "po") and i != 2:  # rows of the padded sequence keep what was there
                pad = slice(int(to_host(t["cu"])[5]), int(to_host(t["cu"])[6]))
                if n != "po":
                    assert bool((live[pad] == 3.0).all())
                live, ref = live[: pad.start], ref[: pad.start]
            elif n in ("o", "lse"):
                live, ref = live[: int(to_host(t["cu"])[5])], ref[: int(to_host(t["cu"])[5])]
            assert torch.equal(live, ref), (i, n)


def test_two_calls_at_once_on_streams_of_their_own():
    ts, calls = zip(*[_step("bf16", g) for g in (True, False, True)])
    for t, call in zip(ts, calls):
        call(t)
    torch.cuda.synchronize()
    want = [{n: t[n].clone() for n in OUTS} for t in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    for rep in range(3):
        for t in ts:
            t["ws"].fill_(rep)
        torch.cuda.synchronize()
        for _ in range(4):
            for t, call, s in zip(ts, calls, streams):
                call(t, stream=s)
        torch.cuda.synchronize()
        for t, w in zip(ts, want):
            for n in OUTS:
                assert torch.equal(t[n], w[n]), n


def test_a_workspace_of_the_bindings_on_another_stream():
    d = _decode_inputs(63, "bf16", 64, 4, 2, [1] * 8, [200 + i for i in range(8)], 16)
    want = _decode_call(d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _decode_call(d, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


# ---------------------------------------------------------------------------
def test_pages_behind_four_gigabytes():
    """The pages in use lie at both ends of caches of 5 GiB each."""
    HK, page, D = 2, 64, 128
    num = (5 << 30) // (HK * page * D * 2)
    kp = torch.zeros(num, HK, page, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    r = np.random.default_rng(71)
    table = np.array([[num - 1, 0, num - 2, num // 2 + 1], [num - 3, num - 4, 1, 2]], np.int32)
    lens = [200, 150]
    cu = np.array([0, 200, 350], np.int32)
    (q, qw), (k, kw), (v, vw) = normal(r, (350, 4, D), "bf16"), normal(r, (350, HK, D), "bf16"), normal(r, (350, HK, D), "bf16")
    qr, kr = gdr.gdr_rope_append_paged(q, k, v, k_pages=kp, v_pages=vp, page_table=to_dev(table), cu_seqlens=to_dev(cu))
    assert torch.equal(qr, q) and torch.equal(kr, k)       # no rotation: copied
    for n, L in enumerate(lens):
        for t in (0, 63, 64, L - 1):
            assert torch.equal(kp[int(table[n, t // page]), :, t % page], k[cu[n] + t])
            assert torch.equal(vp[int(table[n, t // page]), :, t % page], v[cu[n] + t])
    last = torch.tensor([199, 349], device="cuda")
    o, lse = gdr.gdr_attn_decode_paged(qr[last].contiguous(), kp, vp, to_dev(table), to_dev(np.array(lens, np.int32) - 1), output_lse=True)
    ref = attn.prefill(qw, kw, vw, cu, 1 / np.sqrt(D))
    check_attention(f64(o), f64(lse), {x: ref[x][[199, 349]] for x in ref}, "bf16", np.arange(2))


def test_rows_behind_four_gigabytes():
    """Tokens 64 KiB apart: the batch's last rows lie behind 2^32 bytes."""
    T, D = 70000, 64
    t = torch.zeros(T, 1 << 15, dtype=torch.bfloat16, device="cuda")
    r = np.random.default_rng(72)
    (x, xw) = normal(r, (300, 4, D), "bf16")
    t[-300:, :256] = x.view(300, 256)
    rows = t[:, :256].view(T, 4, D)
    q, k, v = rows[:, :2], rows[:, 2:3], rows[:, 3:4]
    cu = np.array([0, 5, T - 300, T - 299, T], np.int32)
    o = gdr.gdr_attn_prefill_fwd(q, k, v, cu_seqlens=to_dev(cu))
    ref = attn.prefill(xw[:, :2], xw[:, 2:3], xw[:, 3:4], [0, 1, 300], 1 / 8)
    check_attention(f64(o[-300:]), None, ref, "bf16", np.arange(300))
    assert bool((o[:5] == 0).all())
    qo, ko = gdr.gdr_rope_append_paged(q, k, inv_freq=to_dev(_freq(1, 32)), cu_seqlens=to_dev(cu))
    pos = np.concatenate([[0], np.arange(299)])[None]
    _rotated_close(f64(qo[-300:]), xw[:, :2], attn.angles(pos, _freq(1, 32)), False, "bf16", "q")
    _rotated_close(f64(ko[-300:]), xw[:, 2:3], attn.angles(pos, _freq(1, 32)), False, "bf16", "k")


def test_most_sequences():
    """65535 sequences, a token or none each, groups over some of them: against the same call in parts of the batch."""
    N, D = 65535, 64
    r = np.random.default_rng(73)
    lens, ctx = r.integers(0, 2, N), r.integers(-1, 40, N)
    ctx[:300] = 47
    lens[:300] = 1
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    table = r.integers(0, 500, (N, 3)).astype(np.int32)
    table[:300, :2] = table[0, :2]
    (q, qw), (k, kw), (v, vw) = normal(r, (int(cu[-1]), 2, D), "f32"), normal(r, (500, 1, 16, D), "f32"), normal(r, (500, 1, 16, D), "f32")
    o = torch.full((int(cu[-1]), 2, D), 7.0, device="cuda")
    gdr.gdr_attn_decode_paged(q, k, v, to_dev(table), to_dev(ctx.astype(np.int32)), cu_seqlens=to_dev(cu), o=o,
                              group_offsets=to_dev(np.array([0, 300], np.int32)), prefix_lens=to_dev(np.array([32], np.int32)))
    plain = torch.full_like(o, 7.0)
    gdr.gdr_attn_decode_paged(q, k, v, to_dev(table), to_dev(ctx.astype(np.int32)), cu_seqlens=to_dev(cu), o=plain)
    some = np.unique(np.concatenate([np.arange(320), r.integers(0, N, 300), [N - 1]]))
    for out in (o, plain):
        out = f64(out)
        for n in some:
            a, b = cu[n], cu[n + 1]
            if a == b:
                continue
            if ctx[n] < 0:
                assert (out[a] == 7.0).all()
                continue
            ref = attn.decode(qw[a:b], [0, 1], ctx[n:n + 1], kw, vw, table[n:n + 1], 1 / 8)
            check_attention(out[a:b], None, ref, "f32", np.arange(1), f"sequence {n}")
    # prompts of as many sequences
    (q, qw), (k, kw), (v, vw) = normal(r, (int(cu[-1]), 2, D), "f32"), normal(r, (int(cu[-1]), 1, D), "f32"), normal(r, (int(cu[-1]), 1, D), "f32")
    o = gdr.gdr_attn_prefill_fwd(q, k, v, cu_seqlens=to_dev(cu))
    # one token sees itself: w v / w, where w v and 1 / w and their product are rounded, by 2^-24, 2^-23 and 2^-24 at most
    assert bool(((o - v).abs() <= v.abs() * 2.0 ** -22).all())


@pytest.mark.parametrize("HQ,HK", [(256, 1), (300, 300), (1000, 8)])
def test_many_heads(HQ, HK):
    """More rows of a key head than a block's, more key heads than a launch's workgroups."""
    d = _decode_inputs(HQ, "bf16", 64, HQ, HK, [2, 1], [70, 20], 16)
    o, lse = _decode_call(d, output_lse=True)
    ref = attn.decode(d["qw"], d["cu"], d["ctx"], d["kw"], d["vw"], d["table"], 1 / 8)
    check_attention(f64(o), f64(lse), ref, "bf16", np.arange(3))
    d = _decode_inputs(HQ + 1, "bf16", 64, HQ, HK, [1] * 3, [70, 65, 90], 16, groups=[(3, 64)])
    ref = attn.decode(d["qw"], d["cu"], d["ctx"], d["kw"], d["vw"], d["table"], 1 / 8)
    check_attention(f64(_decode_call(d)), None, ref, "bf16", np.arange(3))
    r = np.random.default_rng(HQ)
    (q, qw), (k, kw), (v, vw) = normal(r, (40, HQ, 64), "bf16"), normal(r, (40, HK, 64), "bf16"), normal(r, (40, HK, 64), "bf16")
    o = gdr.gdr_attn_prefill_fwd(q, k, v)
    check_attention(f64(o), None, attn.prefill(qw, kw, vw, [0, 40], 1 / 8), "bf16", np.arange(40))
    qo, ko = gdr.gdr_rope_append_paged(q, k, inv_freq=to_dev(_freq(1, 32)))
    _rotated_close(f64(qo), qw, attn.angles(np.arange(40)[None], _freq(1, 32)), False, "bf16", "q")
    _rotated_close(f64(ko), kw, attn.angles(np.arange(40)[None], _freq(1, 32)), False, "bf16", "k")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,HQ,HK", [(700, 4, 2), (1500, 16, 4), (1400, 64, 8), (1000, 8, 8), (1300, 24, 8), (2000, 16, 4)])
def test_every_size_of_row_blocks(T, HQ, HK, D, io):
    """The three ways to cut a batch into workgroups, with one tile in the LDS or two: the first and the last head."""
    r = np.random.default_rng(T + D)
    (q, qw), (k, kw), (v, vw) = normal(r, (T, HQ, D), io), normal(r, (T, HK, D), io), normal(r, (T, HK, D), io)
    cu = np.array([0, T // 3, T // 3, T - 5], np.int32)
    o = torch.full((T, HQ, D), 7.0, dtype=TORCH[io], device="cuda")
    gdr.gdr_attn_prefill_fwd(q, k, v, cu_seqlens=to_dev(cu), o=o)
    assert bool((o[T - 5:] == 7.0).all())
    o = f64(o)
    for h in (0, HQ - 1):
        ref = attn.prefill(qw[:, h:h + 1], kw[:, h * HK // HQ][:, None], vw[:, h * HK // HQ][:, None], cu, 1 / np.sqrt(D))
        check_attention(o[:, h:h + 1], None, ref, io, np.arange(T - 5), f"head {h}")


def test_appending_more_tokens_than_a_launch_takes():
    T = (1 << 23) + 1000
    q, k = torch.empty(T, 1, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(T, 1, 64, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, (1 << 22) - 1, 1 << 22, (1 << 23) - 1, 1 << 23, T - 1], device="cuda")
    x, w = normal(np.random.default_rng(74), (len(at), 2, 64), "bf16")
    q[at], k[at] = x[:, :1], x[:, 1:]
    for half in (1, 32):     # one pair takes the kernel for any number of channels
        qo, ko = gdr.gdr_rope_append_paged(q, k, inv_freq=to_dev(_freq(1, half)))
        theta = attn.angles(to_host(at)[None], _freq(1, half))
        _rotated_close(f64(qo[at]), w[:, :1], theta, False, "bf16", "q")
        _rotated_close(f64(ko[at]), w[:, 1:], theta, False, "bf16", "k")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_appending_past_the_caches(io, interleaved):
    """A batch that no cache holds, stored as one call and as two of half the tokens."""
    r = np.random.default_rng(77)
    T, HQ, HK, D, page = 16000 if io == "bf16" else 8000, 16, 8, 128, 16
    (q, _), (k, _), (v, _) = normal(r, (T, HQ, D), io), normal(r, (T, HK, D), io), normal(r, (T, HK, D), io)
    need = T // page + 1
    table, freq = r.permutation(need).astype(np.int32)[None], to_dev(_freq(1, D // 2))
    got = []
    for parts in (1, 2):
        kp, vp = torch.zeros(need, HK, page, D, dtype=TORCH[io], device="cuda"), torch.zeros(need, HK, page, D, dtype=TORCH[io], device="cuda")
        outs = []
        for i in range(parts):
            a, n = i * T // parts, T // parts
            outs.append(gdr.gdr_rope_append_paged(q[a:a + n], k[a:a + n], v[a:a + n], freq, k_pages=kp, v_pages=vp, page_table=to_dev(table),
                                                  cu_seqlens=to_dev(np.array([0, n], np.int32)), context_lens=to_dev(np.array([a], np.int32)),
                                                  interleaved=interleaved))
        got.append([kp, vp] + [torch.cat(x) for x in zip(*outs)])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    some = [0, 1, T // 2, T - 1]
    _rotated_close(f64(got[0][2][some]), f64(q[some]), attn.angles(np.array([some]), _freq(1, D // 2)), interleaved, io, "q")


def test_joining_more_rows_than_a_launch_has_waves():
    """640000 rows with a prefix: their kernel's launch has half a wave for 524288."""
    N = 20000
    d = _decode_inputs(75, "f32", 64, 32, 1, [1] * N, [20 + n % 3 for n in range(N)], 16, groups=[(N, 16)])
    o, lse = _decode_call(d, output_lse=True)
    rows = np.unique(np.concatenate([[0, N // 2, N - 1], np.random.default_rng(75).integers(0, N, 500)]))
    for n in rows:
        ref = attn.decode(d["qw"][n:n + 1], [0, 1], d["ctx"][n:n + 1], d["kw"], d["vw"], d["table"][n:n + 1], 1 / 8)
        check_attention(f64(o[n:n + 1]), f64(lse[n:n + 1]), ref, "f32", np.arange(1), f"sequence {n}")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len", [1, 3])
def test_infinities_that_are_seen(q_len, D, io):
    """An infinite value of the last key that a row sees: that channel is infinite, the others are as ever; so with one in
    a prefix."""
    lens = [1, 2, 15, 16, 17, 33, 63, 64, 65, 100, 127, 128, 129]
    cu = np.concatenate([[0], np.cumsum([q_len] * len(lens))])
    for groups in (None, [(len(lens), 0)], [(5, 48)]):
        ctx = [max(x, 48) if groups and groups[0][1] else x for x in lens]
        d = _decode_inputs(76, io, D, 4, 2, [q_len] * len(lens), ctx, 16, groups=groups)
        for n, c in enumerate(ctx):
            last = c + q_len - 1
            page = int(d["table"][n][last // 16])
            d["v"][page, 1, last % 16, 5], d["vw"][page, 1, last % 16, 5] = float("inf"), 0.0
        if groups and groups[0][1]:
            page = int(d["table"][0][2])
            d["v"][page, 0, 15, 7], d["vw"][page, 0, 15, 7] = -float("inf"), 0.0
        o = f64(_decode_call(d))
        want = np.zeros(o.shape)
        want[cu[1:] - 1, 2:, 5] = np.inf
        if groups and groups[0][1]:
            want[: cu[5], :2, 7] = -np.inf
        assert np.array_equal(np.where(np.isinf(want), want, 0), np.where(np.isfinite(o), 0, o))
        ref = attn.decode(d["qw"], d["cu"], d["ctx"], d["kw"], d["vw"], d["table"], 1 / np.sqrt(D))
        fine = np.where(np.isinf(want), ref["o"], o)
        check_attention(fine, None, ref, io, np.arange(len(o)))


def test_nothing_to_do():
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    kp, vp = z(2, 1, 16, 64), z(2, 1, 16, 64)
    assert gdr.gdr_attn_prefill_fwd(z(0, 2, 64), z(0, 1, 64), z(0, 1, 64), cu_seqlens=i(4)).shape == (0, 2, 64)
    assert gdr.gdr_attn_decode_paged(z(0, 2, 64), kp, vp, i(0, 4), i(0)).shape == (0, 2, 64)
    assert gdr.gdr_attn_decode_paged(z(0, 2, 64), kp, vp, i(3, 4), i(3), cu_seqlens=i(4)).shape == (0, 2, 64)
    q, k = gdr.gdr_rope_append_paged(z(0, 2, 64), z(0, 1, 64), z(0, 1, 64), z(32), k_pages=kp, v_pages=vp, page_table=i(0, 4), context_lens=i(0))
    assert q.shape == (0, 2, 64) and k.shape == (0, 1, 64)
    odd = torch.zeros(4, 64, 2, device="cuda").transpose(1, 2)[:0]      # strides of a tensor without tokens mean nothing
    assert gdr.gdr_attn_prefill_fwd(odd, odd, odd, cu_seqlens=i(4)).shape == (0, 2, 64)
    # all padded; a table without columns: rows see nothing
    o = gdr.gdr_attn_decode_paged(torch.ones(3, 2, 64, device="cuda"), kp, vp, i(3, 4), i(3) - 1, o=z(3, 2, 64) + 7)
    assert bool((o == 7).all())
    o, lse = gdr.gdr_attn_decode_paged(torch.ones(3, 2, 64, device="cuda"), kp, vp, i(3, 0), i(3), o=z(3, 2, 64) + 7, output_lse=True)
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())
    o, lse = gdr.gdr_attn_decode_paged(torch.ones(3, 2, 64, device="cuda"), kp, vp, i(3, 0), i(3), o=z(3, 2, 64) + 7, output_lse=True,
                                       group_offsets=i(2) + torch.tensor([0, 3], dtype=torch.int32, device="cuda"), prefix_lens=i(1) + 16)
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())


def test_binding_refusals():
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, kp = z(6, 4, 64), z(6, 2, 64), z(3, 2, 16, 64)
    for bad in (lambda: gdr.gdr_attn_prefill_fwd(q, k, z(6, 2, 128)), lambda: gdr.gdr_attn_prefill_fwd(q, k[:5], k[:5]),
                lambda: gdr.gdr_attn_prefill_fwd(q, z(6, 64, 2).transpose(1, 2), k), lambda: gdr.gdr_attn_prefill_fwd(z(4, 6, 64).transpose(0, 1), k, k),
                lambda: gdr.gdr_attn_prefill_fwd(q, k, k, lse=z(6, 4).float()[:, :3]),
                lambda: gdr.gdr_attn_decode_paged(q, kp, z(3, 2, 32, 64), i(6, 1), i(6)), lambda: gdr.gdr_attn_decode_paged(q, kp, kp, i(5, 1), i(6)),
                lambda: gdr.gdr_attn_decode_paged(q, kp, kp, i(6, 1), i(6), group_offsets=i(2)),
                lambda: gdr.gdr_attn_decode_paged(q, kp, kp, i(6, 1), i(6), group_offsets=i(2), prefix_lens=i(3)),
                lambda: gdr.gdr_rope_append_paged(q, k, inv_freq=z(2, 32).float()[:, :16]),
                lambda: gdr.gdr_rope_append_paged(q, k, inv_freq=z(3, 32).float(), positions=i(2, 6)),
                lambda: gdr.gdr_rope_append_paged(q, k, k, k_pages=kp, v_pages=kp),
                lambda: gdr.gdr_rope_append_paged(q, k[:4])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: gdr.gdr_attn_prefill_fwd(q, k.float(), k), lambda: gdr.gdr_attn_decode_paged(q, kp.float(), kp.float(), i(6, 1), i(6)),
                lambda: gdr.gdr_attn_decode_paged(q, kp, kp, i(6, 1).long(), i(6)), lambda: gdr.gdr_rope_append_paged(q, k, inv_freq=z(32)),
                lambda: gdr.gdr_attn_prefill_fwd(q.half(), k.half(), k.half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: gdr.gdr_attn_prefill_fwd(z(6, 4, 96), z(6, 2, 96), z(6, 2, 96)), lambda: gdr.gdr_attn_decode_paged(q, z(3, 2, 24, 64), z(3, 2, 24, 64), i(6, 1), i(6)),
                lambda: gdr.gdr_attn_decode_paged(q, kp, kp, i(6, 1), i(6), max_q_len=13), lambda: gdr.gdr_attn_prefill_fwd(q, z(6, 3, 64), z(6, 3, 64)),
                lambda: gdr.gdr_attn_decode_paged(q, kp, kp, i(6, 1), i(6), workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")),
                lambda: gdr.gdr_rope_append_paged(q, k, inv_freq=z(3, 32).float()), lambda: gdr.gdr_rope_append_paged(q, k, inv_freq=z(40).float()),
                lambda: gdr.gdr_attn_prefill_fwd(z(7 * 256)[4:4 + 6 * 256].view(6, 4, 64), k, k)):
        with pytest.raises(gdr.GdrError):
            bad()
