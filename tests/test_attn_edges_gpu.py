"""Full attention of serving at the edges of its kernels' bookkeeping, against the fp64 oracle (tolerances: _attn.py)."""
import numpy as np
import pytest
import torch

from _attn import HALF, TORCH, check_attention, normal
from _dev import f64, to_dev
from gated_delta_rule_63_amd import gdr
from oracle import attn
from test_attn_gpu import _decode_call, _decode_inputs

pytestmark = pytest.mark.gpu


def _repeated(seed, io, D, HQ, HK, lens, ctx, pages=12, page=16, groups=None):
    """Inputs of a paged step whose sequences name the same few pages many times (groups: [(sequences, pages)] whose first
    pages are the same)."""
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    ctx = np.asarray(ctx, np.int32)
    most = -(-int((ctx + np.asarray(lens)).max()) // page)
    table = r.integers(0, pages, (len(lens), most)).astype(np.int32)
    d = dict(cu=cu, ctx=ctx, table=table, io=io, D=D, HQ=HQ, HK=HK, page=page, lens=list(lens), args={})
    if groups is not None:
        offsets = np.concatenate([[0], np.cumsum([n for n, _ in groups])]).astype(np.int32)
        for g, (_, shared) in enumerate(groups):
            table[offsets[g]: offsets[g + 1], :shared] = table[offsets[g], :shared]
        d["args"] = dict(group_offsets=to_dev(offsets), prefix_lens=to_dev(np.array([p * page for _, p in groups], np.int32)))
    d["q"], d["qw"] = normal(r, (int(cu[-1]), HQ, D), io, 2.0)
    (d["k"], d["kw"]), (d["v"], d["vw"]) = normal(r, (pages, HK, page, D), io), normal(r, (pages, HK, page, D), io)
    return d


def _run(d, **kw):
    T = int(d["cu"][-1])
    o = torch.full((T, d["HQ"], d["D"]), 7.0, dtype=TORCH[d["io"]], device="cuda")
    lse = torch.full((T, d["HQ"]), 7.0, device="cuda")
    gdr.gdr_attn_decode_paged(d["q"], d["k"], d["v"], to_dev(d["table"]), to_dev(d["ctx"]), cu_seqlens=to_dev(d["cu"]),
                              max_q_len=max(d["lens"]), o=o, lse=lse, **d["args"], **kw)
    torch.cuda.synchronize()
    return f64(o), f64(lse)


def _check_key_heads(d, heads, what=""):
    """every row of the query heads of some key heads"""
    o, lse = _run(d)
    per = d["HQ"] // d["HK"]
    live = np.repeat(d["ctx"] >= 0, d["lens"])
    for h in heads:
        of = slice(h * per, (h + 1) * per)
        ref = attn.decode(d["qw"][:, of], d["cu"], d["ctx"], d["kw"][:, h:h + 1], d["vw"][:, h:h + 1], d["table"], 1 / np.sqrt(d["D"]))
        check_attention(o[:, of], lse[:, of], ref, d["io"], np.nonzero(live)[0], f"{what} key head {h}")
    assert (o[~live] == 7.0).all() and (lse[~live] == 7.0).all()


# ---------------------------------------------------------------------------
# A workgroup finds 64 sequences, or row blocks, of its stretch at a time.
@pytest.mark.parametrize("io,D,per,q_len", [("bf16", 64, 1, 1), ("bf16", 128, 1, 3), ("f32", 64, 2, 2), ("f32", 128, 1, 1), ("bf16", 64, 5, 12),
                                            ("f32", 128, 4, 12), ("bf16", 128, 12, 12)])
@pytest.mark.parametrize("shared", [False, True])
def test_stretches_of_many_sequences(shared, io, D, per, q_len):
    """A workgroup per key head, each with the whole line of 200 sequences: some padded, some without tokens, one of several
    tiles; with groups, 90 prefixes on a line of their own."""
    HK, n = 520, 200
    r = np.random.default_rng(per + D)
    lens = r.integers(0 if q_len > 1 else 1, q_len + 1, n)
    ctx = np.where(r.random(n) < 0.2, -1, r.integers(16, 60, n))
    ctx[37], lens[37] = 700, q_len
    d = _repeated([per, D], io, D, per * HK, HK, lens.tolist(), ctx, groups=[(2, i % 2) for i in range(90)] if shared else None)
    _check_key_heads(d, [0, 7, HK - 1])


@pytest.mark.parametrize("io,D", [("bf16", 64), ("f32", 128)])
@pytest.mark.parametrize("at", [0, 60, 149])
def test_one_long_context_beside_many_short_ones(at, io, D):
    """Eight workgroups per key head: the long sequence's tiles make stretches that hold all of the short ones, before it
    and behind it."""
    HK, n = 64, 150
    r = np.random.default_rng(at)
    ctx = np.where(r.random(n) < 0.3, -1, r.integers(0, 50, n))
    ctx[at] = 64 * 80 * 8
    d = _repeated([at, D], io, D, HK, HK, [1] * n, ctx)
    _check_key_heads(d, [0, 31, HK - 1])


# ---------------------------------------------------------------------------
# A row that sees nothing has o = 0 and lse = -inf; one that sees scores of -inf only has neither.  Every query's channel 2
# is -1 here, so that a key with an infinity there scores -inf.
def _finite_sizes(ref, clean):
    """the tolerance's sums come from the keys that are finite"""
    return {**ref, "size": clean["size"]}


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("HQ,HK,lens,heads", [(4, 2, [5, 70, 1, 300], 0), (1, 1, [700], 0), (32, 8, [40] * 70 + [300], 3)])
def test_prompts_with_scores_of_minus_infinity(HQ, HK, lens, heads, D, io):
    """The first keys of each sequence, one to 200 of them, in one key head."""
    r = np.random.default_rng(D + len(lens))
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    (q, qw), (k, kw), (v, vw) = (normal(r, (int(cu[-1]), h, D), io) for h in (HQ, HK, HK))
    q[:, :, 2], qw[:, :, 2] = -1.0, -1.0
    k[:, heads, 2], kw[:, heads, 2] = 0.0, 0.0
    per = HQ // HK
    some = slice(heads * per, (heads + 1) * per) if len(lens) > 60 else slice(0, HQ)    # of many sequences: the head itself
    of = lambda x, y, z: (x[:, some], y[:, some.start // per: some.stop // per], z[:, some.start // per: some.stop // per])  # noqa: E731
    clean = attn.prefill(*of(qw, kw, vw), cu, 1 / np.sqrt(D))
    for n, L in enumerate(lens):
        bad = slice(int(cu[n]), int(cu[n]) + min(L, (1, 3, 70, 200)[n % 4]))
        k[bad, heads, 2], kw[bad, heads, 2] = float("inf"), np.inf
    o, lse = gdr.gdr_attn_prefill_fwd(q, k, v, cu_seqlens=to_dev(cu), output_lse=True)
    with np.errstate(invalid="ignore"):
        ref = attn.prefill(*of(qw, kw, vw), cu, 1 / np.sqrt(D))
    assert np.isnan(ref["o"]).any() and np.isnan(ref["lse"]).any() and not np.isnan(ref["o"]).all()
    check_attention(f64(o)[:, some], f64(lse)[:, some], _finite_sizes(ref, clean), io, np.arange(int(cu[-1])))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("HQ", [2, 8, 24])
@pytest.mark.parametrize("shared", [False, True])
def test_steps_with_scores_of_minus_infinity(shared, HQ, D, io):
    lens = [1, 1, 2, 12, 12, 1, 3, 1, 2, 1, 3]
    ctx = [210, 699, 699, 210, 200, 300, 0, 0, 80, -1, 30]
    #      the prefix of two groups is all such keys, the prefix of a third is none
    groups = [(3, 210), (2, 200), (1, 300), (0, 0)] if shared else None
    d = _decode_inputs([HQ, D], io, D, HQ, 2, lens, ctx, 16, groups=groups)
    d["q"][:, :, 2], d["qw"][:, :, 2] = -1.0, -1.0
    d["k"][:, 0, :, 2], d["kw"][:, 0, :, 2] = 0.0, 0.0
    table, num = d["table"], d["kw"].shape[0]
    if not shared:
        table[8, :] = -1            # sees nothing
        table[2, 5] = table[7, 0] = -1
        table[10, 0] = num          # its first page is none, the others' keys are all such
    clean = attn.decode(d["qw"], d["cu"], d["ctx"], d["kw"], d["vw"], table, 1 / np.sqrt(D))
    #        whole contexts, all but the last keys, the first ones, the last ones
    spans = {0: (0, 211), 1: (0, 700), 2: (0, 400), 3: (0, 222), 4: (0, 200), 5: (288, 301), 6: (0, 2), 10: (16, 33)}
    for n, (a, b) in spans.items():
        for j in range(a, b):
            p = attn.place(table, num, 16, n, j)
            if p is not None:
                d["k"][p[0], 0, p[1], 2], d["kw"][p[0], 0, p[1], 2] = float("inf"), np.inf
    o, lse = _decode_call(d, output_lse=True)
    with np.errstate(invalid="ignore"):
        ref = attn.decode(d["qw"], d["cu"], d["ctx"], d["kw"], d["vw"], table, 1 / np.sqrt(D))
    live = np.nonzero(np.repeat(np.asarray(ctx) >= 0, lens))[0]
    assert np.isnan(ref["o"][live, 0, 0]).sum() > 10 and not np.isnan(ref["o"][live, HQ - 1]).any()
    if not shared:
        assert (ref["o"][d["cu"][8]: d["cu"][9]] == 0).all()
    check_attention(f64(o), f64(lse), _finite_sizes(ref, clean), io, live)


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("shared", [False, True])
def test_the_longest_table_row(shared):
    """2^31 - 128 keys, of which the table names the same few pages over and over; with a prefix, own tiles that begin in the
    middle of 64 keys.  Equal scores and values: o is the value, lse the logarithm of the keys.  A lane adds up 2^20 weights of
    1 and a workgroup 2^22, exactly; the join adds up at most 514 such sums, each time off by 2^-24 of the total at most.
    Weights times values have eight more bits: an accumulator takes 2^21 keys, and the i-th addition rounds a sum that is i
    2^-21 of the last one by 2^-24, together 2^20 2^-24; then the join, the division and the output's rounding."""
    D, page, most = 64, 16, (1 << 27) - 8
    k = torch.randn(4, 1, page, D, device="cuda").bfloat16()
    value = torch.randn(D, device="cuda").bfloat16()
    v = value.expand(4, 1, page, D).contiguous()
    table = torch.randint(0, 4, (1, most), dtype=torch.int32, device="cuda")
    ctx = torch.tensor([most * page - 1], dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 2, D, dtype=torch.bfloat16, device="cuda")
    args = dict(group_offsets=to_dev(np.array([0, 1], np.int32)), prefix_lens=to_dev(np.array([48], np.int32))) if shared else {}
    o, lse = gdr.gdr_attn_decode_paged(q, k, v, table, ctx, output_lse=True, **args)
    assert (np.abs(f64(o) - f64(value)) <= np.abs(f64(value)) * (2.0 ** -4 + 520 * 2.0 ** -24 + 2.0 ** -8)).all()
    assert np.abs(f64(lse) - np.log(2.0 ** 31 - 128)).max() < 514 * 2.0 ** -24 + 100 * 2.0 ** -24
    with pytest.raises(gdr.GdrError):      # one page more
        gdr.gdr_attn_decode_paged(q, k, v, torch.zeros(1, most + 1, dtype=torch.int32, device="cuda"), ctx)


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.0, 1e-39, -3e-39, 2e-42, 3e-45])
def test_scales_near_zero_of_large_scores(scale, io):
    """q . k of 10^37: no scale below the smallest normal number may be taken for a larger one.  (A scale's conversion to base
    2 is off by half of 2^-149: times scores below 2^127 that is 2^-23, of the 64 u for such things.)"""
    r = np.random.default_rng(91)
    HQ, HK, D, lens = 4, 2, 64, [150, 3, 70]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    (q, qw), (k, kw), (v, vw) = (normal(r, (int(cu[-1]), h, D), io, x) for h, x in ((HQ, 1e18), (HK, 1e18), (HK, 1.0)))
    assert np.abs(np.einsum("thd,thd->th", qw[:, ::2], kw)).max() > 5e36
    scale = np.float32(scale).item()
    o, lse = gdr.gdr_attn_prefill_fwd(q, k, v, cu_seqlens=to_dev(cu), scale=scale, output_lse=True)
    check_attention(f64(o), f64(lse), attn.prefill(qw, kw, vw, cu, scale), io, np.arange(int(cu[-1])))
    d = _decode_inputs(92, io, D, HQ, HK, [2, 1, 3], [300, 30, 77], 16, sharp=1e18)
    d["k"].mul_(1e18)
    d["kw"] = f64(d["k"])
    o, lse = _decode_call(d, scale=scale, output_lse=True)
    ref = attn.decode(d["qw"], d["cu"], d["ctx"], d["kw"], d["vw"], d["table"], scale)
    check_attention(f64(o), f64(lse), ref, io, np.arange(6))


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_the_largest_scale(sign, D, io):
    """Scores are a key's first channel times +-2^127: the largest has a weight of 1 and the others none, also where they are
    past fp32 (3 and -3) and lse is infinite."""
    r = np.random.default_rng(101)
    scale, HQ, HK = sign * 2.0 ** 127, 4, 2
    lens = [330, 40, 700]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    x = np.full(T, -3.0)
    for n, a in enumerate((150, 0, 400)):                  # from there on growing; one of 3 at the very end
        x[cu[n] + a:cu[n + 1]] = np.array([-0.5, -0.25, 0.0, 0.25, 0.5, 0.625, 0.75, 1.0])[np.arange(lens[n] - a) * 8 // (lens[n] - a)]
    first = np.array([np.argmax(x[cu[n]:cu[n] + i + 1]) + cu[n] for n in range(3) for i in range(lens[n])])
    ties = np.array([int((x[cu[n]:cu[n] + i + 1] == x[f]).sum()) for (n, i), f in zip([(n, i) for n in range(3) for i in range(lens[n])], first)])
    q, k = np.zeros((T, HQ, D)), np.zeros((T, HK, D))
    q[:, :, 0], k[:, :, 0] = 1.0, sign * x[:, None]
    k[T - 1, :, 0] = sign * 3.0
    q, k = to_dev(q.astype(np.float32)).to(TORCH[io]), to_dev(k.astype(np.float32)).to(TORCH[io])
    v, vw = normal(r, (T, HK, D), io)
    top = x[first]
    want = np.stack([vw[f:f + c].mean(0) for f, c in zip(first, ties)])[:, np.arange(HQ) // (HQ // HK)]
    lse_want = np.where(top == -3.0, -np.inf, top * 2.0 ** 127)
    want[T - 1], lse_want[T - 1] = vw[T - 1][np.arange(HQ) // (HQ // HK)], np.inf
    most = np.abs(vw).max()

    def check(o, lse, rows, what):
        # c values and the division: (c + 2) u of the largest; lse: the two constants, three products and the sum, 6 u, and the
        # logarithm of up to 100 keys
        past = np.isinf(lse_want[rows])
        assert (lse[past] == lse_want[rows][past][:, None]).all() and past.any() and not past.all(), what
        allowed = (ties[rows][:, None, None] + 2) * 2.0 ** -24 * most + HALF[io] * np.abs(want[rows])
        assert (np.abs(o - want[rows]) <= allowed).all(), what
        lse, fine = lse[~past], lse_want[rows][~past][:, None]
        assert (np.abs(lse - fine) <= 6 * 2.0 ** -24 * np.abs(fine) + 5).all(), what

    o, lse = gdr.gdr_attn_prefill_fwd(q, k, v, cu_seqlens=to_dev(cu), scale=scale, output_lse=True)
    check(f64(o), f64(lse), np.arange(T), "prompts")
    # the same from a cache: four tokens of each of several lengths
    page = 16
    table = np.zeros((8, 48), np.int32)
    ends = [(0, 100), (0, 152), (0, 330), (1, 4), (1, 40), (2, 390), (2, 405), (2, 700)]
    pages = []
    for s, (n, e) in enumerate(ends):
        for i in range(-(-e // page)):
            table[s, i] = len(pages)
            pages.append((cu[n] + i * page + np.arange(page)).clip(0, T - 1))
    at = to_dev(np.stack(pages)).long()
    kp, vp = k[at].transpose(1, 2).contiguous(), v[at].transpose(1, 2).contiguous()
    rows = np.concatenate([cu[n] + np.arange(e - 4, e) for n, e in ends])
    ctx = np.array([e - 4 for _, e in ends], np.int32)
    for groups in (None, ([0, 1, 2, 3], [96, 144, 160]), ([0, 6, 7, 8], [0, 400, 688])):
        args = {} if groups is None else dict(zip(("group_offsets", "prefix_lens"), (to_dev(np.array(x, np.int32)) for x in groups)))
        o, lse = gdr.gdr_attn_decode_paged(q[to_dev(rows).long()].contiguous(), kp, vp, to_dev(table), to_dev(ctx),
                                           cu_seqlens=to_dev(np.arange(0, 33, 4, dtype=np.int32)), max_q_len=4, scale=scale, output_lse=True, **args)
        check(f64(o), f64(lse), rows, f"steps {groups}")


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,mean,HQ,HK", [(70, 300, 1, 1), (65, 205, 2, 1), (65, 205, 1, 1), (100, 30, 16, 4), (90, 30, 24, 8), (70, 45, 32, 8), (100, 40, 64, 8), (80, 20, 80, 10),
                                          (65, 200, 40, 5)])
def test_many_ragged_prompts(n, mean, HQ, HK, D, io):
    """More sequences than are cut at their own borders: workgroups of 32, 64 and 128 rows (one or two heads of long prompts, few
    heads, many heads) that hold several sequences, some without tokens; the first, an inner and the last head."""
    r = np.random.default_rng([n, HQ])
    lens = np.where(r.random(n) < 0.1, 0, r.integers(1, 2 * mean, n))
    lens[n // 2] = 5 * mean
    lens[-1] = 3
    if HQ < 3:                                             # long ones for all
        lens = np.maximum(lens, 200) if mean > 205 else r.integers(195, 216, n)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    end, T = int(cu[-1]), int(cu[-1]) + 5
    (q, qw), (k, kw), (v, vw) = (normal(r, (T, h, D), io, x) for h, x in ((HQ, 2.0), (HK, 1.0), (HK, 1.0)))
    o = torch.full((T, HQ, D), 7.0, dtype=TORCH[io], device="cuda")
    lse = torch.full((T, HQ), 7.0, device="cuda")
    gdr.gdr_attn_prefill_fwd(q, k, v, cu_seqlens=to_dev(cu), o=o, lse=lse)
    assert bool((o[end:] == 7.0).all()) and bool((lse[end:] == 7.0).all())
    o, lse = f64(o), f64(lse)
    for h in sorted({0, HQ // 2 - HQ // 7, HQ - 1}):
        ref = attn.prefill(qw[:end, h:h + 1], kw[:end, h * HK // HQ][:, None], vw[:end, h * HK // HQ][:, None], cu, 1 / np.sqrt(D))
        check_attention(o[:end, h:h + 1], lse[:end, h:h + 1], ref, io, np.arange(end), f"head {h}")


# ---------------------------------------------------------------------------
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("shared", [False, True])
def test_a_prompt_in_pieces(shared, io):
    """Tokens of a prompt behind others of it that are in the cache: stored first, then attended to as sequences of up to 12
    tokens with the same table row, whose common tokens are a prefix.  The last piece's rows are those of the whole prompt."""
    r = np.random.default_rng(111)
    HQ, HK, D, page, lens = 8, 2, 64, 16, [150, 40, 230]
    cut = [70, 33, 128]                                    # tokens of the first piece
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    (q, qw), (k, kw), (v, vw) = (normal(r, (int(cu[-1]), h, D), io) for h in (HQ, HK, HK))
    table = r.permutation(45).reshape(3, 15).astype(np.int32)
    kp = torch.full((45, HK, page, D), float("nan"), dtype=TORCH[io], device="cuda")
    vp = kp.clone()
    for part in (0, 1):
        rows = np.concatenate([cu[n] + (np.arange(cut[n]) if part == 0 else np.arange(cut[n], lens[n])) for n in range(3)])
        at, have = to_dev(rows).long(), [0, 0, 0] if part == 0 else cut
        many = np.concatenate([[0], np.cumsum([cut[n] if part == 0 else lens[n] - cut[n] for n in range(3)])]).astype(np.int32)
        gdr.gdr_rope_append_paged(q[at], k[at], v[at], k_pages=kp, v_pages=vp, page_table=to_dev(table), cu_seqlens=to_dev(many),
                                  context_lens=to_dev(np.array(have, np.int32)))
    ctx = [c for n in range(3) for c in range(cut[n], lens[n], 12)]
    of = [n for n in range(3) for _ in range(cut[n], lens[n], 12)]
    steps = np.concatenate([[0], np.cumsum([min(12, lens[n] - c) for c, n in zip(ctx, of)])]).astype(np.int32)
    offsets = np.searchsorted(of, np.arange(4)).astype(np.int32)
    args = dict(group_offsets=to_dev(offsets), prefix_lens=to_dev(np.array(cut, np.int32))) if shared else {}
    o, lse = gdr.gdr_attn_decode_paged(q[at], kp, vp, to_dev(table[of]), to_dev(np.array(ctx, np.int32)), cu_seqlens=to_dev(steps),
                                       max_q_len=12, output_lse=True, **args)
    ref = attn.prefill(qw, kw, vw, cu, 1 / np.sqrt(D))
    check_attention(f64(o), f64(lse), {x: ref[x][rows] for x in ref}, io, np.arange(len(rows)))
