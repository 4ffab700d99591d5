"""Full attention of serving on the GPU (rotary append, prefill, paged decode) against the fp64 oracle.  Tolerances
of the attention: _attn.py.  Rotation: a cosine and a sine rounded to fp32, two products and a sum, 4 u (|x| + |y|),
the angle's 64-bit error below them, and the output's half step."""
import numpy as np
import pytest
import torch

from _attn import HALF, TORCH, U, check, check_attention, normal, pages_for, wide
from _dev import f64, to_dev, to_host
from gated_delta_rule_63_amd import gdr
from oracle import attn

pytestmark = pytest.mark.gpu


def _freq(axes, half, base=10000.0):
    f = np.zeros((axes, half), np.float32)
    for i in range(half):
        f[i % axes, i] = base ** (-i / max(1, half))
    return f


def _rotated_close(got, x, theta, interleaved, io, what):
    want = attn.rotate(x, theta, interleaved)
    size = np.abs(x)
    half = theta.shape[1]
    if half:
        a, b = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
        size = size.copy()
        size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    allowed = 4 * U * size + HALF[io] * np.abs(want)
    allowed[..., 2 * half:] = 0.0     # channels that do not turn are copied
    check(got, want, allowed, what)


def _append_case(seed, io, D, HQ, HK, lens, ctx, rotary, interleaved, axes, page, tail=0, fused=True, positions=None,
                 table=None, num_pages=None, one_token=False):
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T, end = int(cu[-1]) + tail, int(cu[-1])
    if fused:
        t, w = normal(r, (T, HQ + 2 * HK + 1, D), io)
        parts = [(0, HQ), (HQ, HQ + HK), (HQ + HK, HQ + 2 * HK)]
        (q, k, v), (qw, kw, vw) = [t[:, a:b] for a, b in parts], [w[:, a:b] for a, b in parts]
    else:
        (q, qw), (k, kw), (v, vw) = normal(r, (T, HQ, D), io), normal(r, (T, HK, D), io), normal(r, (T, HK, D), io)
    ctx = np.asarray(ctx, np.int32)
    if table is None:
        table, num_pages = pages_for(r, np.maximum(ctx, 0) + np.asarray(lens), page)
    freq = _freq(axes, rotary // 2)
    if positions is None and axes > 1:
        positions = r.integers(0, 1 << 20, (axes, T)).astype(np.int32)
    sent = lambda *s: torch.full(s, 7.0, dtype=TORCH[io], device="cuda")  # noqa: E731
    kp, vp = sent(num_pages, HK, page, D), sent(num_pages, HK, page, D)
    qo, ko = sent(T, HQ, D), sent(T, HK, D)
    got = gdr.gdr_rope_append_paged(q, k, v, to_dev(freq), k_pages=kp, v_pages=vp, page_table=to_dev(table),
                                    context_lens=to_dev(ctx), cu_seqlens=None if one_token else to_dev(cu),
                                    positions=None if positions is None else to_dev(positions), interleaved=interleaved,
                                    q_out=qo, k_out=ko)
    assert got[0] is qo and got[1] is ko
    torch.cuda.synchronize()
    place = np.concatenate([int(c) + np.arange(n) for c, n in zip(ctx, lens)] + [np.zeros(tail)])
    theta = attn.angles(place[None] if positions is None else positions, freq)
    live = np.zeros(T, bool)
    for n in range(len(lens)):
        live[cu[n]:cu[n + 1]] = ctx[n] >= 0
    qo, ko = f64(qo), f64(ko)
    _rotated_close(qo[live], qw[live], theta[live], interleaved, io, "q")
    _rotated_close(ko[live], kw[live], theta[live], interleaved, io, "k")
    assert (qo[~live] == 7.0).all() and (ko[~live] == 7.0).all()
    want_k, want_v = np.full(kp.shape, 7.0), np.full(vp.shape, 7.0)
    for n in range(len(lens)):
        for i in range(int(lens[n]) if ctx[n] >= 0 else 0):
            w = attn.place(table, num_pages, page, n, int(ctx[n]) + i)
            if w is not None:
                want_k[w[0], :, w[1]], want_v[w[0], :, w[1]] = ko[cu[n] + i], vw[cu[n] + i]
    assert np.array_equal(f64(kp), want_k) and np.array_equal(f64(vp), want_v)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", ["all", "half", 34, 2, 0])
def test_append(rotary, interleaved, D, io):
    R = {"all": D, "half": D // 2}.get(rotary, rotary)
    _append_case(R + D, io, D, 6, 2, [5, 1, 0, 40, 17, 3], [0, 31, 5, 16, -1, 100], R, interleaved, 1, 16, tail=4)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("axes", [2, 3, 8])
def test_append_several_axes(axes, io):
    _append_case(axes, io, 64, 4, 4, [33, 20], [0, 7], 48, axes == 3, axes, 32)


@pytest.mark.parametrize("page", [16, 64, 1024])
def test_append_one_token_each_and_page_sizes(page):
    r = np.random.default_rng(page)
    ctx = r.integers(-1, 3 * page, 37)
    _append_case(page, "bf16", 128, 8, 1, [1] * 37, ctx, 128, False, 1, page, one_token=True)


def test_append_a_long_batch():
    """Enough tokens for several per workgroup, sequence borders inside them."""
    _append_case(3, "bf16", 64, 2, 1, [1, 2, 3, 5000, 7, 0, 0, 1100, 1], [0, 5, 0, 3, -3, 0, 9, 64, 2], 64, False, 1, 64, tail=11)


def test_append_far_positions():
    pos = np.array([[0, 1, 65535, 10 ** 6, 2 ** 31 - 1, 12345678, -1, -(10 ** 6)]], np.int32)
    _append_case(4, "f32", 128, 2, 1, [8], [0], 128, False, 1, 16, positions=pos)


def test_append_outside_the_table():
    """Pages out of range and tokens behind the table's last page are not stored."""
    table = np.array([[3, -1, 1], [0, 9, 2], [-7, 4, 1 << 30]], np.int32)
    _append_case(5, "f32", 64, 2, 2, [70, 10, 30], [0, 14, 20], 64, False, 1, 16, table=table, num_pages=6)
    _append_case(6, "bf16", 64, 2, 2, [1, 1], [2 ** 31 - 1, 40], 64, False, 1, 16, table=table[:2], num_pages=6, one_token=True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("rotary,interleaved", [(64, False), (64, True), (18, False)])
def test_rotation_in_place_without_a_cache(rotary, interleaved, io):
    r = np.random.default_rng(7)
    (q, qw), (k, kw) = normal(r, (50, 3, 64), io), normal(r, (50, 1, 64), io)
    freq = to_dev(_freq(1, rotary // 2))
    want = gdr.gdr_rope_append_paged(q, k, inv_freq=freq, interleaved=interleaved)
    got = gdr.gdr_rope_append_paged(q, k, inv_freq=freq, interleaved=interleaved, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    theta = attn.angles(np.arange(50)[None], _freq(1, rotary // 2))
    _rotated_close(f64(q), qw, theta, interleaved, io, "q")
    _rotated_close(f64(k), kw, theta, interleaved, io, "k")


# ---------------------------------------------------------------------------
def _prefill_case(seed, io, D, HQ, HK, lens, tail=0, scale=None, fused=False, sharp=2.0):
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T, end = int(cu[-1]) + tail, int(cu[-1])
    if fused:
        t, w = normal(r, (T, HQ + 2 * HK, D), io)
        parts = [(0, HQ), (HQ, HQ + HK), (HQ + HK, HQ + 2 * HK)]
        (q, k, v), (qw, kw, vw) = [t[:, a:b] for a, b in parts], [w[:, a:b] for a, b in parts]
    else:
        (q, qw), (k, kw), (v, vw) = normal(r, (T, HQ, D), io, sharp), normal(r, (T, HK, D), io), normal(r, (T, HK, D), io)
    o = torch.full((T, HQ, D), 7.0, dtype=TORCH[io], device="cuda")
    lse = torch.full((T, HQ), 7.0, device="cuda")
    gdr.gdr_attn_prefill_fwd(q, k, v, cu_seqlens=to_dev(cu), scale=scale, o=o, lse=lse)
    torch.cuda.synchronize()
    ref = attn.prefill(qw, kw, vw, cu, 1 / np.sqrt(D) if scale is None else scale)
    o, lse = f64(o), f64(lse)
    check_attention(o, lse, ref, io, np.arange(end))
    assert (o[end:] == 7.0).all() and (lse[end:] == 7.0).all()


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[1], [2, 1], [33], [64, 65], [127, 1, 0, 3], [128, 129], [0, 0, 300, 0, 31, 32]])
def test_prefill(lens, D, io):
    _prefill_case(sum(lens) + D, io, D, 4, 2, lens, tail=sum(lens) % 3)


@pytest.mark.parametrize("HQ,HK", [(1, 1), (3, 1), (5, 5), (8, 1), (8, 8), (16, 2), (24, 8)])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prefill_heads(HQ, HK, io):
    _prefill_case(HQ, io, 64, HQ, HK, [70, 150], fused=HQ % 2 == 0)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prefill_many_short_sequences(io):
    r = np.random.default_rng(11)
    _prefill_case(11, io, 64, 2, 1, r.integers(0, 5, 300).tolist())
    _prefill_case(12, io, 128, 2, 2, [1] * 130 + [200] + [1] * 60, tail=100)


@pytest.mark.parametrize("scale", [1.0, -0.125, 0.0, 30.0, 1e-30])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prefill_scales(scale, io):
    _prefill_case(13, io, 64, 2, 1, [100, 7], scale=scale)


def test_prefill_a_longer_prompt():
    _prefill_case(14, "bf16", 128, 2, 1, [1500, 700])
    _prefill_case(15, "f32", 128, 1, 1, [1100])


# ---------------------------------------------------------------------------
def _decode_inputs(seed, io, D, HQ, HK, lens, ctx, page, spare=3, sharp=2.0, groups=None, width=None):
    """groups: [(sequences, prefix)] - members' first ``prefix`` tokens are the same, whole pages of them shared"""
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    ctx = np.asarray(ctx, np.int32)
    table, pages = pages_for(r, np.maximum(ctx, 0) + np.asarray(lens), page, spare, width)
    (q, qw), (k, kw), (v, vw) = normal(r, (int(cu[-1]), HQ, D), io, sharp), normal(r, (pages, HK, page, D), io), normal(r, (pages, HK, page, D), io)
    d = dict(q=q, k=k, v=v, qw=qw, kw=kw, vw=vw, cu=cu, ctx=ctx, table=table, io=io, D=D, page=page, lens=list(lens))
    if groups is not None:
        at, offsets = 0, [0]
        for count, prefix in groups:
            rows = [n for n in range(at, at + count) if ctx[n] >= 0]
            whole = prefix // page
            for n in rows[1:]:
                table[n, :whole] = table[rows[0], :whole]
                if prefix % page:
                    a, b = int(table[rows[0], whole]), int(table[n, whole])
                    for w, t in ((kw, k), (vw, v)):
                        w[b, :, : prefix % page] = w[a, :, : prefix % page]
                        t[b, :, : prefix % page] = t[a, :, : prefix % page]
            at += count
            offsets.append(at)
        d["offsets"], d["prefix"] = np.array(offsets, np.int32), np.array([p for _, p in groups], np.int32)
    return d


def _decode_call(d, **kw):
    args = dict(cu_seqlens=to_dev(d["cu"]), max_q_len=max([1] + d["lens"]))
    if "offsets" in d:
        args.update(group_offsets=to_dev(d["offsets"]), prefix_lens=to_dev(d["prefix"]))
    args.update(kw)
    return gdr.gdr_attn_decode_paged(d["q"], d["k"], d["v"], to_dev(d["table"]), to_dev(d["ctx"]), **args)


def _decode_check(d, scale=None, **kw):
    T, HQ, D = d["q"].shape
    o = torch.full((T, HQ, D), 7.0, dtype=TORCH[d["io"]], device="cuda")
    lse = torch.full((T, HQ), 7.0, device="cuda")
    _decode_call(d, scale=scale, o=o, lse=lse, **kw)
    torch.cuda.synchronize()
    ref = attn.decode(d["qw"], d["cu"], d["ctx"], d["kw"], d["vw"], d["table"], 1 / np.sqrt(D) if scale is None else scale)
    o, lse = f64(o), f64(lse)
    live = np.concatenate([np.full(n, c >= 0) for n, c in zip(d["lens"], d["ctx"])] + [np.zeros(0, bool)])
    check_attention(o, lse, ref, d["io"], np.nonzero(live)[0])
    assert (o[~live] == 7.0).all() and (lse[~live] == 7.0).all()
    return o


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("HQ,HK", [(1, 1), (8, 2), (5, 1), (16, 4)])
def test_decode_one_token(HQ, HK, D, io):
    _decode_check(_decode_inputs(HQ + D, io, D, HQ, HK, [1] * 9, [0, 1, 62, 63, 64, 200, -1, 700, 15], 16), cu_seqlens=None)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 32, 128, 4096])
@pytest.mark.parametrize("HQ,HK", [(4, 4), (8, 1), (16, 1)])
def test_decode_several_tokens(HQ, HK, page, io):
    """Rows of a block from 12 to 192."""
    _decode_check(_decode_inputs(HQ + page, io, 64, HQ, HK, [12, 1, 0, 5, 12, 7], [0, 0, 40, 100, 500, -1], page))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_decode_long_context(io):
    _decode_check(_decode_inputs(21, io, 128, 2, 1, [1], [5000], 64))
    _decode_check(_decode_inputs(22, io, 128, 2, 2, [3, 2], [3000, 1], 64))


def test_decode_more_sequences_than_workgroups():
    r = np.random.default_rng(23)
    _decode_check(_decode_inputs(23, "bf16", 64, 2, 2, r.integers(0, 3, 1500).tolist(), r.integers(-1, 90, 1500), 16))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 20.0])
def test_decode_scales(scale, io):
    _decode_check(_decode_inputs(24, io, 64, 4, 2, [2, 1], [90, 300], 16), scale=scale)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len", [1, 4])
def test_decode_shared_prefix(q_len, D, io):
    lens = [1 + i % q_len for i in range(11)]
    #      one group whose first sequence is padded, one alone, one without a prefix, two outside
    groups = [(4, 200), (1, 64), (3, 0), (1, 15)]
    ctx = [-1, 200, 333, 205, 70, 10, -1, 90, 31, 44, 0]
    _decode_check(_decode_inputs(q_len + D, io, D, 8, 2, lens, ctx, 16, groups=groups))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_decode_shared_prefix_of_many_rows(io):
    """Several row blocks over a prefix that is cut into parts; contexts that end with it."""
    _decode_check(_decode_inputs(31, io, 64, 16, 2, [1] * 40, [1024 + (i % 3) * 5 for i in range(40)], 64, groups=[(40, 1024)]))


def test_decode_result_with_and_without_sharing():
    d = _decode_inputs(32, "f32", 64, 4, 2, [2] * 6, [300 + i for i in range(6)], 32, groups=[(6, 290)])
    a = _decode_check(d)
    b = _decode_check({k: v for k, v in d.items() if k != "offsets"})
    assert np.abs(a - b).max() < 1e-5


def test_decode_pages_outside_the_cache():
    """What such a page would hold is not seen; a sequence without any page gives zeros and -inf."""
    d = _decode_inputs(33, "f32", 64, 4, 2, [1, 3, 2, 1], [100, 50, 20, 500], 16, width=8)
    d["table"][0, 2], d["table"][1, 0], d["table"][2, :] = -1, 1 << 30, -5
    o = _decode_check(d)
    assert (o[4:6] == 0).all()


def test_decode_views_of_wider_rows():
    d = _decode_inputs(34, "bf16", 128, 4, 1, [2, 3], [40, 90], 16)
    t = torch.randn(5, 9, 128, device="cuda").to(torch.bfloat16)
    t[:, 3:7] = d["q"]
    d["q"] = t[:, 3:7]
    _decode_check(d)


# ---------------------------------------------------------------------------
# values that are not finite reach the rows that see them, and no others
def _put(t, w, index, value):
    t[index] = value
    w[index] = value


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
def test_prefill_special_values(D, io):
    """In a value: that channel of the rows that see it.  In a key or a query: NaN in those rows.  Other sequences,
    earlier tokens, other heads: as if it were not there."""
    r = np.random.default_rng(17 + D)
    lens, HQ, HK = [70, 90, 40, 130], 4, 2
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    (q, qw), (k, kw), (v, vw) = normal(r, (T, HQ, D), io), normal(r, (T, HK, D), io), normal(r, (T, HK, D), io)
    clean = attn.prefill(qw, kw, vw, cu, 1 / np.sqrt(D))
    spots = [(75, 0, 3, np.nan), (100, 1, D - 1, np.inf), (100, 0, 0, -np.inf), (159, 0, 7, np.nan), (160, 1, 9, np.inf),
             (170, 1, 9, -np.inf), (330 - 1, 1, 5, np.nan)]
    for j, h, c, x in spots:
        _put(v, vw, (j, h, c), x)
    o, lse = gdr.gdr_attn_prefill_fwd(q, k, v, cu_seqlens=to_dev(cu), output_lse=True)
    o, lse, want = f64(o), f64(lse), clean["o"].copy()
    end = np.repeat(cu[1:], lens)
    for j, h, c, x in spots:
        for hh in (2 * h, 2 * h + 1):
            with np.errstate(invalid="ignore"):
                want[j:end[j], hh, c] += x
    check_attention(o, lse, {**clean, "o": want}, io, np.arange(T))
    # a key and a query
    _put(k, kw, (80, 1, 2), np.nan)
    _put(q, qw, (20, 0, 0), np.nan)
    o, lse = (f64(x) for x in gdr.gdr_attn_prefill_fwd(q, k, v, cu_seqlens=to_dev(cu), output_lse=True))
    want[80:160, 2:], want[20, 0] = np.nan, np.nan
    ref = {**clean, "o": want, "lse": clean["lse"].copy()}
    ref["lse"][80:160, 2:], ref["lse"][20, 0] = np.nan, np.nan
    check_attention(o, lse, ref, io, np.arange(T))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("HQ", [2, 8, 16])
def test_decode_special_values(HQ, D, io):
    """The cache's unused rows and pages hold NaN; drafted tokens hold values that earlier ones must not feel."""
    d = _decode_inputs(41 + HQ + D, io, D, HQ, 2, [12, 5, 1, 12, 9], [60, 3, 100, 250, 500], 16)
    used = np.zeros(d["kw"].shape[0::2][:2], bool)
    for n, (c, m) in enumerate(zip(d["ctx"], d["lens"])):
        for j in range(int(c) + m):
            used[attn.place(d["table"], used.shape[0], 16, n, j)] = True
    for t, w in ((d["k"], d["kw"]), (d["v"], d["vw"])):
        t[to_dev(~used)[:, None, :, None].expand(t.shape)] = float("nan")
        w[np.broadcast_to(~used[:, None, :, None], w.shape)] = np.nan
    clean = attn.decode(d["qw"], d["cu"], d["ctx"], d["kw"], d["vw"], d["table"], 1 / np.sqrt(D))
    want, per = clean["o"].copy(), HQ // 2
    for n, j, h, c, x in [(0, 65, 0, 1, np.nan), (0, 70, 1, D - 1, np.inf), (3, 250, 1, 0, -np.inf), (3, 261, 0, 9, np.inf),
                          (4, 508, 1, 4, np.nan), (1, 7, 0, 2, np.inf), (4, 100, 1, 8, -np.inf)]:
        p, row = attn.place(d["table"], used.shape[0], 16, n, j)
        _put(d["v"], d["vw"], (p, h, row, c), x)
        for i in range(d["lens"][n]):
            if j <= d["ctx"][n] + i:
                with np.errstate(invalid="ignore"):
                    want[d["cu"][n] + i, h * per:(h + 1) * per, c] += x
    o, lse = _decode_call(d, output_lse=True)
    check_attention(f64(o), f64(lse), {**clean, "o": want}, io, np.arange(len(want)))
