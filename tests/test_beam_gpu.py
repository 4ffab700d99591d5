"""Beam search on the GPU: selection against the fp64 oracle (parents and tokens equal, scores to the
rounding of an fp32 value: the sums behind a score are good to 3e-6 absolutely, half the distance below
which the kernel forms them again in 64 bits), state reordering bit for bit, and both in a decode loop."""
import numpy as np
import pytest
import torch

from _dev import f64, to_dev, to_host
from gated_delta_rule_63_amd import gdr, inputs
from oracle import beam

pytestmark = pytest.mark.gpu


def _dev_logits(lg, io, pad):
    t = to_dev(lg.astype(np.float32))
    wide = torch.full(lg.shape[:2] + (lg.shape[2] + pad,), 50.0, device="cuda")
    wide[:, :, :lg.shape[2]] = t
    return wide.to(torch.bfloat16 if io == "bf16" else torch.float32)[:, :, :lg.shape[2]]


def _compare(lg, sc, K, io, pad=0, finished=None, eos=-1):
    d = _dev_logits(lg, io, pad)
    fin = None if finished is None else to_dev(finished.astype(np.uint8))
    s, p, t = gdr.gdr_beam_select(d, to_dev(sc), K, finished=fin, eos_token=eos)
    torch.cuda.synchronize()
    want = beam.select(f64(d), sc.astype(np.float64), K, finished, eos)
    assert np.array_equal(to_host(p), want[1]), "parents"
    assert np.array_equal(to_host(t), want[2]), "tokens"
    got = f64(s)
    assert np.array_equal(np.isneginf(got), np.isneginf(want[0]))
    fine = np.isfinite(want[0])
    assert np.all(np.abs(got - want[0])[fine] <= 3e-6 + 2.0 ** -24 * np.abs(want[0])[fine])


def _logits(seed, B, W, V, sd=2.5):
    return np.random.default_rng(seed).normal(size=(B, W, V)) * sd


def _scores(seed, B, W):
    return (-10 - np.cumsum(np.random.default_rng(seed).uniform(0, 1.5, (B, W)), 1)).astype(np.float32)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("B,W,V,K,pad", [(1, 1, 1, 1, 0), (1, 1, 64, 64, 0), (3, 4, 1000, 8, 0), (2, 5, 4097, 5, 3),
                                         (2, 32, 777, 64, 1), (1, 4, 32000, 8, 0), (2, 3, 50257, 6, 47),
                                         (1, 16, 20001, 1, 7), (1, 2, 262147, 17, 0), (2, 1, 70000, 64, 8)])
def test_sizes(B, W, V, K, pad, io):
    _compare(_logits(V, B, W, V), _scores(K, B, W), K, io, pad)


def test_largest_vocabulary_and_many_rows():
    _compare(_logits(1, 1, 1, 1 << 20), _scores(1, 1, 1), 64, "bf16")
    _compare(_logits(2, 150, 7, 600), _scores(2, 150, 7), 14, "f32")


@pytest.mark.parametrize("io,offset", [("bf16", 1), ("bf16", 3), ("f32", 1), ("f32", 2)])
def test_rows_that_begin_between_multiples_of_16_bytes(io, offset):
    lg, sc = _logits(30 + offset, 2, 3, 5003), _scores(31, 2, 3)
    lg[:, :, :9] += 8.0   # good candidates at both ends of the rows
    lg[:, :, -9:] += 8.0
    t = _dev_logits(lg, io, 0)
    flat = torch.empty(t.numel() + offset, dtype=t.dtype, device="cuda")
    view = flat[offset:].view(t.shape)
    view.copy_(t)
    want = beam.select(f64(t), sc.astype(np.float64), 20)
    s, p, tok = gdr.gdr_beam_select(view, to_dev(sc), 20)
    assert np.array_equal(to_host(p), want[1]) and np.array_equal(to_host(tok), want[2])


def test_most_lists():
    """32 beams over 2^20 tokens in fp32: the most parts that a merge sees.  Distinct random logits."""
    g = torch.Generator(device="cuda").manual_seed(3)
    lg = torch.randn(1, 32, 1 << 20, device="cuda", generator=g)
    sc = to_dev(_scores(32, 1, 32))
    s, p, t = gdr.gdr_beam_select(lg, sc, 64)
    x = lg[0].double()
    x = x - torch.logsumexp(x, 1, keepdim=True) + sc[0].double()[:, None]
    best, at = x.flatten().topk(64)
    assert bool((best[:-1] > best[1:]).all())
    assert torch.equal(p[0].long() * (1 << 20) + t[0].long(), at)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_ties_go_to_the_lower_index(io):
    for sd in (0.0, 0.25):  # all equal; a handful of distinct values
        lg = np.round(_logits(3, 2, 4, 9000, sd) * 4) / 4
        _compare(lg, np.zeros((2, 4), np.float32), 33, io)
        _compare(lg[:, :1], np.zeros((2, 1), np.float32), 64, io)
    # equal beams: the same logits and scores
    lg = np.repeat(_logits(4, 1, 1, 5000), 6, axis=1)
    _compare(lg, np.full((1, 6), -3.0, np.float32), 12, io)
    lg = np.zeros((1, 2, 3000))
    lg[..., ::2] = -0.0
    _compare(lg, np.zeros((1, 2), np.float32), 20, io)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_concentrated_logits(io):
    """Every large logit in few lanes' hands (neighbours, or a fixed distance apart), and sorted rows."""
    V = 40000
    for step in (1, 8, 256, 2048):
        lg = _logits(5, 1, 2, V, 0.5)
        at = (np.arange(300) * step) % V
        lg[:, :, np.unique(at)] += 10 + np.random.default_rng(6).normal(size=(1, 2, len(np.unique(at))))
        _compare(lg, _scores(7, 1, 2), 64, io)
    up = np.sort(_logits(8, 1, 2, V), axis=2)
    _compare(up, _scores(9, 1, 2), 50, io)
    _compare(up[:, :, ::-1].copy(), _scores(9, 1, 2), 50, io)


@pytest.mark.parametrize("fill", [-np.inf, np.nan, -3.3e38])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_masked_tokens(fill, io):
    r = np.random.default_rng(10)
    for kept in (0, 1, 3, 100):  # tokens that the mask leaves of each row
        lg = np.full((2, 3, 6001), fill)
        for b in range(2):
            for w in range(3):
                at = r.permutation(6001)[:kept]
                lg[b, w, at] = r.normal(size=kept) * 3
        if np.isfinite(fill):
            lg = lg.astype(np.float32).astype(np.float64)
        _compare(lg, _scores(11, 2, 3), 16, io)
    lg = _logits(12, 2, 3, 6001)
    lg[0, 1] = fill                       # one row with nothing left
    lg[1, :2] = fill
    _compare(lg, _scores(13, 2, 3), 20, io)


def test_rows_and_scores_without_candidates():
    lg = _logits(14, 3, 4, 900)
    sc = _scores(15, 3, 4)
    sc[0, 1:] = -np.inf                   # the first step of a search: one live beam
    sc[1] = [-np.inf, np.nan, np.inf, -np.inf]
    lg[2, 0, 5] = np.inf
    _compare(lg, sc, 30, "f32")
    _compare(lg, sc, 30, "bf16")
    _compare(lg[:, :, :3], sc, 3, "f32")


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_ended_beams(io):
    r = np.random.default_rng(16)
    lg, sc = _logits(17, 4, 5, 3000), _scores(18, 4, 5)
    fin = (r.uniform(size=(4, 5)) < 0.5).astype(np.uint8)
    fin[2], fin[3] = 1, 0
    sc[2, 1] = -np.inf
    for eos in (0, 2, 2999):
        _compare(lg, sc, 10, io, finished=fin, eos=eos)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("dead", [-1e9, -1e30, float(np.finfo(np.float32).min)])
@pytest.mark.parametrize("W,V,K", [(4, 32000, 8), (4, 32000, 16), (8, 131072, 16), (3, 131072, 64), (4, 700, 8)])
def test_beams_of_a_large_negative_score(W, V, K, dead, io):
    """A search's first step with finite scores for the beams that do not count yet: their logits round to the
    same 64-bit score, in more lists than results.  Then with fewer tokens left to the live beam than results."""
    lg = _logits(41 + K, 2, W, V)
    sc = np.full((2, W), dead, np.float32)
    sc[0, 0] = sc[1, W - 1] = 0.0
    _compare(lg, sc, K, io)
    lg[0, 0, 3:] = lg[1, W - 1, 3:] = -np.inf
    _compare(lg, sc, K, io)


@pytest.mark.parametrize("K", [8, 16, 64])
def test_logits_that_round_to_equal_scores(K):
    """Logits of 1e-17, and of 1e-17 beside one of 3: in a score of -10 they make no difference, their order does."""
    lg = _logits(45, 1, 4, 32000) * 1e-17
    _compare(lg, _scores(46, 1, 4), K, "f32")
    _compare(lg, np.full((1, 4), -5.0, np.float32), K, "f32")
    lg[0, :, 777] = 3.0
    _compare(lg, _scores(46, 1, 4), K, "f32")


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("W,V,K", [(4, 900, 8), (8, 32000, 16), (5, 4096, 5), (32, 600, 64), (8, 32000, 4), (2, 70000, 3)])
def test_ended_beams_of_equal_scores(W, V, K, io):
    """Some or all beams of a row have ended with one score or with scores a step apart, with as many lists as
    results, fewer and more: these scores are exact, and the live beams' candidates may lie as near to them."""
    B = 12
    lg, sc = _logits(48, B, W, V), _scores(49, B, W)
    fin = np.zeros((B, W), np.uint8)
    for b in range(B):
        some = np.random.default_rng(50 + b).permutation(W)[:W if b % 3 == 0 else max(2, W // 2)]
        fin[b, some] = 1
        sc[b, some] = sc[b, some[0]] + (0 if b % 2 else 1) * np.float32(1e-6) * np.arange(len(some), dtype=np.float32)
    x = lg[1].max(1) - np.log(np.exp(lg[1]).sum(1))
    live = np.flatnonzero(fin[1] == 0)
    if len(live):  # a live beam's best candidate beside the ended ones
        sc[1, live[0]] = np.float32(sc[1, fin[1] == 1][0] - x[live[0]])
    fin[2] = 1
    sc[2] = -3.0
    for eos in (0, V - 1):
        _compare(lg, sc, K, io, finished=fin, eos=eos)


def test_near_ties_between_beams_are_settled_in_64_bits():
    """Beams whose candidates differ by 1e-8 to 1e-6, below what 32-bit sums resolve."""
    r = np.random.default_rng(19)
    for trial in range(6):
        V = 5000 + trial
        base = r.normal(size=V) * 2
        lg = np.stack([r.permutation(base) for _ in range(6)])[None].astype(np.float32).astype(np.float64)
        # every row has the same sum; scores that differ by one fp32 step (5e-7 at 5) or not at all
        sc = np.full((1, 6), -5.0, np.float32)
        for w in range(1, 6):
            sc[0, w] = np.nextafter(sc[0, w - 1], np.float32(0)) if trial % 2 else sc[0, 0]
        lg[0, :, :] += (np.arange(6) * 1e-7)[:, None]
        lg = lg.astype(np.float32).astype(np.float64)
        d = _dev_logits(lg, "f32", 0)
        s, p, t = gdr.gdr_beam_select(d, to_dev(sc), 12)
        p, t = to_host(p)[0], to_host(t)[0]
        x = f64(d)[0]
        val = lambda w, v: sc[0, w].astype(np.float64) + (x[w, v] - (x[w].max() + np.log(np.exp(x[w] - x[w].max()).sum())))  # noqa: E731
        got = [val(w, v) for w, v in zip(p, t)]
        every = np.sort(np.concatenate([sc[0, w].astype(np.float64) + (x[w] - (x[w].max() + np.log(np.exp(x[w] - x[w].max()).sum()))) for w in range(6)]))[::-1]
        # in descending order and the best ones, to the rounding of 64-bit sums over V terms
        assert np.allclose(got, every[:12], rtol=0, atol=1e-12)


@pytest.mark.parametrize("K", [1, 2, 5])
def test_scores_that_round_to_coarse_steps(K):
    """Two beams with the same logits in another order and scores of -1e11, whose 64-bit steps are 2^-16.  The
    best candidates are equal and lie beside the middle between two steps: 32-bit sums that differ by 1e-8 put
    them on different ones."""
    B, V, step = 128, 3001, 2.0 ** -16
    lg, r = np.empty((B, 2, V)), np.random.default_rng(60)
    for b in range(B):
        x = (r.normal(size=V) * 2.5).astype(np.float32)
        x[0] = np.nextafter(x.max(), np.float32(100))
        tops = (x[:1].view(np.int32) + np.arange(4000, dtype=np.int32)).view(np.float32).astype(np.float64)
        rest = x[1:].astype(np.float64)
        at = (tops - (tops + np.log1p(np.exp(rest[None] - tops[:, None]).sum(1)))) / step
        off = np.abs(at - np.floor(at) - 0.5)
        x[0] = tops[np.where(off > 1e-6, off, 1.0).argmin()]  # 1e-6 steps are 1.5e-11: far more than 64-bit sums err
        lg[b] = x, r.permutation(x)
    _compare(lg, np.full((B, 2), -1e11, np.float32), K, "f32")


@pytest.mark.parametrize("V,K,equal", [(3001, 1, 2), (3001, 4, 6), (40000, 1, 2), (40000, 4, 9), (40000, 64, 300)])
def test_near_ties_behind_equal_candidates(V, K, equal):
    """The last result and those behind it are one beam's equal logits; another beam's best comes behind them
    all by the 32-bit sums, or before them, and is better by less than one fp32 step of its score."""
    B, r = 64, np.random.default_rng(23 + V + K)
    lg = (r.normal(size=(B, 2, V)) * 2).astype(np.float32).astype(np.float64)
    sc = np.full((B, 2), -0.5, np.float32)
    for b in range(B):
        lg[b, 0, r.choice(V, equal, replace=False)] = lg[b, 0].max()
        top = lg[b].max(1)
        lse = top + np.log(np.exp(lg[b] - top[:, None]).sum(1))
        first = float(sc[b, 0]) + (top[0] - lse[0])
        lg[b, 1] = np.minimum(lg[b, 1], top[1] - 1e-3 * (np.arange(V) != lg[b, 1].argmax()))
        lse1 = top[1] + np.log(np.exp(lg[b, 1].astype(np.float32).astype(np.float64) - top[1]).sum())
        s = np.float32(first - (top[1] - lse1))
        while float(s) + (top[1] - lse1) <= first:
            s = np.nextafter(s, np.float32(np.inf))
        sc[b, 1] = s
    want = beam.select(lg.astype(np.float32).astype(np.float64), sc.astype(np.float64), K)
    assert np.all(want[1][:, 0] == 1) and np.all(want[1][:, 1:] == 0)
    assert K == 1 or np.all(want[0][:, 0] - want[0][:, 1] > 1e-12)
    _compare(lg, sc, K, "f32")


def test_select_captured_and_on_another_stream():
    lg, sc = _logits(20, 3, 4, 20000), _scores(21, 3, 4)
    d, dsc = _dev_logits(lg, "bf16", 0), to_dev(sc)
    want = gdr.gdr_beam_select(d, dsc, 8)
    ws = torch.full((gdr.gdr_beam_workspace_size(d, 8),), 0x5A, dtype=torch.uint8, device="cuda")
    out = [torch.empty_like(t) for t in want]
    args = dict(out_scores=out[0], out_parents=out[1], out_tokens=out[2], workspace=ws)
    gdr.gdr_beam_select(d, dsc, 8, **args)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gdr.gdr_beam_select(d, dsc, 8, **args)
    for _ in range(3):
        for t in out:
            t.zero_()
        g.replay()
        gdr.gdr_beam_select(d, dsc, 8)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = gdr.gdr_beam_select(d, dsc, 8, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))


def test_select_offsets_past_32_bits():
    """Rows behind 2^31 logits: the last batch rows against the oracle."""
    B, W, V = 3300, 16, 41000
    lg = torch.randn(B, W, V, device="cuda", dtype=torch.bfloat16, generator=torch.Generator(device="cuda").manual_seed(2))
    sc = _scores(33, B, W)
    s, p, t = gdr.gdr_beam_select(lg, to_dev(sc), 8)
    want = beam.select(f64(lg[-2:]), sc[-2:].astype(np.float64), 8)
    assert np.array_equal(to_host(p)[-2:], want[1]) and np.array_equal(to_host(t)[-2:], want[2])


def test_reorder_offsets_past_32_bits():
    pool = torch.empty(2, 1100, 1 << 20, dtype=torch.bfloat16, device="cuda")
    pool[1, 1099] = 3.0
    pool[1, 1098] = 4.0
    pool[0, 1099] = 5.0
    idx, par = np.array([[1099, 1098]], np.int32), np.array([[0, 0]], np.int32)
    new = gdr.gdr_beam_reorder(pool, to_dev(idx), to_dev(par), slot_dim=1)
    assert to_host(new).tolist() == [[1099, 1098]]
    assert bool((pool[1, 1098] == 3.0).all()) and bool((pool[0, 1098] == 5.0).all())


# ---------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,W,layers,shape", [(1, 1, 1, (8,)), (3, 4, 1, (2, 128, 64)), (2, 32, 3, (77,)), (5, 7, 2, (1, 1)),
                                              (1, 8, 24, (4096,)), (4, 5, 1, (32, 65, 64))])
def test_reorder(B, W, layers, shape, dt):
    r = np.random.default_rng(B * W)
    slots = B * W + 5
    for trial in range(3):
        pool = torch.randn(layers, slots, *shape, device="cuda").to(dt)
        idx = r.permutation(slots)[:B * W].reshape(B, W).astype(np.int32)
        par = r.integers(0, W, (B, W)).astype(np.int32)
        if trial == 1:
            par[:] = 0
        if trial == 2:
            par = np.tile(np.arange(W, dtype=np.int32)[::-1], (B, 1)).copy()
        want, moves = beam.reorder(idx, par, slots)
        after = pool.clone()
        for s, dst in moves:
            after[:, dst] = pool[:, s]
        new = gdr.gdr_beam_reorder(pool, to_dev(idx), to_dev(par), slot_dim=1)
        torch.cuda.synchronize()
        assert np.array_equal(to_host(new), want)
        assert torch.equal(pool, after)
        assert trial != 2 or not moves


def test_reorder_leaves_padded_and_invalid_rows():
    idx = np.array([[0, 1, 2], [3, -1, 5], [6, 7, 8], [9, 10, 12], [-1, -1, -1]], np.int32)
    par = np.array([[0, 0, 0], [0, 0, 0], [2, 2, 3], [1, 1, 1], [0, 0, 0]], np.int32)
    pool = torch.randn(12, 40, device="cuda")
    before = pool.clone()
    new = gdr.gdr_beam_reorder(pool, to_dev(idx), to_dev(par))
    want = idx.copy()
    before[1] = before[2] = before[0]
    torch.cuda.synchronize()
    assert np.array_equal(to_host(new), want) and torch.equal(pool, before)


def test_reorder_writes_slots_beside_those_it_reads_but_not_over_them():
    idx, par = np.array([[4, 2, 0]], np.int32), np.array([[2, 2, 1]], np.int32)
    buf = torch.zeros(9, dtype=torch.int32, device="cuda")
    buf[:3], buf[6:] = to_dev(par[0]), to_dev(idx[0])
    pool = torch.randn(6, 16, device="cuda")
    want, after = beam.reorder(idx, par, 6)[0], pool.clone()
    after[4] = pool[0]
    args = pool, buf[6:].view(1, 3), buf[:3].view(1, 3)
    for at in (2, 4, 5):
        with pytest.raises(gdr.GdrError):
            gdr.gdr_beam_reorder(*args, state_indices_out=buf[at:at + 3].view(1, 3))
    new = gdr.gdr_beam_reorder(*args, state_indices_out=buf[3:6].view(1, 3))
    torch.cuda.synchronize()
    assert np.array_equal(to_host(new), want) and torch.equal(pool, after)


def test_reorder_unaligned_slots():
    for n in (1, 3, 6, 10):                   # slots of 2, 6, 12, 20 bytes
        pool = torch.randn(2, 8, n, device="cuda").bfloat16()
        after = pool.clone()
        idx, par = np.array([[7, 2, 5]], np.int32), np.array([[1, 1, 1]], np.int32)
        new = gdr.gdr_beam_reorder(pool, to_dev(idx), to_dev(par), slot_dim=1)
        after[:, 7] = after[:, 5] = after[:, 2]
        torch.cuda.synchronize()
        assert to_host(new).tolist() == [[2, 7, 5]] and torch.equal(pool, after)


# ---------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("W,io,pool_dt", [(4, "bf16", "f32"), (3, "bf16", "bf16"), (2, "f32", "f32")])
def test_reorder_of_the_kda_decode_front(W, io, pool_dt):
    """The front's two pools, states and convolution windows: a step, the reordering, a step from the new slots,
    which equals the step from copies of the parents' states in slots of their own."""
    p = inputs.kda_front_problem(70 + W, B=6, q_len=1, H=2, R=16, W=W, num_slots=9, io_dtype=io, pool_dtype=pool_dt)
    d = {n: to_dev(getattr(p, n)) for n in ("q", "k", "v", "conv_weight", "gate_in", "gate_weight", "A_log", "dt_bias", "b",
                                            "conv_bias", "norm_weight", "norm_gate")}

    def step(pool, conv, slots):
        return gdr.gdr_kda_decode_fused(d["q"], d["k"], d["v"], d["conv_weight"], conv, d["gate_in"], d["gate_weight"],
                                        d["A_log"], d["dt_bias"], d["b"], pool, slots, scale=p.scale,
                                        conv_bias=d["conv_bias"], norm_weight=d["norm_weight"], norm_gate=d["norm_gate"])
    pool, conv, idx = to_dev(p.pool), to_dev(p.conv_state), to_dev(p.state_indices)
    step(pool, conv, idx)
    par = to_dev(np.array([[1, 1, 0], [2, 2, 2]], np.int32))
    old = idx.view(2, 3).long()
    of_parent = old.gather(1, par.long()).flatten()
    want_pool, want_conv = pool[of_parent].clone(), conv[of_parent].clone()
    new = gdr.gdr_beam_reorder(pool, idx.view(2, 3), par)
    assert torch.equal(new, gdr.gdr_beam_reorder(conv, idx.view(2, 3), par))
    at = new.flatten().long()
    assert torch.equal(pool[at], want_pool) and torch.equal(conv[at], want_conv)
    o = step(pool, conv, new.flatten())
    want = step(want_pool, want_conv, torch.arange(6, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(pool[at], want_pool) and torch.equal(conv[at], want_conv)


def test_scores_updated_in_place():
    """out_scores may be scores where there are as many results as beams."""
    lg, sc = _logits(71, 5, 6, 9000), _scores(72, 5, 6)
    d, held = _dev_logits(lg, "bf16", 0), to_dev(sc)
    want = gdr.gdr_beam_select(d, held, 6)
    got = gdr.gdr_beam_select(d, held, 6, out_scores=held)
    assert got[0] is held and all(torch.equal(a, b) for a, b in zip(got, want))


def test_largest_batches():
    """65504 rows of beams (65535 is the most), and a reordering of as many and of 65535 layers."""
    B, W, V, K = 2047, 32, 67, 4
    g = torch.Generator(device="cuda").manual_seed(4)
    lg, sc = torch.randn(B, W, V, device="cuda", generator=g), torch.rand(B, W, device="cuda", generator=g)
    s, p, t = gdr.gdr_beam_select(lg, sc, K)
    x = lg.double()
    best, at = (x - torch.logsumexp(x, 2, keepdim=True) + sc.double()[:, :, None]).flatten(1).topk(K + 1)
    clear = (best[:, :-1] - best[:, 1:] > 1e-12).all(1)     # distinct to the rounding of 64-bit sums
    assert int(clear.sum()) > B - 3
    assert torch.equal((p.long() * V + t.long())[clear], at[clear, :K])
    pool = torch.randn(B * W, 2, device="cuda")
    idx = torch.randperm(B * W, device="cuda", generator=g).view(B, W).int()
    want = pool[idx.long().gather(1, p.long()[:, torch.arange(W) % K]).flatten()]
    new = gdr.gdr_beam_reorder(pool, idx, p[:, torch.arange(W) % K].contiguous())
    assert torch.equal(pool[new.flatten().long()], want)
    pool = torch.randn(65535, 3, 2, device="cuda")
    after = pool.clone()
    after[:, 0] = pool[:, 2]
    new = gdr.gdr_beam_reorder(pool, to_dev(np.array([[2, 0]], np.int32)), torch.zeros(1, 2, dtype=torch.int32, device="cuda"), slot_dim=1)
    assert new.tolist() == [[2, 0]] and torch.equal(pool, after)


def test_empty_batches_and_strided_rows():
    i32 = torch.int32
    out = gdr.gdr_beam_select(torch.empty(0, 4, 100, device="cuda"), torch.empty(0, 4, device="cuda"), 7)
    assert [t.shape for t in out] == [(0, 7)] * 3
    pool = torch.randn(5, 8, device="cuda")
    none = torch.empty(0, 4, dtype=i32, device="cuda")
    assert gdr.gdr_beam_reorder(pool, none, none).shape == (0, 4)
    lg = torch.randn(6, 5, 333, device="cuda")
    sc = to_dev(_scores(73, 6, 5))
    for rows in ((slice(None), slice(2, 3)), (slice(3, 4), slice(1, 4)), (slice(1, 5), slice(None))):
        want = gdr.gdr_beam_select(lg[rows].contiguous(), sc[rows].contiguous(), 9)
        got = gdr.gdr_beam_select(lg[rows], sc[rows].contiguous(), 9)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    for bad in (lg[:, 1:3], lg[:, :, ::2], lg.transpose(0, 1)):
        with pytest.raises(ValueError):
            gdr.gdr_beam_select(bad, sc[:bad.shape[0], :bad.shape[1]].contiguous(), 9)


def test_a_captured_step_of_the_search():
    """Decode, selection and reordering of a linear layer's states in one graph, replayed with eager work between
    the replays: each step as the eager one from the same states."""
    B, W, D, V = 3, 4, 192, 1000
    g = torch.Generator(device="cuda").manual_seed(6)
    emb = torch.randn(V, D, device="cuda", generator=g)
    gate = -torch.rand(V, D, device="cuda", generator=g)
    head = torch.randn(D, V, device="cuda", generator=g) * 0.3

    def fresh():
        gg = torch.Generator(device="cuda").manual_seed(7)
        return dict(pool=torch.randn(B * W + 3, D, device="cuda", generator=gg), idx=torch.arange(B * W, device="cuda").view(B, W).int(),
                    scores=-torch.rand(B, W, device="cuda", generator=gg), tok=torch.zeros(B, W, dtype=torch.int32, device="cuda"))

    def step(s):
        t = s["tok"].flatten().long()
        y = gdr.gdr_linear_decode_paged(emb[t], gate[t], gdr.GDR_LINEAR_LOG_DECAY, s["pool"], s["idx"].flatten())
        sc, par, tok = gdr.gdr_beam_select((y @ head).view(B, W, V), s["scores"], W)
        new = gdr.gdr_beam_reorder(s["pool"], s["idx"], par)
        s["scores"].copy_(sc)
        s["tok"].copy_(tok)
        s["idx"].copy_(new)
    a, b = fresh(), fresh()
    warm = fresh()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(warm)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for _ in range(4):
        graph.replay()
        step(b)
        torch.cuda.synchronize()
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_beam_search_over_paged_states():
    """Decode, selection and reordering together: a small model of one delta-rule layer and one linear
    layer, 2 searches of 3 beams for 6 steps.  The states in the slots of each beam, after every step, equal
    the states of running that beam's whole token history from scratch."""
    torch.manual_seed(5)
    dev, B, W, H, K, D, V = "cuda", 2, 3, 2, 64, 128, 50
    emb = {n: torch.randn(V, *s, device=dev) for n, s in dict(q=(H, K), k=(H, K), v=(H, K), x=(D,), g=(D,)).items()}
    emb["q"], emb["k"] = (torch.nn.functional.normalize(emb[n], dim=-1) for n in "qk")
    emb["g"] = -emb["g"].abs()
    decay, beta = -torch.rand(V, H, device=dev), torch.rand(V, H, device=dev)
    head = torch.randn(H * K + D, V, device=dev) * 0.7
    pool_m = torch.zeros(B * W + 2, H, K, K, device=dev)
    pool_c = torch.zeros(B * W + 2, D, device=dev)
    idx = torch.randperm(B * W + 2, device=dev)[:B * W].view(B, W).int()
    scores = torch.tensor([[0.0] + [-np.inf] * (W - 1)] * B, device=dev)
    tokens = torch.zeros(B, W, dtype=torch.int32, device=dev)
    hist = [[[0] for _ in range(W)] for _ in range(B)]

    def step(tok, pm, pc, slots):
        t = tok.flatten().long()
        o = gdr.gdr_decode_paged(emb["q"][t], emb["k"][t], emb["v"][t], decay[t], beta[t], pm, slots, scale=1.0)
        y = gdr.gdr_linear_decode_paged(emb["x"][t], emb["g"][t], gdr.GDR_LINEAR_LOG_DECAY, pc, slots)
        return torch.cat([o.flatten(1), y], 1) @ head

    for _ in range(6):
        logits = step(tokens, pool_m, pool_c, idx.flatten()).view(B, W, V)
        scores, parents, tokens = gdr.gdr_beam_select(logits, scores, W)
        new = gdr.gdr_beam_reorder(pool_m, idx, parents)
        assert torch.equal(new, gdr.gdr_beam_reorder(pool_c, idx, parents))
        idx = new
        par, tok = parents.tolist(), tokens.tolist()
        hist = [[hist[b][par[b][j]] + [tok[b][j]] for j in range(W)] for b in range(B)]
        for b in range(B):
            for j in range(W):
                pm, pc = torch.zeros(1, H, K, K, device=dev), torch.zeros(1, D, device=dev)
                zero = torch.zeros(1, dtype=torch.int32, device=dev)
                for v in hist[b][j][:-1]:
                    step(torch.tensor([v], device=dev), pm, pc, zero)
                assert torch.equal(pool_m[idx[b, j]], pm[0]) and torch.equal(pool_c[idx[b, j]], pc[0])
