"""Gated linear recurrence on the GPU (scan, gradients, paged decode) against the fp64 oracle.

Tolerance per value: u * C * e + half * |value| + tiny, with u = 2^-24, e the oracle's error sum (what a
rounding of every step to u relative accuracy can add up to), half the half step of the stored type and
C = 24: per token the kernels round the gate's exponential and reciprocal (2 u each), their product (u) and
the complement (u), the input b (3 u), the step (2 u), and, where runs are composed, the run's decay (2 u)
and its application (2 u, once for the waves of a tile and once for the tiles), and the first pass over a
run repeats the same roundings as the second: 12 + 12.  The backward pass adds the same terms again in its
own sums (the oracle's e of the gradients holds both)."""
import numpy as np
import pytest
import torch

from _dev import f64, to_dev, to_host
from gated_delta_rule_63_amd import gdr, inputs
from oracle import linear

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
KINDS = {"log": linear.LOG_DECAY, "sigmoid": linear.SIGMOID}


def _cast(x, io):
    x = np.asarray(x, np.float32)
    return inputs.f32_to_bf16_bits(x) if io == "bf16" else x


def _check(got, want, err, half, what):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, what
    off = np.abs(got - want) - (24 * U * err + half * np.abs(want) + 1e-37)
    bad = ~(off <= 0)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {tuple(np.argwhere(bad)[0])}: " \
                          f"{got[bad][0]!r} for {want[bad][0]!r}"


def _problem(seed, lens, D, kind, io, h0=True, tail=0):
    r = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1]) + tail
    if kind == "log":
        gate = -np.exp(r.uniform(np.log(1e-5), np.log(3.0), (1, D))) * r.uniform(0, 1.5, (T, D))
        gate[r.uniform(size=(T, D)) < 0.02] = 0.0
        gate = gate.astype(np.float32)
    else:
        gate = _cast(r.normal(size=(T, D)) * 2 + r.uniform(-3, 9, (1, D)), io)
    p = dict(cu=cu, x=_cast(r.normal(size=(T, D)), io), gate=gate, dy=_cast(r.normal(size=(T, D)), io),
             h0=r.normal(size=(len(lens), D)).astype(np.float32) if h0 else None,
             dF=r.normal(size=(len(lens), D)).astype(np.float32) if h0 else None, kind=KINDS[kind], io=io, T=T, D=D)
    return p


def _wide(v):
    return None if v is None else inputs.widen(v) if v.dtype == np.uint16 else v.astype(np.float64)


def _dev(p):
    return {k: to_dev(p[k]) if p[k] is not None else None for k in ("cu", "x", "gate", "dy", "h0", "dF")}


def _forward(p, d, **kw):
    return gdr.gdr_linear_scan_fwd(d["x"], d["gate"], p["kind"], cu_seqlens=d["cu"], initial_state=d["h0"],
                                   output_block_states=True, **kw)


def _run_both(p):
    d = _dev(p)
    sent = torch.full_like(d["x"], 7.0)
    y, final, blocks = _forward(p, d, y=sent.clone())
    dx, dgate, dh0 = gdr.gdr_linear_scan_bwd(d["x"], d["gate"], p["kind"], d["dy"], blocks, cu_seqlens=d["cu"],
                                             initial_state=d["h0"], d_final_state=d["dF"], dx=sent.clone(),
                                             dgate=torch.full_like(d["gate"], 7.0))
    torch.cuda.synchronize()
    end = int(p["cu"][-1])
    w = {k: _wide(p[k]) for k in ("x", "gate", "dy", "h0", "dF")}
    f = linear.scan(w["x"][:end], w["gate"][:end], p["kind"], p["cu"], w["h0"])
    b = linear.grads(w["x"][:end], w["gate"][:end], p["kind"], p["cu"], w["dy"][:end], w["h0"], w["dF"])
    half = HALF[p["io"]]
    _check(f64(y)[:end], f["y"], f["err"], half, "y")
    _check(f64(final), f["final"], f["err_final"], U, "final")
    _check(f64(dx)[:end], b["dx"], b["err_dx"], half, "dx")
    _check(f64(dgate)[:end], b["dgate"], b["err_dgate"], U if p["kind"] == linear.LOG_DECAY else half, "dgate")
    _check(f64(dh0), b["dh0"], b["err_dh0"], U, "dh0")
    for t in (y, dx, dgate):  # rows behind the last sequence
        assert bool((t[end:] == 7.0).all())
    for k in ("x", "gate", "dy", "h0", "dF", "cu"):
        if p[k] is not None:
            assert np.array_equal(to_host(d[k]), p[k]), f"input {k} changed"


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["log", "sigmoid"])
@pytest.mark.parametrize("D", [1, 63, 256, 260, 515])
def test_one_token_and_one_tile(D, kind, io):
    _run_both(_problem(D, [1], D, kind, io))
    _run_both(_problem(D + 1, [3, 1, 0, 29], D, kind, io))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["log", "sigmoid"])
@pytest.mark.parametrize("lens", [[700], [64, 64, 128], [1] * 70, [63, 1, 65, 0, 0, 127, 200, 1, 0], [0, 0, 5], [129, 511]])
def test_ragged(lens, kind, io):
    _run_both(_problem(sum(lens), lens, 72, kind, io))


@pytest.mark.parametrize("kind", ["log", "sigmoid"])
@pytest.mark.parametrize("D", [7, 64, 320])
def test_long_without_states_and_with_a_tail(D, kind):
    _run_both(_problem(5 + D, [3000, 1, 1500], D, kind, "f32", h0=False, tail=37))
    _run_both(_problem(6 + D, [2049], D, kind, "bf16", tail=64))


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["log", "sigmoid"])
@pytest.mark.parametrize("D", [640, 641])
def test_large_tiles(D, kind, io):
    """Enough tokens and channels for the large tiles, with borders inside them, at their ends, empty sequences
    and rows behind the last one."""
    _run_both(_problem(40 + D, [256, 255, 1, 0, 4096, 128, 64, 0, 1, 1, 1, 3389, 37], D, kind, io, tail=29))


@pytest.mark.parametrize("T", [63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 400, 512, 513])
def test_lengths_around_the_tiles(T):
    _run_both(_problem(60 + T, [T], 66, "log", "bf16"))
    _run_both(_problem(61 + T, [T - 40, 40], 33, "sigmoid", "f32", tail=3))


def test_a_long_chain_of_narrow_tiles():
    _run_both(_problem(70, [30000], 64, "log", "f32"))


def test_many_sequences_and_wide_rows():
    r = np.random.default_rng(9)
    _run_both(_problem(9, r.integers(0, 4, 3000).tolist(), 8, "log", "f32"))
    _run_both(_problem(10, [40, 100], 4100, "sigmoid", "bf16"))


def test_most_sequences():
    """65535 sequences, a third of them empty, in a scan and in a decode step."""
    r = np.random.default_rng(21)
    _run_both(_problem(22, r.integers(0, 3, 65535).tolist(), 3, "sigmoid", "f32", tail=5))
    N, D = 65535, 12
    x, g = torch.randn(N, D, device="cuda"), -torch.rand(N, D, device="cuda")
    pool, slots = torch.randn(N + 9, D, device="cuda"), torch.randperm(N + 9, device="cuda")[:N].int()
    slots[5::7] = -1
    live = slots >= 0
    want = pool.double()
    want[slots[live].long()] = g[live].double().exp() * want[slots[live].long()] + x[live].double()
    y = gdr.gdr_linear_decode_paged(x, g, gdr.GDR_LINEAR_LOG_DECAY, pool, slots, y=torch.full_like(x, 7.0))
    # an exponential (4 u: 2^-23 of the instruction and its argument's rounding), a product and a sum
    bound = 7 * U * (want.abs() + 2 * x.abs().max().item() + 2 * pool.abs().max().item())
    assert bool(((pool.double() - want).abs() <= bound).all())
    assert torch.equal(y[live], pool[slots[live].long()]) and bool((y[~live] == 7.0).all())


def test_decode_of_no_sequences():
    x, i = torch.empty(0, 40, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    pool = torch.randn(3, 40, device="cuda")
    before = pool.clone()
    y = gdr.gdr_linear_decode_paged(x, x, gdr.GDR_LINEAR_LOG_DECAY, pool, i)
    assert y.shape == (0, 40) and torch.equal(pool, before)


@pytest.mark.parametrize("D", [64, 65])
def test_no_cu_seqlens_equals_one_sequence(D):
    p = _problem(11, [1000], D, "log", "bf16")
    d = _dev(p)
    one = _forward(p, d)
    d["cu"] = None
    two = _forward(p, d)
    for a, b in zip(one, two):
        assert torch.equal(a, b)
    g = [gdr.gdr_linear_scan_bwd(d["x"], d["gate"], p["kind"], d["dy"], one[2], cu_seqlens=c, initial_state=d["h0"],
                                 d_final_state=d["dF"]) for c in (None, to_dev(p["cu"]))]
    for a, b in zip(*g):
        assert torch.equal(a, b)


def test_slow_channels_with_constant_input():
    """Decays of 1e-6 to 1e-4 per token over 20000 tokens of constant input: the state is a multiple of its
    last place and every step adds the same amount, so the roundings of neighbouring steps all point the same
    way and add up: e[t] = a e[t-1] + h[t] roundings of the state.  Per token the kernels round the state once
    in a step, once more in the run's own first pass, and the run's decay twice (its effect is that share of
    the state): 4 u e, which no order of the fp32 recurrence can avoid."""
    T, D = 20000, 64
    g = -np.exp(np.linspace(np.log(1e-6), np.log(1e-4), D)).astype(np.float32)[None].repeat(T, 0)
    x = np.ones((T, D), np.float32)
    y, final = gdr.gdr_linear_scan_fwd(to_dev(x), to_dev(g), gdr.GDR_LINEAR_LOG_DECAY)
    t = np.arange(1, T + 1)[:, None]

    def check(got, log_a, b):
        want = b * np.expm1(log_a * t) / np.expm1(log_a)
        e, tol = np.zeros_like(want[0]), np.empty_like(want)
        for i in range(T):
            e = np.exp(log_a) * e + want[i]
            tol[i] = 4 * U * e
        assert np.all(np.abs(got - want) <= tol)
    check(f64(y), g[0].astype(np.float64), 1.0)
    z = np.full((T, D), 11.0, np.float32)      # 1 - a = 1.7e-5
    y, _ = gdr.gdr_linear_scan_fwd(to_dev(x), to_dev(z), gdr.GDR_LINEAR_SIGMOID)
    q = 1 / (1 + np.exp(11.0))
    # b = q x holds three roundings of q, in the same direction every token
    check(f64(y) / (1 + 3 * U), np.full(D, np.log1p(-q)), q)


def test_slow_channels_keep_their_decay():
    """The same decays with inputs that differ, so that the states' roundings do not line up: their random sum
    is at most sqrt(4 T) u = 1.7e-5 of the state, and 6e-5 leaves 3.5 of that.  A decay rounded to u of 1 would
    be off by up to u / 2 in every token, T u / 2 = 6e-4 at the last and half of it over the norm."""
    r = np.random.default_rng(31)
    T, D = 20000, 64
    g = -np.exp(np.linspace(np.log(1e-6), np.log(1e-4), D)).astype(np.float32)[None].repeat(T, 0)
    x, h0 = r.normal(size=(T, D)).astype(np.float32), r.uniform(100, 200, (1, D)).astype(np.float32)
    y, _ = gdr.gdr_linear_scan_fwd(to_dev(x), to_dev(g), gdr.GDR_LINEAR_LOG_DECAY, initial_state=to_dev(h0))
    want = linear.scan(x, g, linear.LOG_DECAY, [0, T], h0)["y"]
    off = np.linalg.norm(f64(y) - want, axis=0) / np.linalg.norm(want, axis=0)
    assert off.max() < 6e-5


@pytest.mark.parametrize("T", [40, 900])
def test_special_values_stay_in_their_sequence_and_channel(T):
    p = _problem(12, [T, T, T], 68, "log", "f32")
    p["x"][T + 5, 3] = np.nan
    p["x"][T + 6, 4] = np.inf
    p["gate"][T + 7, 5] = np.nan
    p["gate"][T + 8, 6] = -np.inf            # forgets everything
    p["h0"][1, 7] = np.inf
    p["dy"][2 * T - 3, 8] = np.nan
    d = _dev(p)
    y, final, blocks = _forward(p, d)
    dx, dg, dh0 = gdr.gdr_linear_scan_bwd(d["x"], d["gate"], p["kind"], d["dy"], blocks, cu_seqlens=d["cu"],
                                          initial_state=d["h0"], d_final_state=d["dF"])
    y, dx, dg = f64(y), f64(dx), f64(dg)
    clean = {k: v.copy() if isinstance(v, np.ndarray) else v for k, v in p.items()}
    mid = slice(T, 2 * T)
    f = linear.scan(*(clean[k].astype(np.float64) for k in ("x", "gate")), p["kind"], p["cu"], p["h0"])
    touched = [3, 4, 5, 7]
    rest = [c for c in range(68) if c not in touched]
    for s in (slice(0, T), slice(2 * T, 3 * T)):
        _check(y[s], f["y"][s], f["err"][s], U, "other sequences")
        assert np.isfinite(dx[s]).all() and np.isfinite(dg[s]).all()
    with np.errstate(invalid="ignore"):
        _check(y[mid][:, rest], f["y"][mid][:, rest], f["err"][mid][:, rest], U, "other channels")
    assert np.isfinite(y[T:T + 5, 3]).all() and np.isnan(y[T + 5:2 * T, 3]).all()
    assert np.isfinite(y[T:T + 6, 4]).all() and np.isposinf(y[T + 6, 4]) and not np.isfinite(y[T + 6:2 * T, 4]).any()
    assert np.isnan(y[T + 7:2 * T, 5]).all()
    assert y[T + 8, 6] == p["x"][T + 8, 6] and dg[T + 8, 6] == 0
    assert np.isnan(dx[T:2 * T - 2, 8]).all() and np.isfinite(dx[2 * T - 2:2 * T, 8]).all()
    nan_free = [c for c in rest if c not in (6, 8)]
    assert np.isfinite(dx[:, nan_free]).all() and np.isfinite(dg[:, nan_free]).all()
    assert np.isfinite(f64(dh0)[[0, 2]]).all()


@pytest.mark.parametrize("T", [40, 900])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_special_values_of_the_sigmoid_gate(T, io):
    """Lowest values as inputs and gates are ordinary numbers; infinities and NaN stay where they are."""
    p = _problem(19, [T, T, T], 68, "sigmoid", "f32")
    low = inputs.widen(inputs.f32_to_bf16_bits(np.array([-3.3e38], np.float32)))[0]
    x, z = p["x"].astype(np.float64), p["gate"].astype(np.float64)
    x[T + 4, 1], x[T + 5, 2], z[T + 6, 3], z[T + 7, 4] = low, -low, low, -low   # forget all, keep all
    x[T + 5, 10], x[T + 5, 11], x[T + 6, 12], z[T + 7, 13] = np.inf, -np.inf, np.nan, np.nan
    z[T + 5, 10:12] = 3.0, -3.0                  # a near 1, a near 0
    z[T + 8, 14], z[T + 9, 15] = -np.inf, np.inf
    p["x"], p["gate"], p["io"] = _cast(x, io), _cast(z, io), io
    p["dy"] = _cast(p["dy"], io)
    d = _dev(p)
    y, final, blocks = _forward(p, d)
    dx, dz, dh0 = gdr.gdr_linear_scan_bwd(d["x"], d["gate"], p["kind"], d["dy"], blocks, cu_seqlens=d["cu"],
                                          initial_state=d["h0"], d_final_state=d["dF"])
    y, dx, dz = f64(y), f64(dx), f64(dz)
    with np.errstate(invalid="ignore"):
        f = linear.scan(_wide(p["x"]), _wide(p["gate"]), p["kind"], p["cu"], p["h0"])
    rest = [c for c in range(68) if c not in (10, 11, 12, 13)]
    for s in (slice(0, T), slice(2 * T, 3 * T)):
        _check(y[s], f["y"][s], f["err"][s], HALF[io], "other sequences")
        assert np.isfinite(dx[s]).all() and np.isfinite(dz[s]).all()
    mid = slice(T, 2 * T)
    _check(y[mid][:, rest], f["y"][mid][:, rest], f["err"][mid][:, rest], HALF[io], "other channels")
    for c, t in ((10, 5), (11, 5), (12, 6), (13, 7)):
        assert np.isfinite(y[T:T + t, c]).all() and not np.isfinite(y[T + t:2 * T, c]).any()
    assert np.isposinf(y[T + 5, 10])
    for t, c in ((6, 3), (8, 14)):
        assert y[T + t, c] == _wide(p["x"])[T + t, c]
    plain = [c for c in rest if c not in (1, 2)]  # the lowest values' gates have gradients past fp32
    assert np.isfinite(dx[:, plain]).all() and np.isfinite(dz[:, plain]).all()
    assert np.isfinite(f64(dh0)[[0, 2]]).all()


def test_misaligned_rows_take_the_narrow_path():
    p = _problem(13, [300, 20], 64, "sigmoid", "bf16")
    d = _dev(p)
    want = _forward(p, d)
    off = torch.empty(d["x"].numel() + 1, dtype=torch.bfloat16, device="cuda")[1:].view_as(d["x"])
    off.copy_(d["x"])
    got = gdr.gdr_linear_scan_fwd(off, d["gate"], p["kind"], cu_seqlens=d["cu"], initial_state=d["h0"])
    w = {k: _wide(p[k]) for k in ("x", "gate", "h0")}
    f = linear.scan(w["x"], w["gate"], p["kind"], p["cu"], w["h0"])
    for y, final in (want[:2], got):
        _check(f64(y), f["y"], f["err"], HALF["bf16"], "y")
        _check(f64(final), f["final"], f["err_final"], U, "final")


def test_calls_are_repeatable_and_captured():
    p = _problem(14, [2000, 800], 200, "sigmoid", "bf16")
    d = _dev(p)
    want = _forward(p, d)
    bw = lambda blocks, **kw: gdr.gdr_linear_scan_bwd(d["x"], d["gate"], p["kind"], d["dy"], blocks,  # noqa: E731
                                                      cu_seqlens=d["cu"], initial_state=d["h0"],
                                                      d_final_state=d["dF"], **kw)
    want_b = bw(want[2])
    need = gdr.gdr_linear_workspace_size(d["x"], d["gate"], p["kind"], 2)
    ws = torch.full((need,), 0x5A, dtype=torch.uint8, device="cuda")  # need not be initialised
    out = [torch.empty_like(t) for t in want]
    out_b = [torch.empty_like(t) for t in want_b]
    torch.cuda.synchronize()

    def call():
        _forward(p, d, y=out[0], final_state=out[1], block_states=out[2], workspace=ws)
        bw(out[2], dx=out_b[0], dgate=out_b[1], d_initial_state=out_b[2], workspace=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        for t in out + out_b:
            t.zero_()
        g.replay()
        _forward(p, d)  # the program's own work between replays
        torch.cuda.synchronize()
        for a, b in zip(out + out_b, list(want) + list(want_b)):
            assert torch.equal(a, b)


def test_states_beside_each_other():
    """Initial and final states, and their gradients, as neighbours in one buffer, and over one another."""
    p = _problem(18, [700, 41], 64, "log", "f32")
    d = _dev(p)
    want = _forward(p, d)
    bw = dict(cu_seqlens=d["cu"], initial_state=d["h0"])
    want_b = gdr.gdr_linear_scan_bwd(d["x"], d["gate"], p["kind"], d["dy"], want[2], d_final_state=d["dF"], **bw)
    buf = torch.empty(5, 64, device="cuda")
    buf[:2] = d["dF"]
    got = gdr.gdr_linear_scan_bwd(d["x"], d["gate"], p["kind"], d["dy"], want[2], d_final_state=buf[:2],
                                  d_initial_state=buf[2:4], **bw)
    for a, b in zip(got, want_b):
        assert torch.equal(a, b)
    with pytest.raises(gdr.GdrError):
        gdr.gdr_linear_scan_bwd(d["x"], d["gate"], p["kind"], d["dy"], want[2], d_final_state=buf[:2],
                                d_initial_state=buf[1:3], **bw)
    buf[2:4] = d["h0"]
    d["h0"] = buf[2:4]
    for a, b in zip(_forward(p, d, final_state=buf[:2]), want):
        assert torch.equal(a, b)
    for at in (1, 2, 3):
        with pytest.raises(gdr.GdrError):
            _forward(p, d, final_state=buf[at:at + 2])


@pytest.mark.parametrize("kind,io", [("log", "f32"), ("sigmoid", "bf16")])
def test_the_two_scans_as_an_autograd_function(kind, io):
    """The layer that a user writes from them: its gradients are the gradients of every input."""
    class Scan(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, gate, h0, cu):
            y, final, blocks = gdr.gdr_linear_scan_fwd(x, gate, KINDS[kind], cu_seqlens=cu, initial_state=h0,
                                                       output_block_states=True)
            ctx.save_for_backward(x, gate, h0, cu, blocks)
            return y, final

        @staticmethod
        def backward(ctx, dy, d_final):
            x, gate, h0, cu, blocks = ctx.saved_tensors
            return *gdr.gdr_linear_scan_bwd(x, gate, KINDS[kind], dy.contiguous(), blocks, cu_seqlens=cu, initial_state=h0,
                                            d_final_state=d_final.contiguous()), None
    p = _problem(23, [130, 0, 77, 1], 66, kind, io)
    d = _dev(p)
    leaves = [d[k].requires_grad_() for k in ("x", "gate", "h0")]
    y, final = Scan.apply(*leaves, d["cu"])
    torch.autograd.backward([y, final], [d["dy"], d["dF"]])
    w = {k: _wide(p[k]) for k in ("x", "gate", "dy", "h0", "dF")}
    b = linear.grads(w["x"], w["gate"], p["kind"], p["cu"], w["dy"], w["h0"], w["dF"])
    for t, name in zip(leaves, ("dx", "dgate", "dh0")):
        _check(f64(t.grad), b[name], b["err_" + name], HALF["bf16"] if t.dtype == torch.bfloat16 else U, name)


def test_another_stream():
    p = _problem(15, [5000], 512, "log", "bf16")
    d = _dev(p)
    want = _forward(p, d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [_forward(p, d, stream=s) for _ in range(4)]
    big = [torch.full((1 << 22,), float(i), device="cuda") for i in range(4)]  # work on the current stream meanwhile
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)
    assert all(bool((b == i).all()) for i, b in enumerate(big))


def test_two_streams_at_once():
    """Chains of two calls in flight together, each with its own workspace."""
    p, q = _problem(16, [9000], 512, "log", "bf16"), _problem(17, [7000, 3000], 513, "sigmoid", "f32")
    d, e = _dev(p), _dev(q)
    want, want2 = _forward(p, d), _forward(q, e)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = [(_forward(p, d, stream=s1), _forward(q, e, stream=s2)) for _ in range(5)]
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(x, y) for x, y in zip(a, want)) and all(torch.equal(x, y) for x, y in zip(b, want2))


def test_batches_without_tokens():
    x, g = torch.empty(0, 40, device="cuda"), torch.empty(0, 40, device="cuda")
    h0, cu = torch.randn(3, 40, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    y, final, blocks = gdr.gdr_linear_scan_fwd(x, g, gdr.GDR_LINEAR_LOG_DECAY, cu_seqlens=cu, initial_state=h0,
                                               output_block_states=True)
    dx, dg, dh0 = gdr.gdr_linear_scan_bwd(x, g, gdr.GDR_LINEAR_LOG_DECAY, x, blocks, cu_seqlens=cu, initial_state=h0,
                                          d_final_state=h0 * 2)
    assert y.shape == x.shape and torch.equal(final, h0) and torch.equal(dh0, h0 * 2)
    y, final = gdr.gdr_linear_scan_fwd(x, g, gdr.GDR_LINEAR_LOG_DECAY, cu_seqlens=cu)
    assert bool((final == 0).all())
    y, final = gdr.gdr_linear_scan_fwd(x, g, gdr.GDR_LINEAR_LOG_DECAY, cu_seqlens=cu[:1])   # no sequences
    assert final.shape == (0, 40)
    # all sequences empty, rows behind them
    x, g = torch.randn(300, 40, device="cuda"), -torch.rand(300, 40, device="cuda")
    y = torch.full_like(x, 7.0)
    _, final = gdr.gdr_linear_scan_fwd(x, g, gdr.GDR_LINEAR_LOG_DECAY, cu_seqlens=cu, initial_state=h0, y=y)
    assert torch.equal(final, h0) and bool((y == 7.0).all())


@pytest.mark.parametrize("T", [1, 300])
def test_widest_rows(T):
    """2^22 channels, the most: constant gates, so that every channel's state is known."""
    D = 1 << 22
    x = torch.full((T, D), 2.0, device="cuda", dtype=torch.bfloat16)
    g = torch.full((T, D), float(np.log(0.5)), device="cuda")
    y, final, blocks = gdr.gdr_linear_scan_fwd(x, g, gdr.GDR_LINEAR_LOG_DECAY, output_block_states=True)
    want = 4.0 * (1.0 - 0.5 ** np.arange(1, T + 1))   # the oracle's error sum is below 40 here
    for t in {0, T - 1, T // 2}:
        assert bool(((y[t].float() - want[t]).abs() <= HALF["bf16"] * want[t] + 24 * U * 40).all())
    assert bool(((final[0] - want[-1]).abs() <= 24 * U * 40).all())
    del y
    dx, dg, dh0 = gdr.gdr_linear_scan_bwd(x, g, gdr.GDR_LINEAR_LOG_DECAY, x, blocks)
    D0 = 4.0 * (1.0 - 0.5 ** T)                        # gradients run the other way
    assert bool(((dx[0].float() - D0).abs() <= HALF["bf16"] * D0 + 24 * U * 40).all())
    assert bool(((dh0[0] - D0 / 2).abs() <= 24 * U * 40).all()) and bool((dg[0] == 0).all())


def test_sizes_past_32_bits_are_refused():
    """2^32 + 64 channels, tokens of a vocabulary or slots: not taken for 64 of them."""
    n, i32 = (1 << 32) + 64, torch.int32
    x, idx = torch.empty(1, n, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, dtype=i32, device="cuda")
    with pytest.raises(ValueError):
        gdr.gdr_linear_scan_fwd(x, x, gdr.GDR_LINEAR_SIGMOID)
    with pytest.raises(ValueError):
        gdr.gdr_linear_decode_paged(x, x, gdr.GDR_LINEAR_SIGMOID, x, idx)
    with pytest.raises(ValueError):
        gdr.gdr_linear_decode_paged(x[:, :1].contiguous(), x[:, :1].contiguous(), gdr.GDR_LINEAR_SIGMOID, x.view(n, 1), idx)
    with pytest.raises(ValueError):
        gdr.gdr_beam_select(x[None], torch.zeros(1, 1, device="cuda"), 1)
    with pytest.raises(ValueError):
        gdr.gdr_beam_reorder(x.view(n, 1), idx[None], idx[None])
    some = torch.zeros(1, 1, 8, device="cuda")
    for bad in (dict(num_out=(1 << 32) + 1), dict(num_out=1, eos_token=1 << 32, finished=torch.zeros(1, 1, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            gdr.gdr_beam_select(some, some[:, :, 0].contiguous(), **bad)
    one = torch.zeros(1, 8, device="cuda")
    with pytest.raises(ValueError):
        gdr.gdr_linear_decode_paged(one, one, gdr.GDR_LINEAR_LOG_DECAY, one, idx, max_q_len=(1 << 32) + 1)


def test_offsets_past_32_bits():
    """2^31 elements and more: the last rows (for the gradients: the first), which gates of one half forget
    everything 300 tokens away from, against the oracle on those rows alone."""
    T, D, n = (1 << 20) + 77, 2112, 300
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, D, device="cuda", dtype=torch.bfloat16, generator=g)
    z = torch.randn(T, D, device="cuda", dtype=torch.bfloat16, generator=g)
    y, final, blocks = gdr.gdr_linear_scan_fwd(x, z, gdr.GDR_LINEAR_SIGMOID, output_block_states=True)
    f = linear.scan(f64(x[-n:]), f64(z[-n:]), linear.SIGMOID, [0, n])
    _check(f64(y[-40:]), f["y"][-40:], f["err"][-40:], HALF["bf16"], "y")
    _check(f64(final), f["final"], f["err_final"], U, "final")
    del y
    dx, dz, dh0 = gdr.gdr_linear_scan_bwd(x, z, gdr.GDR_LINEAR_SIGMOID, x, blocks)
    for rows, keep in ((slice(0, n), slice(0, 40)), (slice(T - n, T), slice(n - 40, n))):
        b = linear.grads(f64(x[rows]), f64(z[rows]), linear.SIGMOID, [0, n], f64(x[rows]))
        _check(f64(dx[rows])[keep], b["dx"][keep], b["err_dx"][keep], HALF["bf16"], "dx")
        _check(f64(dz[rows])[keep], b["dgate"][keep], b["err_dgate"][keep], HALF["bf16"], "dz")
        if rows.start == 0:
            _check(f64(dh0), b["dh0"], b["err_dh0"], U, "dh0")
    # a pool of the same size: its last slot
    slots = torch.tensor([T - 1, 5], dtype=torch.int32, device="cuda")
    before = f64(x[[T - 1, 5, T - 2]])
    o = gdr.gdr_linear_decode_paged(z[:2].contiguous(), z[2:4].contiguous(), gdr.GDR_LINEAR_SIGMOID, x, slots)
    want, last, err, err_last = linear.decode_paged(f64(z[:2]), f64(z[2:4]), linear.SIGMOID, [0, 1, 2], before, [0, 1])
    _check(f64(o), want, err, HALF["bf16"], "y")
    _check(f64(x[[T - 1, 5]]), np.stack([last[0], last[1]]), np.stack([err_last[0], err_last[1]]), HALF["bf16"], "pool")
    assert np.array_equal(f64(x[T - 2]), before[2])


# ---------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind", ["log", "sigmoid"])
@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("pool_dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,q", [(1, 1), (100, 1), (37, 12), (1024, 3), (1030, 5)])
def test_decode(D, q, pool_dt, io, kind):
    r = np.random.default_rng(D + q)
    n = 9
    lens = r.integers(0 if q > 1 else 1, q + 1, n)
    lens[3] = q
    p = _problem(20 + D, lens.tolist(), D, kind, io, h0=False)
    pool = _cast(r.normal(size=(14, D)), pool_dt)
    slots = r.permutation(14)[:n].astype(np.int32)
    slots[[1, 6]] = -1
    for commit in (False, True):
        d, dpool = _dev(p), to_dev(pool)
        y = torch.full_like(d["x"], 7.0)
        gdr.gdr_linear_decode_paged(d["x"], d["gate"], p["kind"], dpool, to_dev(slots), cu_seqlens=d["cu"], max_q_len=q,
                                    commit=commit, y=y)
        torch.cuda.synchronize()
        want, final, err, err_final = linear.decode_paged(_wide(p["x"]), _wide(p["gate"]), p["kind"], p["cu"],
                                                          _wide(pool), slots)
        live = ~np.isnan(want)
        got = f64(y)
        assert (got[~live] == 7.0).all()
        _check(got[live], want[live], err[live], HALF[io], "y")
        after = to_host(dpool)
        kept = [s for s in range(14) if not commit or s not in final]
        assert np.array_equal(after[kept], pool[kept])
        if commit:
            for s in final:
                _check(inputs.widen(after[s]) if pool_dt == "bf16" else after[s], final[s], err_final[s],
                       HALF[pool_dt], "pool")


def test_decode_continues_a_scan():
    """Prefill, then token by token from its final states: the same outputs as one scan over everything."""
    p = _problem(30, [300, 41], 96, "sigmoid", "f32", h0=False)
    d = _dev(p)
    y, _ = gdr.gdr_linear_scan_fwd(d["x"], d["gate"], p["kind"], cu_seqlens=d["cu"])
    cut = [(0, 290), (300, 331)]
    rows = torch.cat([torch.arange(a, b) for a, b in cut]).cuda()
    cu = torch.tensor([0, 290, 321], dtype=torch.int32, device="cuda")
    _, final = gdr.gdr_linear_scan_fwd(d["x"][rows].contiguous(), d["gate"][rows].contiguous(), p["kind"], cu_seqlens=cu)
    pool = torch.zeros(5, 96, device="cuda")
    idx = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    pool[idx.long()] = final
    f = linear.scan(_wide(p["x"]), _wide(p["gate"]), p["kind"], p["cu"])
    for i in range(10):
        at = torch.tensor([290 + i, 331 + i], device="cuda")
        o = gdr.gdr_linear_decode_paged(d["x"][at].contiguous(), d["gate"][at].contiguous(), p["kind"], pool, idx)
        a = at.cpu().numpy()
        _check(f64(o), f["y"][a], f["err"][a], U, "y")
        _check(f64(y[at]), f["y"][a], f["err"][a], U, "scan")
