"""Host-side refusals of the gated linear recurrence's and beam search's entry points (CPU: validation
fails before any launch, or the problem is empty)."""
import ctypes

import pytest
import torch

from gated_delta_rule_63_amd import gdr

PTR = ctypes.c_void_p(0x1000)  # never dereferenced
ODD = ctypes.c_void_p(0x1010)


def _lp(T=100, N=2, D=64, gate=0, io=1):
    return gdr.LinearProblem(T, N, D, gate, io)


def _fwd(p, x=PTR, gate=PTR, cu=PTR, y=PTR, ht=None, ws=PTR, nb=1 << 20):
    return gdr.lib().gdr_linear_scan_fwd(ctypes.byref(p) if p else None, x, gate, cu, None, y, ht, None, ws, nb, None)


def _bwd(p, x=PTR, gate=PTR, cu=PTR, bs=PTR, dy=PTR, dx=PTR, dg=PTR, dh0=None, ws=PTR, nb=1 << 20):
    return gdr.lib().gdr_linear_scan_bwd(ctypes.byref(p) if p else None, x, gate, cu, None, bs, dy, None, dx, dg, dh0,
                                         ws, nb, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
@pytest.mark.parametrize("p,expect", [
    (None, 1), (_lp(T=-1), 1), (_lp(N=-1), 1), (_lp(D=0), 1), (_lp(gate=2), 1), (_lp(io=3), 1),
    (_lp(N=0), 1), (_lp(N=65536), 2), (_lp(T=1 << 40, D=1 << 20), 2), (_lp(D=(1 << 22) + 1), 2)])
def test_scan_rejects_bad_metadata(call, p, expect):
    assert call(p) == expect


@pytest.mark.parametrize("call,names", [(_fwd, "x gate y"), (_bwd, "x gate bs dy dx dg")])
def test_scan_rejects_missing_tensors_and_workspaces(call, names):
    for n in names.split():
        assert call(_lp(), **{n: None}) == 1, n
    assert call(_lp(), cu=None) == 1                       # N > 1
    assert call(_lp(), ws=None) == 1
    assert call(_lp(), ws=ODD) == 1                        # not 256-byte aligned
    need = gdr.lib().gdr_linear_workspace_size(ctypes.byref(_lp()))
    assert need > 0 and call(_lp(), nb=need - 1) == 1


def test_scan_accepts_empty_batches_without_the_device():
    assert _fwd(_lp(T=0, N=0), x=None, gate=None, y=None, cu=None, ws=None, nb=0) == 0
    assert _fwd(_lp(T=0, N=3), x=None, gate=None, y=None, ws=None, nb=0) == 0
    assert _bwd(_lp(T=0, N=3), x=None, gate=None, bs=None, dy=None, dx=None, dg=None, ws=None, nb=0) == 0


@pytest.mark.parametrize("off", [-508, -4, 0, 4, 508])
def test_scan_rejects_states_written_over_those_it_reads(off):
    """2 x 64 fp32 states: 512 bytes."""
    L, p, here, there = gdr.lib(), ctypes.byref(_lp()), ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10000 + off)
    assert L.gdr_linear_scan_fwd(p, PTR, PTR, PTR, here, PTR, there, None, PTR, 1 << 20, None) == 1
    assert L.gdr_linear_scan_bwd(p, PTR, PTR, PTR, None, PTR, PTR, here, PTR, PTR, there, PTR, 1 << 20, None) == 1


def test_scan_workspace_size():
    size = lambda **k: gdr.lib().gdr_linear_workspace_size(ctypes.byref(_lp(**k)))  # noqa: E731
    assert size(T=0) == 0 and size(D=0) == 0
    # it grows with tokens and channels, and its size is 64-bit
    assert 0 < size(T=6400, D=64) < size(T=6400, D=128) < size(T=12800, D=128)
    assert size(T=1 << 28, D=4096) > 1 << 32


def _dec(p, q=1, x=PTR, gate=PTR, cu=None, pool=PTR, pdt=0, slots=4, idx=PTR, commit=1, y=PTR):
    return gdr.lib().gdr_linear_decode_paged(ctypes.byref(p), q, x, gate, cu, pool, pdt, slots, idx, commit, y, None)


def test_decode_rejects_bad_metadata():
    p = _lp(T=4, N=4)
    for kw in (dict(q=0), dict(q=13), dict(pool=None), dict(slots=0), dict(idx=None), dict(pdt=4), dict(commit=2),
               dict(x=None), dict(gate=None), dict(y=None)):
        assert _dec(p, **kw) == 1, kw
    assert _dec(_lp(T=5, N=4)) == 1                        # no cu_seqlens but T != N
    assert _dec(_lp(T=30, N=2), q=12, cu=PTR) == 1         # T > N max_q_len
    assert _dec(_lp(T=0, N=4), cu=PTR) == 0


def test_decode_of_no_sequences_needs_no_indices():
    assert _dec(_lp(T=0, N=0), x=None, gate=None, idx=None, y=None) == 0
    assert _dec(_lp(T=0, N=1), cu=PTR, x=None, gate=None, idx=None, y=None) == 1


def _bp(B=2, W=4, V=100, K=8, stride=100, eos=0, io=1):
    return gdr.BeamProblem(B, W, V, K, stride, eos, io)


def _sel(p, lg=PTR, sc=PTR, fin=None, o=PTR, ws=PTR, nb=1 << 24):
    return gdr.lib().gdr_beam_select(ctypes.byref(p) if p else None, lg, sc, fin, o, o, o, ws, nb, None)


@pytest.mark.parametrize("p,expect", [
    (None, 1), (_bp(B=-1), 1), (_bp(W=0), 1), (_bp(V=0), 1), (_bp(K=0), 1), (_bp(V=7, K=8), 1), (_bp(stride=99), 1),
    (_bp(io=2), 1), (_bp(W=33), 2), (_bp(K=65), 2), (_bp(V=(1 << 20) + 1, stride=1 << 21), 2), (_bp(B=20000), 2)])
def test_select_rejects_bad_metadata(p, expect):
    assert _sel(p) == expect
    if p is not None:
        assert gdr.lib().gdr_beam_workspace_size(ctypes.byref(p)) == 0


def test_select_rejects_missing_tensors():
    assert _sel(_bp(), lg=None) == 1 and _sel(_bp(), sc=None) == 1 and _sel(_bp(), o=None) == 1
    assert _sel(_bp(), ws=None) == 1 and _sel(_bp(), ws=ODD) == 1
    need = gdr.lib().gdr_beam_workspace_size(ctypes.byref(_bp()))
    assert need > 0 and _sel(_bp(), nb=need - 1) == 1
    assert _sel(_bp(eos=-1), fin=PTR) == 1 and _sel(_bp(eos=100), fin=PTR) == 1
    assert _sel(_bp(B=0), lg=None, sc=None, o=None, ws=None, nb=0) == 0


def _reo(B=2, W=4, par=PTR, idx=ctypes.c_void_p(0x2000), out=ctypes.c_void_p(0x3000), pool=PTR, L=1, S=16, nb=64):
    return gdr.lib().gdr_beam_reorder(B, W, par, idx, out, pool, L, S, nb, None)


def test_reorder_rejects_bad_metadata():
    for kw in (dict(B=-1), dict(W=0), dict(L=-1), dict(S=0), dict(nb=0), dict(nb=63), dict(pool=ctypes.c_void_p(0x1001)),
               dict(par=None), dict(idx=None), dict(out=None), dict(pool=None), dict(out=ctypes.c_void_p(0x2000)),
               dict(out=PTR)):
        assert _reo(**kw) == 1, kw
    assert _reo(W=33) == 2 and _reo(B=20000) == 2 and _reo(L=65536) == 2
    assert _reo(B=0) == 0 and _reo(L=0) == 0


def test_reorder_rejects_slots_written_over_those_it_reads():
    for base in (0x1000, 0x2000):                          # parents, state_indices: 2 x 4 entries of 4 bytes
        for off in (-28, -4, 0, 4, 28):
            assert _reo(out=ctypes.c_void_p(base + off)) == 1, (hex(base), off)


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        gdr.gdr_linear_scan_fwd(x, x, gdr.GDR_LINEAR_LOG_DECAY)
    with pytest.raises(ValueError):
        gdr.gdr_linear_decode_paged(x, x, gdr.GDR_LINEAR_LOG_DECAY, x, torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        gdr.gdr_beam_select(torch.zeros(1, 2, 8), torch.zeros(1, 2), 2)
    with pytest.raises(ValueError):
        gdr.gdr_beam_reorder(x, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32))
