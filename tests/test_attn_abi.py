"""Host-side refusals of the full-attention entry points (CPU: validation fails before any launch, or the problem is
empty)."""
import ctypes

import pytest
import torch

from gated_delta_rule_63_amd import gdr

PTR = ctypes.c_void_p(0x10000)  # never dereferenced
ODD = ctypes.c_void_p(0x10008)


def _ap(T=100, N=2, HQ=8, HK=2, D=64, scale=0.1, q=512, k=128, v=128, io=1):
    return gdr.AttnProblem(T, N, HQ, HK, D, scale, q, k, v, io)


def _kp(k=PTR, v=PTR, table=PTR, n=8, size=16, most=4):
    return gdr.KvPages(k, v, table, n, size, most)


def _rot(freq=PTR, pos=None, R=64, axes=1, inter=0):
    return gdr.Rotary(freq, pos, R, axes, inter)


def _ref(x):
    return ctypes.byref(x) if x is not None else None


FAR = dict(q=ctypes.c_void_p(1 << 32), k=ctypes.c_void_p(2 << 32), v=ctypes.c_void_p(3 << 32), qo=ctypes.c_void_p(4 << 32),
           ko=ctypes.c_void_p(5 << 32))


def _append(p=None, r=None, pages="some", cu=PTR, ctx=PTR, **kw):
    a = dict(FAR, **kw)
    return gdr.lib().gdr_rope_append_paged(_ref(_ap() if p is None else p), _ref(_rot() if r is None else r), a["q"], a["k"],
                                           a["v"], cu, ctx, _ref(_kp() if pages == "some" else pages), a["qo"], a["ko"], None)


def _prefill(p, q=PTR, k=PTR, v=PTR, cu=PTR, o=PTR):
    return gdr.lib().gdr_attn_prefill_fwd(_ref(p), q, k, v, cu, o, None, None)


def _decode(p, ql=12, q=PTR, cu=PTR, ctx=PTR, pages="some", G=0, off=None, pre=None, o=PTR, ws=PTR, nb=1 << 40):
    return gdr.lib().gdr_attn_decode_paged(_ref(p), ql, q, cu, ctx, _ref(_kp() if pages == "some" else pages), G, off, pre, o,
                                           None, ws, nb, None)


BAD = [(_ap(T=-1), 1), (_ap(N=-1), 1), (_ap(HQ=0), 1), (_ap(HK=0), 1), (_ap(HQ=9), 1), (_ap(D=0), 1), (_ap(io=2), 1),
       (_ap(scale=float("nan")), 1), (_ap(scale=float("inf")), 1), (_ap(scale=2.5e38), 1), (_ap(scale=-1.8e38), 1), (_ap(N=0), 1), (_ap(D=96, q=768, k=192, v=192), 2),
       (_ap(D=32), 2), (_ap(N=65536), 2), (_ap(HQ=65538), 2), (_ap(T=(1 << 31) - 1), 2)]


@pytest.mark.parametrize("p,expect", BAD)
def test_problems(p, expect):
    assert _append(p) == expect and _prefill(p) == expect and _decode(p) == expect
    assert gdr.lib().gdr_attn_workspace_size(_ref(p), 1, 0) == 0


def test_no_problem():
    L = gdr.lib()
    assert L.gdr_rope_append_paged(None, _ref(_rot()), PTR, PTR, PTR, PTR, PTR, None, PTR, PTR, None) == 1
    assert _prefill(None) == 1 and _decode(None) == 1 and L.gdr_attn_workspace_size(None, 1, 0) == 0


def test_rows_and_their_alignment():
    for kw in (dict(q=511), dict(q=504), dict(q=(1 << 22) + 8)):
        assert _append(_ap(**kw)) == 1 and _prefill(_ap(**kw)) == 1 and _decode(_ap(**kw)) == 1, kw
    for kw in (dict(k=127), dict(k=132), dict(v=120), dict(v=(1 << 22) + 8)):
        assert _append(_ap(**kw)) == 1 and _prefill(_ap(**kw)) == 1, kw
    assert _append(_ap(v=0), pages=None, v=None, cu=None) == 1            # N = 2, T = 100 without cu_seqlens
    for n in ("q", "k", "v", "o"):
        assert _prefill(_ap(), **{n: ODD}) == 1 and _prefill(_ap(), **{n: None}) == 1, n
    for n in ("q", "o"):
        assert _decode(_ap(T=20), **{n: ODD}) == 1 and _decode(_ap(T=20), **{n: None}) == 1, n
    for n in ("q", "k", "v", "qo", "ko"):
        assert _append(**{n: ctypes.c_void_p(FAR[n].value + 8)}) == 1, n
    assert _prefill(_ap(), cu=None) == 1


def test_append_tensors():
    assert _append(q=None) == 1 and _append(qo=None) == 1                  # both or neither
    assert _append(k=None) == 1 and _append(v=None) == 1
    assert _append(pages=None, ko=None) == 1                               # nothing would be done with k
    for r in (_rot(R=63), _rot(R=66), _rot(R=-2), _rot(axes=0), _rot(axes=9), _rot(inter=2), _rot(freq=None), _rot(axes=3)):
        assert _append(r=r) == 1


def test_append_outputs_over_inputs():
    q, k, v = (FAR[n].value for n in "qkv")
    dense = _ap(T=100, q=512, k=128, v=128)
    fused = _ap(T=100, q=768, k=768, v=768)
    at = lambda x: ctypes.c_void_p(x)  # noqa: E731
    assert _append(fused, qo=at(q)) == 1 and _append(fused, ko=at(k)) == 1          # in place: dense tensors only
    for off in (-102400 + 16, -16, 16, 102400 - 16):                                # 100 x 512 bf16
        assert _append(dense, qo=at(q + off)) == 1, off
    assert _append(dense, qo=at(k)) == 1 and _append(dense, qo=at(v + 512)) == 1
    assert _append(dense, ko=at(q)) == 1 and _append(dense, ko=at(k + 16)) == 1 and _append(dense, ko=at(v)) == 1
    assert _append(dense, ko=at(FAR["qo"].value + 1024)) == 1


def test_append_over_the_cache():
    at = lambda x: ctypes.c_void_p(x)  # noqa: E731
    k, n = 6 << 32, 8 * 2 * 16 * 64 * 2
    far = lambda **kw: _append(pages=_kp(**dict(dict(k=at(k), v=at(k + n)), **kw)))  # noqa: E731
    assert far(v=at(k)) == 1 and far(v=at(k + n - 16)) == 1
    for name in ("q", "k", "v", "qo", "ko"):
        for c in ("k", "v"):
            assert far(**{c: FAR[name]}) == 1 and far(**{c: at(FAR[name].value - n + 16)}) == 1, (name, c)


def test_outputs_of_attention_over_inputs():
    at = lambda x: ctypes.c_void_p(x << 32)  # noqa: E731
    L, p = gdr.lib(), _ap(T=20)

    def prefill(**kw):
        a = dict(dict(q=at(1), k=at(2), v=at(3), o=at(4), lse=at(5)), **kw)
        return L.gdr_attn_prefill_fwd(_ref(p), a["q"], a["k"], a["v"], PTR, a["o"], a["lse"], None)

    def decode(**kw):
        a = dict(dict(q=at(1), k=at(2), v=at(3), o=at(4), lse=at(5), ws=at(6)), **kw)
        return L.gdr_attn_decode_paged(_ref(p), 12, a["q"], PTR, PTR, _ref(_kp(k=a["k"], v=a["v"])), 0, None, None, a["o"], a["lse"],
                                       a["ws"], 1 << 30, None)

    for call, outs in ((prefill, ("o", "lse")), (decode, ("o", "lse", "ws"))):
        for i, name in enumerate(outs):
            for other in ("q", "k", "v") + outs[:i]:
                assert call(**{name: at(9), other: at(9)}) == 1, (name, other)


def test_largest_launches():
    assert _prefill(_ap(T=1 << 30, HQ=8, q=512)) == 2 and _prefill(_ap(T=1 << 24, HQ=128, q=8192), o=ctypes.c_void_p(1 << 45)) == 2


@pytest.mark.parametrize("call", [lambda c: _append(pages=c), lambda c: _decode(_ap(T=20), pages=c)])
def test_pages(call):
    for c in (_kp(k=None), _kp(v=None), _kp(k=ODD), _kp(v=ODD), _kp(n=0), _kp(n=-1), _kp(most=-1), _kp(table=None), _kp(size=0),
              _kp(size=8), _kp(size=48), _kp(size=1 << 17)):
        assert call(c) == 1
    assert call(_kp(size=65536, most=32768)) == 2                           # 2^31 tokens in a row


def test_decode_arguments():
    p = _ap(T=20)
    for kw in (dict(ql=0), dict(ql=13), dict(ctx=None), dict(pages=None), dict(G=-1), dict(G=1), dict(G=1, off=PTR),
               dict(G=1, pre=PTR), dict(ws=None), dict(ws=ctypes.c_void_p(0x10010)), dict(ql=9), dict(cu=None)):
        assert _decode(p, **kw) == 1, kw
    need = gdr.lib().gdr_attn_workspace_size(_ref(p), 12, 0)
    assert need > 0 and _decode(p, nb=need - 1) == 1
    assert _decode(p, G=65536, off=PTR, pre=PTR) == 2
    assert _decode(_ap(T=1 << 19, N=65535, HQ=4096, HK=4096, q=1 << 18)) == 2        # T * HQ
    assert _decode(_ap(T=70000, N=65000), pages=_kp(size=65536, most=32767)) == 2    # tiles in 32 bits


def test_workspace_size():
    size = lambda ql=1, g=0, **k: gdr.lib().gdr_attn_workspace_size(_ref(_ap(**k)), ql, g)  # noqa: E731
    assert size(T=0) == 0 and size(ql=0) == 0 and size(ql=13) == 0 and size(g=-1) == 0 and size(g=65536) == 0
    assert 0 < size() < size(g=1) and size(ql=4) < size(ql=12) and size(D=64) < size(D=128, q=1024, k=256, v=256)
    assert size(T=60000, N=60000, HQ=64, HK=64, D=128, q=8192, g=4) > 1 << 32


def test_empty_batches_need_no_device():
    none = dict(q=None, k=None, v=None, qo=None, ko=None)
    assert _append(_ap(T=0, N=3), cu=PTR, pages=None, **none) == 0 and _append(_ap(T=0, N=0), cu=None, ctx=None, pages=None, **none) == 0
    assert _prefill(_ap(T=0, N=0), None, None, None, None, None) == 0 and _prefill(_ap(T=0, N=4)) == 0
    assert _decode(_ap(T=0, N=0), q=None, cu=None, ctx=None, o=None, ws=None, nb=0, pages=_kp(table=None)) == 0


def test_binding_refuses_host_tensors():
    x, i = torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        gdr.gdr_rope_append_paged(x, x)
    with pytest.raises(ValueError):
        gdr.gdr_attn_prefill_fwd(x, x, x)
    with pytest.raises(ValueError):
        gdr.gdr_attn_decode_paged(x, torch.zeros(3, 2, 16, 64), torch.zeros(3, 2, 16, 64), i[:, None], i)
