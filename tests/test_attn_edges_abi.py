"""Host-side refusals of the full-attention entry points at the ends of their ranges (CPU: validation fails before any
launch)."""
import ctypes

from test_attn_abi import PTR, _append, _ap, _decode, _kp


def test_the_longest_table_rows():
    """Attention counts keys in 32 bits, a tile or two behind a row's last one; the append counts in 64."""
    p = _ap(T=2)
    for size, most in ((16, (1 << 27) - 1), (16, (1 << 27) - 7), (32, (1 << 26) - 1), (64, (1 << 25) - 1)):
        assert _decode(p, ws=None, pages=_kp(size=size, most=most)) == 2, (size, most)
    for size, most in ((16, (1 << 27) - 8), (32, (1 << 26) - 4), (64, (1 << 25) - 2), (128, (1 << 24) - 1), (65536, 32767)):
        assert _decode(p, ws=None, pages=_kp(size=size, most=most)) == 1, (size, most)       # as far as the workspace
    misplaced = ctypes.c_void_p(0x10000 + 8)
    assert _append(k=misplaced, pages=_kp(size=16, most=(1 << 27) - 1)) == 1                 # as far as the rows
    assert _decode(_ap(T=0, N=0), pages=_kp(size=16, most=(1 << 27) - 1)) == 2
