"""Inputs and tolerances of the full-attention tests.

Tolerance of an output, from the oracle's sums (u = 2^-24):

  o:   weight * (h + 2 d) + half * |o|        lse:  d + 2 u |lse|

with weight = sum_j p_j |v_j|, half the half step of the output's type, h the half step of the type in which the
weights p enter the product with v (2^-8 in bf16; 0 in fp32, where d holds it), and d what the fp32 arithmetic can
leave in the log of a weight or of the sum:

  d = u * (2 (D + 8) size + 8 keys / 16 + 2 keys + 64)

  (D + 8) size   a score is a sum of D products (D u of the sum of their absolute values; bf16 products are exact),
                 and the scale, its conversion to base 2, the maximum's subtraction and the exponential's argument
                 round values of at most ``size``; once for the score and once for the maximum it is measured from
  8 keys / 16    every tile or part (16 keys at least) rescales what is there: an exponential (2 u), a product and a
                 sum, in the output and in the sum of the weights
  2 keys         the sums over the keys, in the output and in the sum of the weights
  64             exponentials, logarithm, reciprocal, join
The weights enter o twice, in the numerator and the denominator: 2 d."""
import numpy as np
import torch

from _dev import to_dev
from gated_delta_rule_63_amd import inputs

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def cast(x, io):
    x = np.asarray(x, np.float32)
    return inputs.f32_to_bf16_bits(x) if io == "bf16" else x


def wide(x):
    return inputs.widen(x) if x.dtype == np.uint16 else x.astype(np.float64)


def normal(r, shape, io, scale=1.0):
    """(device tensor, its values in fp64)"""
    x = cast(r.normal(size=shape) * scale, io)
    return to_dev(x), wide(x)


def check(got, want, allowed, what):
    got = np.asarray(got, np.float64)
    assert got.shape == want.shape, what
    with np.errstate(invalid="ignore"):
        same = (got == want) | (np.isnan(got) & np.isnan(want))
        bad = ~(same | (np.abs(got - want) <= allowed))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {tuple(np.argwhere(bad)[0])}: " \
                          f"{got[bad][0]!r} for {want[bad][0]!r}, allowed {np.broadcast_to(allowed, bad.shape)[bad][0]!r}"


def check_attention(o, lse, ref, io, rows, what=""):
    """o [T, H, D], lse [T, H] or None in fp64, compared on the token rows ``rows``"""
    D = ref["o"].shape[2]
    keys = ref["keys"][rows][:, None]
    d = U * (2 * (D + 8) * ref["size"][rows] + keys / 2 + 2 * keys + 64)
    h = HALF[io] if io == "bf16" else 0.0
    check(o[rows], ref["o"][rows], ref["weight"][rows] * (h + 2 * d)[..., None] + HALF[io] * np.abs(ref["o"][rows]) + 1e-37, what + " o")
    if lse is not None:
        with np.errstate(invalid="ignore"):
            allowed = np.where(np.isfinite(ref["lse"][rows]), d + 2 * U * np.abs(ref["lse"][rows]), 0.0)
        check(lse[rows], ref["lse"][rows], allowed, what + " lse")


def pages_for(r, need, page, spare=3, width=None):
    """Distinct pages in random order for each sequence's ``need`` tokens (as many as ``width`` pages hold):
    (table [N, most], pages)"""
    count = [min(-(-int(n) // page), width or 1 << 30) for n in need]
    order = r.permutation(sum(count) + spare)
    table = np.full((len(need), width or max([1] + count)), -1, np.int32)
    at = 0
    for n, c in enumerate(count):
        table[n, :c] = order[at: at + c]
        at += c
    return table, len(order)
