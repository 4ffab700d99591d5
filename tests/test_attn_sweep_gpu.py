"""Seeded random configurations of the full-attention entry points against the fp64 oracle (tolerances: _attn.py)."""
import numpy as np
import pytest
import torch

from test_attn_gpu import _append_case, _decode_check, _decode_inputs, _prefill_case

pytestmark = pytest.mark.gpu


def _heads(r, most=12):
    per, HK = int(r.choice([1, 1, 2, 3, 4, 5, 8, most])), int(r.choice([1, 2, 3, 4, 8]))
    return per * HK, HK


def _lens(r, n, long):
    kinds = r.integers(0, 4, n)
    pick = [lambda: 0, lambda: int(r.integers(1, 8)), lambda: int(r.integers(1, 150)), lambda: int(r.integers(1, long))]
    return [pick[k]() for k in kinds]


def append(seed):
    r = np.random.default_rng([seed, 1])
    io, D = r.choice(["bf16", "f32"]), int(r.choice([64, 128]))
    HQ, HK = _heads(r)
    n = int(r.integers(1, 20))
    one = r.random() < 0.25
    lens = [1] * n if one else _lens(r, n, 400)
    ctx = np.where(r.random(n) < 0.15, -1, r.integers(0, 200, n))
    rotary = int(r.choice([D, D // 2, 2 * int(r.integers(0, D // 2 + 1))]))
    axes = int(r.choice([1, 1, 2, 3, 8])) if rotary else 1
    _append_case([seed, 2], io, D, HQ, HK, lens, ctx, rotary, bool(r.integers(0, 2)), axes, int(r.choice([16, 32, 64, 512])),
                 tail=0 if one else int(r.integers(0, 4)), fused=bool(r.integers(0, 2)), one_token=one)


def prefill(seed):
    r = np.random.default_rng([seed, 3])
    io, D = r.choice(["bf16", "f32"]), int(r.choice([64, 128]))
    HQ, HK = _heads(r)
    many = r.random() < 0.25
    lens = _lens(r, int(r.integers(60, 100)), 30) if many else _lens(r, int(r.integers(1, 7)), int(r.choice([100, 500, 900])))
    scale = None if r.random() < 0.7 else float(r.normal() * 0.3)
    _prefill_case([seed, 4], io, D, HQ, HK, lens, tail=int(r.integers(0, 3)), scale=scale, fused=bool(r.integers(0, 2)))


def decode(seed):
    r = np.random.default_rng([seed, 5])
    io, D = r.choice(["bf16", "f32"]), int(r.choice([64, 128]))
    HQ, HK = _heads(r, 20)
    n = int(r.choice([1, 2, 5, 17, 40, 150]))
    ctx = np.where(r.random(n) < 0.1, -1, r.integers(0, int(r.choice([10, 100, 400, 1500 if n < 20 else 200])), n))
    page, most = int(r.choice([16, 32, 64, 256])), int(r.choice([1, 3, 12]))
    lens = r.integers(0 if r.random() < 0.3 else 1, most + 1, n).tolist()
    groups, width = None, None
    if r.random() < 0.6:
        groups, at = [], 0
        while at < n and r.random() < 0.9:
            m = int(r.integers(0, min(n - at, int(r.choice([2, 8, 200]))) + 1))
            live = [int(c) for c in ctx[at:at + m] if c >= 0]
            if live and r.random() < 0.7:       # longer ones, for there to be something to share
                more = int(r.integers(0, 700))
                ctx[at:at + m] = np.where(ctx[at:at + m] >= 0, ctx[at:at + m] + more, -1)
                live = [c + more for c in live]
            groups.append((m, int(r.integers(0, min(live) + 1)) if live else 50))
            at += m
            if m == 0 and r.random() < 0.5:
                break
    elif r.random() < 0.3:
        width = int(r.integers(1, 8))
    d = _decode_inputs([seed, 6], io, D, HQ, HK, lens, ctx, page, groups=groups, width=width)
    if groups is None and r.random() < 0.3:      # pages that are none
        t = d["table"]
        t[r.random(t.shape) < 0.1] = r.choice([-1, -100, 1 << 29])
    if r.random() < 0.5:                         # what nobody sees is not finite
        seen = np.zeros((d["k"].shape[0], page), bool)
        for n in range(len(lens)):
            for j in range(min(int(ctx[n]) + lens[n], d["table"].shape[1] * page) if ctx[n] >= 0 and lens[n] else 0):
                p = d["table"][n, j // page]
                if 0 <= p < len(seen):
                    seen[p, j % page] = True
        nobody = torch.from_numpy(~seen).cuda()[:, None, :, None]
        for x in ("k", "v"):
            d[x].masked_fill_(nobody, float(r.choice([np.nan, np.inf, -np.inf])))
    _decode_check(d, scale=None if r.random() < 0.7 else float(r.normal() * 0.3))


@pytest.mark.parametrize("seed", range(40))
@pytest.mark.parametrize("entry", [append, prefill, decode])
def test_random_configurations(entry, seed):
    entry(seed)
