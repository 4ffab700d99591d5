"""Full attention of serving in fp64 numpy, a sequence and a head at a time: rotary positions with the paged cache's
new rows, causal attention over packed prompts, a few tokens of each sequence against the cache.

Besides values, the attention functions return what a tolerance is made of: ``weight`` [T, H, D] = sum_j p_j |v_j| and
``size`` [T, H] = max_j |scale| sum_c |q_c k_c| over the visible keys, ``keys`` [T] = visible keys."""
import numpy as np


def angles(pos, freq):
    """pos [axes, T], freq [axes, R/2] -> theta [T, R/2]"""
    return np.einsum("at,ai->ti", np.asarray(pos, np.float64), np.asarray(freq, np.float64))


def rotate(x, theta, interleaved):
    """x [T, H, D], theta [T, R/2]"""
    y, half = np.array(x, np.float64), theta.shape[1]
    a, b = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
    c, s = np.cos(theta)[:, None], np.sin(theta)[:, None]
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return y


def place(table, num_pages, page, n, at):
    """(page, row) of token ``at`` of sequence n, or None"""
    i = at // page
    if i >= table.shape[1] or not 0 <= table[n, i] < num_pages:
        return None
    return int(table[n, i]), at % page


def _rows(q, k, v, seen, scale):
    """q [t, HQ, D], k, v [L, HKV, D], seen [t, L]: o, lse, weight, size"""
    t, HQ, D = q.shape
    per = HQ // k.shape[1]
    o, w, lse, size = np.zeros((t, HQ, D)), np.zeros((t, HQ, D)), np.full((t, HQ), -np.inf), np.zeros((t, HQ))
    for h in range(HQ):
        kh, vh = k[:, h // per], v[:, h // per]
        for i in range(t):
            at = np.nonzero(seen[i])[0]
            if len(at) == 0:
                continue
            x = scale * (kh[at] @ q[i, h])
            top = x.max()
            e = np.exp(x - top)
            lse[i, h] = top + np.log(e.sum())
            p = e / e.sum()
            o[i, h], w[i, h] = p @ vh[at], p @ np.abs(vh[at])
            size[i, h] = abs(scale) * (np.abs(kh[at]) @ np.abs(q[i, h])).max()
    return o, lse, w, size


def _empty(T, HQ, D):
    return {"o": np.full((T, HQ, D), np.nan), "lse": np.full((T, HQ), np.nan), "weight": np.zeros((T, HQ, D)),
            "size": np.zeros((T, HQ)), "keys": np.zeros(T, np.int64)}


def prefill(q, k, v, cu, scale):
    r = _empty(*q.shape)
    for a, b in zip(cu[:-1], cu[1:]):
        seen = np.tril(np.ones((b - a, b - a), bool))
        r["o"][a:b], r["lse"][a:b], r["weight"][a:b], r["size"][a:b] = _rows(q[a:b], k[a:b], v[a:b], seen, scale)
        r["keys"][a:b] = 1 + np.arange(b - a)
    return r


def decode(q, cu, context, k_pages, v_pages, table, scale):
    """Rows of padded sequences are NaN."""
    r = _empty(*q.shape)
    num, HK, page, D = k_pages.shape
    for n, ctx in enumerate(int(c) for c in context):
        a, b = int(cu[n]), int(cu[n + 1])
        if ctx < 0 or a == b:
            continue
        where = [place(table, num, page, n, j) for j in range(ctx + b - a)]
        held = [j for j, w in enumerate(where) if w is not None]
        k = np.stack([k_pages[where[j][0], :, where[j][1]] for j in held]) if held else np.zeros((0, HK, D))
        v = np.stack([v_pages[where[j][0], :, where[j][1]] for j in held]) if held else np.zeros((0, HK, D))
        seen = np.array(held)[None, :] <= ctx + np.arange(b - a)[:, None] if held else np.zeros((b - a, 0), bool)
        r["o"][a:b], r["lse"][a:b], r["weight"][a:b], r["size"][a:b] = _rows(q[a:b], k, v, seen, scale)
        r["keys"][a:b] = seen.sum(1)
    return r
