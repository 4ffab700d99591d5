"""Beam search's selection and state reordering in plain numpy (fp64), candidate by candidate."""
import numpy as np


def select(logits, scores, num_out, finished=None, eos_token=-1):
    """logits [B, W, V] fp64, scores [B, W]: (scores fp64, parents, tokens), each [B, num_out].  Equal scores
    stand by the lower beam, in a beam by the higher logit, then by the lower token."""
    B, W, V = logits.shape
    out = np.empty((B, num_out)), np.empty((B, num_out), np.int32), np.empty((B, num_out), np.int32)
    for b in range(B):
        p, inside = np.full((W, V), -np.inf), np.zeros((W, V))
        for w in range(W):
            if not np.isfinite(scores[b, w]):
                continue
            if finished is not None and finished[b, w]:
                p[w, eos_token] = scores[b, w]
                continue
            x = np.where(np.isnan(logits[b, w]), -np.inf, logits[b, w])
            top = x.max()
            if not np.isfinite(top):
                continue
            p[w] = scores[b, w] + (x - (top + np.log(np.exp(x - top).sum())))
            inside[w] = x
        flat = p.ravel()
        best = np.lexsort((np.arange(W * V), -inside.ravel(), np.arange(W * V) // V, -flat))[:num_out]
        out[0][b], out[1][b], out[2][b] = flat[best], best // V, best % V
    return out


def reorder(slots, parents, num_slots):
    """Returns (new slots [B, W], [(source slot, destination slot)])."""
    new, moves = np.array(slots).copy(), []
    B, W = new.shape
    for b in range(B):
        if (np.any(slots[b] < 0) or np.any(slots[b] >= num_slots) or np.any(parents[b] < 0)
                or np.any(parents[b] >= W)):
            continue
        free = [int(slots[b, p]) for p in range(W) if p not in parents[b]]
        seen = set()
        for j, p in enumerate(int(v) for v in parents[b]):
            if p in seen:
                new[b, j] = free.pop(0)
                moves.append((int(slots[b, p]), int(new[b, j])))
            else:
                seen.add(p)
                new[b, j] = slots[b, p]
    return new, moves
