"""The oracles of the gated linear recurrence and of beam search, pinned by closed forms, finite differences
and brute force (CPU)."""
import itertools

import numpy as np
import pytest

from oracle import beam, linear


def test_constant_gate_is_a_geometric_sum():
    g, x = np.log(0.75), 2.0
    f = linear.scan(np.full((20, 1), x), np.full((20, 1), g), linear.LOG_DECAY, [0, 20])
    t = np.arange(1, 21)
    assert np.allclose(f["y"][:, 0], x * (1 - 0.75 ** t) / 0.25, rtol=1e-14)


def test_sigmoid_gate_keeps_a_constant_input():
    z = np.random.default_rng(0).normal(size=(30, 4)) * 4
    f = linear.scan(np.full((30, 4), 1.5), z, linear.SIGMOID, [0, 30], np.full((1, 4), 1.5))
    assert np.allclose(f["y"], 1.5, rtol=1e-14)


def test_sequences_are_separate_and_empty_ones_pass_their_state():
    r = np.random.default_rng(1)
    x, g, h0 = r.normal(size=(9, 3)), -r.uniform(0, 1, (9, 3)), r.normal(size=(4, 3))
    f = linear.scan(x, g, linear.LOG_DECAY, [0, 4, 4, 9, 9], h0)
    for n, (s, e) in enumerate([(0, 4), (4, 4), (4, 9), (9, 9)]):
        one = linear.scan(x[s:e], g[s:e], linear.LOG_DECAY, [0, e - s], h0[n:n + 1])
        assert np.array_equal(f["y"][s:e], one["y"]) and np.array_equal(f["final"][n], one["final"][0])
    assert np.array_equal(f["final"][1], h0[1]) and np.array_equal(f["final"][3], h0[3])


@pytest.mark.parametrize("kind", [linear.LOG_DECAY, linear.SIGMOID])
def test_gradients_against_differences(kind):
    r = np.random.default_rng(2)
    cu = [0, 3, 3, 8]
    x, h0 = r.normal(size=(8, 2)), r.normal(size=(3, 2))
    gate = -r.uniform(0.05, 1, (8, 2)) if kind == linear.LOG_DECAY else r.normal(size=(8, 2))
    dy, dF = r.normal(size=(8, 2)), r.normal(size=(3, 2))

    def loss(x, gate, h0):
        f = linear.scan(x, gate, kind, cu, h0)
        return (f["y"] * dy).sum() + (f["final"] * dF).sum()

    got = linear.grads(x, gate, kind, cu, dy, h0, dF)
    for name, v in (("dx", x), ("dgate", gate), ("dh0", h0)):
        want = np.empty_like(v)
        for i in np.ndindex(v.shape):
            d = np.zeros_like(v)
            d[i] = 1e-5
            args = {"dx": x, "dgate": gate, "dh0": h0}
            hi, lo = dict(args, **{name: v + d}), dict(args, **{name: v - d})
            want[i] = (loss(*hi.values()) - loss(*lo.values())) / 2e-5
        # a central difference of step 1e-5: its third derivative times 1e-10 / 6, and 1e-16 / 1e-5 of rounding
        assert np.allclose(got[name], want, rtol=1e-6, atol=1e-8), name


def test_select_by_brute_force():
    r = np.random.default_rng(3)
    lg = np.round(r.normal(size=(2, 3, 5)) * 2) / 2  # ties
    lg[1, 0, 2], lg[1, 1] = -np.inf, -np.inf
    sc = r.normal(size=(2, 3))
    fin = np.array([[0, 1, 0], [0, 0, 0]])
    s, p, t = beam.select(lg, sc, 7, fin, 4)
    for b in range(2):
        every = []
        for w, v in itertools.product(range(3), range(5)):
            if fin[b, w]:
                val = sc[b, w] if v == 4 else -np.inf
            elif np.isneginf(lg[b, w]).all():
                val = -np.inf
            else:
                val = sc[b, w] + lg[b, w, v] - np.log(np.exp(lg[b, w]).sum())
            every.append((-np.round(val, 12), w, v))
        every.sort()
        assert [(w, v) for _, w, v in every[:7]] == list(zip(p[b], t[b]))


def test_select_tells_equal_scores_apart_by_beam_logit_and_token():
    lg = np.array([[[1.0, 2.0, 3.0, 3.0], [4.0, 1.0, 2.0, 2.0], [0.0, 0.0, 0.0, 0.0]]])
    # in scores of -1e30 the logits make no difference: the lower beam first, there the higher logit
    _, p, t = beam.select(lg, np.array([[-1e30, -1e30, 0.0]]), 4)
    assert list(zip(p[0], t[0])) == [(2, 0), (2, 1), (2, 2), (2, 3)]
    _, p, t = beam.select(lg[:, :2], np.array([[-1e30, -1e30]]), 4)
    assert list(zip(p[0], t[0])) == [(0, 2), (0, 3), (0, 1), (0, 0)]
    lg[0, 0, 3] = -np.inf
    _, p, t = beam.select(lg[:, :2], np.array([[-1e30, -1e30]]), 4)
    assert list(zip(p[0], t[0])) == [(0, 2), (0, 1), (0, 0), (1, 0)]


def test_reorder_moves_every_state_once():
    r = np.random.default_rng(4)
    for _ in range(50):
        W = int(r.integers(1, 9))
        slots = r.permutation(40)[:W][None].astype(np.int32)
        parents = r.integers(0, W, (1, W)).astype(np.int32)
        new, moves = beam.reorder(slots, parents, 40)
        pool = np.arange(40)
        after = pool.copy()
        for s, d in moves:
            assert d not in slots[0, parents[0]]      # no state that is still wanted is overwritten
            after[d] = pool[s]
        assert np.array_equal(after[new[0]], pool[slots[0, parents[0]]])
        assert sorted(new[0]) == sorted(slots[0])
        assert len(moves) == W - len(set(parents[0].tolist()))
