"""The oracle of the full-attention operators, pinned by closed forms and by other ways to the same values (CPU)."""
import numpy as np
import pytest

from oracle import attn


def test_rotation_is_a_complex_product_and_depends_on_differences():
    r = np.random.default_rng(0)
    x, y, f = r.normal(size=(6, 2, 8)), r.normal(size=(6, 2, 8)), r.uniform(0.1, 1, (1, 4))
    pos = np.arange(6)[None]
    for inter in (False, True):
        a = attn.rotate(x, attn.angles(pos, f), inter)
        even, odd = (slice(0, 8, 2), slice(1, 8, 2)) if inter else (slice(0, 4), slice(4, 8))
        z = (x[..., even] + 1j * x[..., odd]) * np.exp(1j * pos[0][:, None] * f)[:, None]
        assert np.allclose(a[..., even], z.real, atol=1e-14) and np.allclose(a[..., odd], z.imag, atol=1e-14)
        moved = [(attn.rotate(x, attn.angles(pos + d, f), inter) * attn.rotate(y, attn.angles(pos + d, f), inter)).sum(-1) for d in (0, 50)]
        assert np.allclose(moved[0], (x * y).sum(-1), atol=1e-12) and np.allclose(moved[0], moved[1], atol=1e-12)
    # channels behind the rotated ones, and an axis of its own for each pair
    f2 = np.array([[0.5, 0.0], [0.0, 2.0]])
    b = attn.rotate(x, attn.angles(np.stack([np.zeros(6), np.ones(6)]), f2), False)
    assert np.array_equal(b[..., 4:], x[..., 4:]) and np.allclose(b[..., 0], x[..., 0])
    assert np.allclose(b[..., 1], x[..., 1] * np.cos(2.0) - x[..., 3] * np.sin(2.0))


def test_equal_keys_give_the_mean():
    q, k, v = np.ones((5, 2, 4)), np.zeros((5, 1, 4)), np.random.default_rng(1).normal(size=(5, 1, 4))
    r = attn.prefill(q, k, v, [0, 2, 5], 0.3)
    assert np.allclose(r["o"][1, 0], v[:2, 0].mean(0)) and np.allclose(r["o"][4, 1], v[2:, 0].mean(0))
    assert np.allclose(r["lse"][4], np.log(3)) and np.array_equal(r["keys"], [1, 2, 1, 2, 3])


def test_against_a_matrix_softmax():
    torch = pytest.importorskip("torch")
    r = np.random.default_rng(2)
    q, k, v = r.normal(size=(7, 4, 8)), r.normal(size=(7, 2, 8)), r.normal(size=(7, 2, 8))
    got = attn.prefill(q, k, v, [0, 7], -0.7)
    for h in range(4):
        x = torch.tensor(-0.7 * q[:, h] @ k[:, h // 2].T).masked_fill(torch.ones(7, 7).triu(1).bool(), -np.inf)
        assert np.allclose(got["o"][:, h], (x.softmax(1) @ torch.tensor(v[:, h // 2])).numpy(), atol=1e-14)
        assert np.allclose(got["lse"][:, h], x.logsumexp(1).numpy(), atol=1e-14)


def test_decode_is_the_end_of_a_prompt():
    r = np.random.default_rng(3)
    q, k, v = r.normal(size=(40, 4, 8)), r.normal(size=(40, 2, 8)), r.normal(size=(40, 2, 8))
    whole = attn.prefill(q, k, v, [0, 40], 0.4)
    pages = r.permutation(5)[None]
    kp, vp = np.full((5, 2, 16, 8), np.nan), np.full((5, 2, 16, 8), np.nan)
    for t in range(40):
        p, row = attn.place(pages, 5, 16, 0, t)
        kp[p, :, row], vp[p, :, row] = k[t], v[t]
    d = attn.decode(q[33:], [0, 7], [33], kp, vp, pages, 0.4)
    assert np.allclose(d["o"], whole["o"][33:], atol=1e-14) and np.allclose(d["lse"], whole["lse"][33:], atol=1e-14)


def test_what_is_not_there_is_not_seen():
    table = np.array([[0, -1, 7]])
    assert attn.place(table, 4, 16, 0, 3) == (0, 3) and attn.place(table, 4, 16, 0, 16) is None
    assert attn.place(table, 4, 16, 0, 40) is None and attn.place(table, 4, 16, 0, 48) is None
    k = np.random.default_rng(4).normal(size=(4, 1, 16, 8))
    d = attn.decode(np.ones((2, 1, 8)), [0, 1, 2], [20, 3], k, k, np.array([[2, -1], [-1, -1]]), 1.0)
    one = attn.prefill(np.ones((16, 1, 8)), k[2, 0][:, None], k[2, 0][:, None], [0, 16], 1.0)
    assert np.allclose(d["o"][0], one["o"][15]) and d["keys"][0] == 16
    assert (d["o"][1] == 0).all() and np.isneginf(d["lse"][1]).all()


def test_one_key_takes_all():
    """Scores far apart: the largest one's value, in a prompt and from a cache, and its score as lse."""
    r = np.random.default_rng(5)
    v = r.normal(size=(9, 2, 4))
    k = np.zeros((9, 2, 4))
    k[:, 0, 0], k[:, 1, 1] = r.permutation(9) * 1000.0, r.permutation(9) * 1000.0
    q = np.ones((9, 4, 4))
    got = attn.prefill(q, k, v, [0, 4, 9], 1.0)
    for t in range(9):
        for h in range(4):
            seen = np.arange(0 if t < 4 else 4, t + 1)
            j = seen[np.argmax(k[seen, h // 2].sum(-1))]
            assert np.allclose(got["o"][t, h], v[j, h // 2]) and np.isclose(got["lse"][t, h], k[j, h // 2].sum())
    pages = lambda x: np.concatenate([x, np.zeros((7, 2, 4))])[None].transpose(0, 2, 1, 3)  # noqa: E731
    d = attn.decode(q[4:], [0, 5], [4], pages(k), pages(v), np.array([[0]]), 1.0)
    assert np.allclose(d["o"][4, 3], v[np.argmax(k[:, 1, 1]), 1])


@pytest.mark.parametrize("n", range(1, 40))
def test_decode_is_the_end_of_a_prompt_wherever_it_begins(n):
    r = np.random.default_rng(n)
    q, k, v = r.normal(size=(40, 2, 4)), r.normal(size=(40, 1, 4)), r.normal(size=(40, 1, 4))
    whole = attn.prefill(q, k, v, [0, 40], 0.4)
    table = r.permutation(3)[None]
    kp, vp = np.full((3, 1, 16, 4), np.nan), np.full((3, 1, 16, 4), np.nan)
    for t in range(40):
        p, row = attn.place(table, 3, 16, 0, t)
        kp[p, :, row], vp[p, :, row] = k[t], v[t]
    d = attn.decode(q[n:], [0, 40 - n], [n], kp, vp, table, 0.4)
    assert np.allclose(d["o"], whole["o"][n:], atol=1e-14) and np.allclose(d["lse"], whole["lse"][n:], atol=1e-14)
    assert np.array_equal(d["keys"], whole["keys"][n:])
