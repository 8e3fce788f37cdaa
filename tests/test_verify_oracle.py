"""The 64-bit definition of drafted tokens' verification, pinned by rows worked by
hand and by the distribution of what it emits."""
import numpy as np

from oracle import verify_oracle as VO


def log(p):
    with np.errstate(divide="ignore"):
        return np.log(np.asarray(p, np.float64))


def one(p, q, ids, u, e, **kw):
    a, t, l = VO.verify(log(p)[None], None if q is None else log(q)[None], np.array([ids]),
                        np.array([u]), np.array([e], np.float64), **kw)
    return int(a[0]), t[0].tolist(), l[0]


def test_accepts_below_the_ratio_of_probabilities():
    p = [[0.5, 0.25, 0.25], [0.2, 0.2, 0.6]]
    q = [[0.25, 0.5, 0.25]]
    # token 1: p / q = 0.5; the next token: largest 0.2, 0.2, 0.6 over e
    a, t, l = one(p, q, [1], [0.49], [1.0, 0.1, 1.0])
    assert (a, t) == (1, [1, 1])
    np.testing.assert_allclose(l, log([0.25, 0.2]))
    # refused: residual [0.25, 0, 0]
    a, t, l = one(p, q, [1], [0.51], [1.0, 0.1, 1.0])
    assert (a, t) == (0, [0, -1])
    np.testing.assert_allclose(l, [np.log(0.5), 0.0])


def test_tokens_without_probabilities():
    p = [[0.5, 0.25, 0.25], [0.2, 0.2, 0.6]]
    assert one(p, None, [2], [0.24], [1, 1, 1])[:2] == (1, [2, 2])
    # refused: the residual is p without the token, which noise favours
    assert one(p, None, [2], [0.26], [1, 1, 1e-9])[:2] == (0, [0, -1])


def test_short_drafts_masks_and_empty_rows():
    p = [[0.5, 0.5, 0.0], [0.0, 1.0, 0.0], [1.0, 0.0, 0.0]]
    q = [[0.5, 0.0, 0.5], [0.5, 0.5, 0.0]]
    assert one(p, q, [0, -1], [0.9, 0.9], [1, 1, 1])[:2] == (1, [0, 1, -1])
    assert one(p, q, [2, 0], [0.0, 0.0], [1, 1, 1])[:2] == (0, [1, -1, -1])  # p(2) = 0
    z = log(p)
    z[1] = -np.inf
    a, t, l = VO.verify(z[None], log(q)[None], np.array([[0, 1]]), np.array([[0.1, 0.1]]), np.ones((1, 3)))
    assert a[0] == 1 and t[0].tolist() == [0, -1, -1] and l[0, 1] == -np.inf
    z[0, 1] = np.nan
    a, t, l = VO.verify(z[None], log(q)[None], np.array([[0, 1]]), np.array([[0.1, 0.1]]), np.ones((1, 3)))
    assert a[0] == 0 and t[0, 0] == -1 and np.isnan(l[0, 0])


def test_emitted_tokens_are_distributed_as_the_target():
    """First emitted token of 40000 sequences: its frequencies are p's within five
    standard deviations, with a draft and without its probabilities."""
    rng = np.random.default_rng(1)
    n, V = 40_000, 5
    p, q = np.array([0.4, 0.3, 0.15, 0.1, 0.05]), np.array([0.1, 0.2, 0.3, 0.3, 0.1])
    P = np.broadcast_to(log(p), (n, 2, V))
    ids = rng.choice(V, size=(n, 1), p=q)
    for Q in (np.broadcast_to(log(q), (n, 1, V)), None):
        d = ids if Q is not None else np.full((n, 1), 2)
        _, t, _ = VO.verify(P, Q, d, rng.random((n, 1)), rng.exponential(size=(n, V)))
        f = np.bincount(t[:, 0], minlength=V) / n
        assert np.all(np.abs(f - p) < 5 * np.sqrt(p * (1 - p) / n))
