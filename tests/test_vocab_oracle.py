"""The vocabulary operators' 64-bit definitions: worked values, and every
gradient formula against central differences of its forward definition."""
import numpy as np
import pytest

from oracle import vocab_oracle as V


def test_logprobs_worked_row():
    # softmax of (log 1, log 2, log 5) is (1, 2, 5) / 8
    x = np.log([[1.0, 2.0, 5.0, 0.0][:3]])
    o = V.token_logprobs(x, [1], 1.0, k=2)
    assert o["logprob"][0] == pytest.approx(np.log(2 / 8))
    assert o["lse"][0] == pytest.approx(np.log(8))
    p = np.array([1, 2, 5]) / 8
    assert o["entropy"][0] == pytest.approx(-(p * np.log(p)).sum())
    assert list(o["top_ids"][0]) == [2, 1]
    # at inverse temperature 2 the weights are squared
    assert V.token_logprobs(x, [1], 2.0)["logprob"][0] == pytest.approx(np.log(4 / 30))


def test_logprobs_rows_at_the_edge():
    n = -np.inf
    x = np.array([[n, n, n], [n, 3.0, n], [1.0, 1.0, 1.0]])
    o = V.token_logprobs(x, [0, 0, -1], 1.0, k=2)
    assert list(o["lse"]) == pytest.approx([n, 3.0, 1 + np.log(3)])
    assert list(o["logprob"]) == [n, n, 0.0]
    assert list(o["entropy"]) == pytest.approx([0.0, 0.0, np.log(3)])
    assert o["top_ids"].tolist() == [[0, 1], [1, 0], [0, 1]]


def test_distill_worked_row():
    # student (1, 2, 5) / 8, teacher (1, 3) / 4 on tokens 2 and 0
    x, t = np.log([[1.0, 2.0, 5.0]]), np.log([[1.0, 3.0]])
    loss, dx, _, _ = V.distill(x, t, [[2, 0]], 1.0)
    assert loss[0] == pytest.approx(0.25 * np.log(0.25 / (5 / 8)) + 0.75 * np.log(0.75 / (1 / 8)))
    assert dx[0] == pytest.approx([1 / 8 - 0.75, 2 / 8, 5 / 8 - 0.25])


def test_distill_matching_student_has_no_loss():
    rng = np.random.default_rng(0)
    t = rng.normal(size=(3, 5))
    x = np.full((3, 9), -np.inf)
    ids = np.array([rng.permutation(9)[:5] for _ in range(3)])
    np.put_along_axis(x, ids, t, 1)
    loss, dx, _, _ = V.distill(x, t, ids, 0.7)
    assert np.abs(loss).max() < 1e-12 and np.abs(dx).max() < 1e-12


def differences(f, x, eps=1e-5):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        if not np.isfinite(x[i]):
            continue
        a, b = x.copy(), x.copy()
        a[i] += eps
        b[i] -= eps
        g[i] = (f(a) - f(b)) / (2 * eps)
    return g


@pytest.mark.parametrize("scale", [1.0, 0.5, 1.7])
def test_logprobs_gradient_against_differences(scale):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(4, 11)) * 2
    x[1, 3:7] = -np.inf
    t = [5, 2, -1, 10]
    g, h = rng.normal(size=4), rng.normal(size=4)

    def f(y):
        o = V.token_logprobs(y, t, scale)
        return (o["logprob"] * g * [1, 1, 0, 1]).sum() + (o["entropy"] * h).sum()
    assert V.token_logprobs_backward(x, t, scale, g, h) == pytest.approx(differences(f, x), abs=1e-8)


@pytest.mark.parametrize("scale", [1.0, 0.5, 1.7])
def test_distill_gradient_against_differences(scale):
    rng = np.random.default_rng(2)
    x, t = rng.normal(size=(5, 12)) * 2, rng.normal(size=(5, 4)) * 2
    ids = np.array([[3, 0, 7, 1], [3, 3, 2, -1], [11, 4, 12, 0], [-1] * 4, [5, 6, 5, 5]])
    w = rng.normal(size=5)
    _, dx, _, _ = V.distill(x, t, ids, scale, w)
    got = differences(lambda y: (V.distill(y, t, ids, scale)[0] * w).sum(), x)
    assert dx == pytest.approx(got, abs=1e-8)
    assert not dx[3].any()


def test_embedding_gradient_against_differences():
    rng = np.random.default_rng(3)
    table, ids, c = rng.normal(size=(6, 3)), [2, 0, 2, -1, 5, 6, 2], rng.normal(size=(7, 3))
    g, _, count = V.embedding_backward(c, ids, 1.3, 6)
    got = differences(lambda y: (V.embedding_forward(y, ids, 1.3) * c).sum(), table)
    assert g == pytest.approx(got, abs=1e-8) and list(count) == [1, 0, 3, 0, 0, 1]
