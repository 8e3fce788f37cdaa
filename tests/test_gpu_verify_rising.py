"""Rows whose logits rise, so that every batch of a thread changes what its weights are
relative to: acceptance and races that binary32 sums do not decide.

Log probabilities: a row's sum is off by 2^-22 + 2^-21 + 0.6 * 2^-22 log2(V) of itself,
2^-24 for each of a thread's batches of 16 logits and 32 more, and 1.25 * 2^-22 for each
batch and six more (exponentials of two ulp): with one warp of each of two blocks for a row
of 50257, 50 batches, 2.5e-5 in all."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import verify_oracle as VO  # noqa: E402
from tests.test_gpu_verify import Case, z  # noqa: E402, F401

pytestmark = pytest.mark.gpu
TOL = 2.5e-5
RISES = [0.02, 0.25, 2.0, 15.0, 90.0, 700.0]


def rising(n, k, V, dtype, draft, seed):
    """The target's rows rise by one of RISES over the row, the draft's by another; some
    fall."""
    c = Case(n, k, V, dtype, draft, seed=seed, spread=0.0, likeness=0.0)
    at = torch.arange(V) / (V - 1)
    g = torch.Generator().manual_seed(seed)
    for s in range(n):
        for j in range(k + 1):
            rise = RISES[(s + 2 * j) % 6] * (-1 if s % 7 == 6 else 1)
            c.x[s, j] = (at * rise + 0.01 * torch.rand(V, generator=g)).to(c.x.dtype)
            if draft and j < k:
                c.y[s, j] = (at * rise * (0.5, 1.0, 1.25)[s % 3] + 0.3 * torch.rand(V, generator=g)).to(c.y.dtype)
    p = c.y if draft else c.x[:, :k]
    c.ids = (p.float() - torch.log(torch.empty(n, k, V).exponential_(generator=g))).argmax(2)
    return c


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("draft", ["same", None])
@pytest.mark.parametrize("n,k,V", [(2, 5, 50257), (310, 1, 3001), (36, 3, 20011)])
def test_rising_rows(z, n, k, V, draft, dtype):  # noqa: F811
    rising(n, k, V, dtype, dtype if draft else None, 50).run(z, tol=TOL)


@pytest.mark.parametrize("draft", ["f32", None])
@pytest.mark.parametrize("n,V", [(40, 50257), (320, 9001)])
def test_acceptance_at_the_border(z, n, V, draft):  # noqa: F811
    """Uniform numbers next to p / q on both sides, one position behind another."""
    c = rising(n, 1, V, "f32", draft, 51)
    at, d = np.arange(n), c.ids[:, 0].numpy()
    lp = np.array([VO._row(c.x[s, 0].double().numpy())[d[s]] for s in range(n)])
    if draft:
        lp = lp - np.array([VO._row(c.y[s, 0].double().numpy())[d[s]] for s in range(n)])
    ratio = np.exp(lp)
    below = ratio.astype(np.float32)
    below = np.where(below.astype(np.float64) >= ratio, np.nextafter(below, np.float32(0)), below)
    u = np.where(at % 2 == 0, below, np.nextafter(below, np.float32(2)))
    far = (np.abs(u.astype(np.float64) / ratio - 1) > 4e-9) & (u < 1)
    assert far.sum() > n // 4
    c.u[:, 0] = torch.from_numpy(np.where(far, u, np.float32(0.5)))
    got = c.run(z, tol=TOL)
    np.testing.assert_array_equal(got[0][far], (u.astype(np.float64) < ratio)[far])


@pytest.mark.parametrize("k,draft", [(0, None), (1, "f32"), (1, None)])
@pytest.mark.parametrize("n,V", [(30, 50257), (310, 5003)])
def test_races_that_are_nearly_tied(z, n, V, k, draft):  # noqa: F811
    """One more token's score lies a step of its noise beside the winner's."""
    c = rising(n, k, V, "f32", draft, 52)
    if k:
        c.u[:] = 0.99999994
        c.x[torch.arange(n), 0, c.ids[:, 0]] = -2000.0  # refused
    for s in range(n):
        p = np.exp(VO._row(c.x[s, 0].double().numpy()))
        r = p
        if k and draft:
            r = p - np.exp(VO._row(c.y[s, 0].double().numpy()))
        elif k:
            r = np.where(np.arange(V) == int(c.ids[s, 0]), 0, p)
        e = c.noise[s].double().numpy()
        win = int(np.argmax(np.where(r > 0, r / e, 0)))
        order = np.argsort(-r, kind="stable")
        other = int(order[1] if order[0] == win else order[0])
        f = np.float32(r[other] * e[win] / r[win])
        c.noise[s, other] = float(np.nextafter(f, np.float32(0)) if s % 2 else np.nextafter(f, np.float32(1e30)))
        gap = abs(r[other] / float(c.noise[s, other]) / (r[win] / e[win]) - 1)
        if gap < 4e-9 * (1 + p[other] / r[other] + p[win] / r[win]):
            c.noise[s, other] = 100.0
    c.run(z, tol=TOL)
