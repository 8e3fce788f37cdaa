"""Verification and sampling where the scaled logits are large: finite masks that
leave a row nothing, and inverse temperatures that make a draw nearly greedy.  The
product of a logit and the inverse temperature then has a rounding error of many
units; the difference to the row's largest, which is what the probabilities are
made of, has not.

The 64-bit definition holds here: a binary32 logit times a binary32 scale is
exact in binary64, and so is its difference to the row's largest where that is
small enough to matter.  Tolerances of the log probabilities as in test_gpu_verify."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import verify_oracle as VO  # noqa: E402
from tests.test_gpu_verify import Case, z  # noqa: E402, F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k,draft", [(0, None), (2, "same"), (2, None)])
@pytest.mark.parametrize("temperature", [0.6, 0.7, 0.9])
@pytest.mark.parametrize("value", [-1e9, -1e10, -1e30, 1e30])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_of_one_finite_value(z, dtype, value, temperature, k, draft):  # noqa: F811
    """Every token as likely as the next, whatever the value: a finite mask that
    covers a row draws from the whole vocabulary.  Every third sequence keeps some
    tokens, in the target or the draft."""
    for n in (6, 320):
        c = Case(n, k, 1203, dtype, dtype if draft else None, seed=30, scale=1 / temperature,
                 draft_scale=1 / temperature)
        keep = torch.rand(n, k + 1, 1203, generator=torch.Generator().manual_seed(2)) < 0.02
        keep[torch.arange(n) % 3 > 0] = False
        if value > 0:
            keep[:] = False
        c.x.masked_fill_(~keep, value)
        if draft:
            c.y[1::2].masked_fill_(torch.ones_like(c.y[1::2], dtype=torch.bool), value)
        c.run(z)


def steps_below(top, steps):
    """Binary32 numbers `steps` representable ones below `top`."""
    i = np.float32(top).view(np.int32) - np.asarray(steps, np.int32)
    return torch.from_numpy(np.atleast_1d(i.astype(np.int32)).view(np.float32).copy())


GREEDY = [(20.0, 1e6), (20.0, 1e7), (16.5, 4e5), (300.0, 1e5), (20.0, 3e8)]


def greedy(n, k, V, top, scale, draft, seed):
    """Rows whose tokens lie 0 to 12 representable numbers below `top` (0.5 to 500
    units once scaled), and far below."""
    c = Case(n, k, V, "f32", draft, seed=seed, scale=scale, draft_scale=scale)
    r = np.random.default_rng(seed)
    # the scaled width of a step decides how many of them matter
    width = float(np.spacing(np.float32(top))) * scale
    most = max(1, int(min(12, 12 / width)))
    rows = lambda m: steps_below(top, np.where(r.random((n, m, V)) < 0.3, r.integers(0, most + 1, (n, m, V)),  # noqa: E731
                                               r.integers(40, 4000, (n, m, V))))
    c.x = rows(k + 1)
    if k:
        c.y = rows(k) if draft else None
        near = c.y if draft else c.x[:, :k]
        c.ids = torch.from_numpy(r.integers(0, V, (n, k)))
        best = (near >= steps_below(top, most)).float() + torch.rand(near.shape, generator=torch.Generator().manual_seed(seed))
        c.ids = best.argmax(2)
    return c


@pytest.mark.parametrize("k,draft", [(0, None), (3, "f32"), (3, None)])
@pytest.mark.parametrize("top,scale", GREEDY)
def test_nearly_greedy_draws(z, top, scale, k, draft):  # noqa: F811
    for n, V in ((9, 700), (310, 901)):
        greedy(n, k, V, top, scale, draft, 31).run(z)


@pytest.mark.parametrize("draft", ["f32", None])
@pytest.mark.parametrize("top,scale", GREEDY)
def test_nearly_greedy_acceptance_at_the_border(z, top, scale, draft):  # noqa: F811
    """Uniform numbers next to p / q on both sides, as in test_gpu_verify."""
    n, V = 150, 1003
    c = greedy(n, 1, V, top, scale, draft, 32)
    at, d = np.arange(n), c.ids[:, 0].numpy()
    s = float(np.float32(scale))
    lp = np.stack([VO._row(c.x[i, 0].double().numpy() * s) for i in range(n)])[at, d]
    if draft:
        lp = lp - np.stack([VO._row(c.y[i, 0].double().numpy() * s) for i in range(n)])[at, d]
    ratio = np.exp(lp)
    below = ratio.astype(np.float32)
    below = np.where(below.astype(np.float64) >= ratio, np.nextafter(below, np.float32(0)), below)
    u = np.where(at % 2 == 0, below, np.nextafter(below, np.float32(2)))
    far = (np.abs(u.astype(np.float64) / ratio - 1) > 4e-9) & (u < 1)
    assert far.sum() > 40
    c.u[:, 0] = torch.from_numpy(np.where(far, u, np.float32(0.5)))
    got = c.run(z)
    np.testing.assert_array_equal(got[0][far], (u.astype(np.float64) < ratio)[far])


@pytest.mark.parametrize("k,draft", [(0, None), (1, "f32"), (1, None)])
@pytest.mark.parametrize("top,scale", GREEDY)
def test_nearly_greedy_races_that_are_nearly_tied(z, top, scale, k, draft):  # noqa: F811
    """As in test_gpu_verify: one more token's score lies a step of its noise beside the
    winner's."""
    n, V = 60, 801
    c = greedy(n, k, V, top, scale, draft, 33)
    s = float(np.float32(scale))
    if k:
        c.u[:] = 0.99999994
        c.x[torch.arange(n), 0, c.ids[:, 0]] = top * 0.5  # refused
    for i in range(n):
        p = np.exp(VO._row(c.x[i, 0].double().numpy() * s))
        r = p
        if k and draft:
            r = p - np.exp(VO._row(c.y[i, 0].double().numpy() * s))
        elif k:
            r = np.where(np.arange(V) == int(c.ids[i, 0]), 0, p)
        e = c.noise[i].double().numpy()
        win = int(np.argmax(np.where(r > 0, r / e, 0)))
        order = np.argsort(-r, kind="stable")
        other = int(order[1] if order[0] == win else order[0])
        if r[other] < 1e-30:
            continue
        f = np.float32(r[other] * e[win] / r[win])
        c.noise[i, other] = float(np.nextafter(f, np.float32(0)) if i % 2 else np.nextafter(f, np.float32(1e30)))
        gap = abs(r[other] / float(c.noise[i, other]) / (r[win] / e[win]) - 1)
        if gap < 4e-9 * (1 + p[other] / r[other] + p[win] / r[win]):
            c.noise[i, other] = 100.0
    c.run(z)


@pytest.mark.parametrize("scale", [2.0 ** -149, 1e-40, 1e-37, 1e37, 3e38])
@pytest.mark.parametrize("k,draft", [(0, None), (2, "f32"), (2, None)])
def test_scales_at_the_ends_of_binary32(z, scale, k, draft):  # noqa: F811
    """Logits in units of 1 / scale as far as binary32 goes: differences up to 4e38."""
    unit = min(1 / scale, 1.5e38)
    for n in (5, 310):
        c = Case(n, k, 901, "f32", draft, seed=34, scale=scale, draft_scale=scale)
        c.x = (c.x.double().clamp(-2, 2) * unit * 0.9).float()
        if draft:
            c.y = (c.y.double().clamp(-2, 2) * unit * 0.9).float()
        c.run(z)


@pytest.mark.parametrize("k,draft", [(0, None), (1, "f32"), (1, None)])
def test_differences_beyond_binary32(z, k, draft):  # noqa: F811
    """Tokens at the lowest numbers in front of tokens at the largest, 6e38 apart."""
    for n in (3, 40, 320):
        c = Case(n, k, 5003, "f32", draft, seed=35)
        c.x[:] = -3.3e38
        g = torch.Generator().manual_seed(36)
        late = torch.rand(n, k + 1, 5003, generator=g) < 0.1
        late[:, :, :2200] = False
        c.x[late] = 3e38
        if draft:
            c.y[:] = c.x[:, :k]
            c.y[:, :, 4000:] = -3.3e38
        if k:
            c.ids[:] = 4500
            c.x[:, 0, 4500] = -3.3e38  # refused
        c.run(z)
