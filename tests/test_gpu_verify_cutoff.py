"""Tokens too unlikely to be drawn: below 2^-126 of the row's largest probability."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_verify import Case, z  # noqa: E402, F401

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("k", [0, 1])
@pytest.mark.parametrize("V", [2, 3, 2011])
@pytest.mark.parametrize("noise", [(INF, 1.0), (1.0, 0.0), (-1.0, 0.0), (0.0, 0.0)])
def test_tokens_below_the_range_are_not_drawn(z, noise, V, k):  # noqa: F811
    """Two tokens, 200 apart (2^-288), whatever the noise: the unlikely one is not drawn,
    and where the likely one is excluded nothing is."""
    for n in (4, 320):
        c = Case(n, k, V, "f32", None, seed=44)
        c.x[:] = -INF
        c.x[:, :, 0], c.x[:, :, V - 1] = 0.0, -200.0
        c.noise[:, 0], c.noise[:, V - 1] = noise
        if k:
            c.ids[:], c.u[:] = 0, 0.5  # accepted: the draw is behind it
        got = c.run(z)
        assert (got[0] == k).all()
        assert (got[1][:, k] == (0 if noise[0] >= 0 and noise[0] < INF else -1)).all()


def test_a_residual_below_the_range_is_none(z):  # noqa: F811
    """The target is above the draft at a token below the range alone: the draw is from the
    target."""
    c = Case(8, 1, 600, "f32", "f32", seed=45)
    c.x[:], c.y[:] = -INF, -INF
    c.x[:, :, 5], c.x[:, 0, 77] = 0.0, -200.0
    c.y[:, :, 5], c.y[:, 0, 77] = 0.0, -300.0
    c.ids[:], c.u[:] = 5, float("nan")  # refused
    c.noise[:, 77] = 1e-30
    got = c.run(z)
    assert (got[0] == 0).all() and (got[1][:, 0] == 5).all()
