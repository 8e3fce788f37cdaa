"""Races whose noise is zero, subnormal or huge."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_verify import Case, z  # noqa: E402, F401

pytestmark = pytest.mark.gpu
INF = float("inf")
DRAFTS = [(0, None), (1, "f32"), (1, None)]


def refused(n, k, V, draft, seed):
    """Flat rows with a refused token (the last one), whose mass is the draft's."""
    c = Case(n, k, V, "f32", draft, seed=seed)
    c.x[:] = 0.0
    if k:
        c.ids[:] = V - 1
        c.u[:] = 0.9999
        c.x[:, 0, V - 1] = -20.0
        if draft:
            c.y[:] = 0.0
            c.y[:, :, V - 1] = 20.0
    c.noise[:] = 1.0
    return c


@pytest.mark.parametrize("k,draft", DRAFTS)
@pytest.mark.parametrize("small", [0.0, 1e-44, 1e-40, 1.1e-38])
def test_the_smallest_noise_wins_behind_a_huge_score(z, small, k, draft):  # noqa: F811
    """A likely token's score of 2^126 comes first; a less likely token with noise below
    the normal numbers has a larger one."""
    for n, V in ((3, 20011), (320, 5003)):
        c = refused(n, k, V, draft, 40)
        c.x[:, :, 3] = 10.0
        c.noise[:, 3] = 2.0 ** -126
        c.x[:, :, V - 900] = 7.0
        c.noise[:, V - 900] = small
        got = c.run(z)
        if small < 1e-39:
            assert (got[1][:, 0] == V - 900).all()


@pytest.mark.parametrize("k,draft", DRAFTS)
def test_noise_above_the_reciprocals_range(z, k, draft):  # noqa: F811
    """1 / e is below the normal numbers: a likely token's score is 2^-127.6, and an
    unlikely one's 2^-130."""
    for n in (3, 320):
        c = refused(n, k, 3001, draft, 41)
        c.noise[:] = INF
        c.noise[:, 17] = 1.5 * 2.0 ** 127
        c.x[:, :, 2000] = -41.5
        c.noise[:, 2000] = 2.0 ** 70
        got = c.run(z)
        assert (got[1][:, 0] == 17).all()


@pytest.mark.parametrize("k,draft", DRAFTS)
def test_scores_that_binary32_holds_to_few_digits(z, k, draft):  # noqa: F811
    """Scores around 2^-140, a hundredth apart."""
    n, V = 200, 301
    c = refused(n, k, V, draft, 42)
    g = torch.Generator().manual_seed(43)
    c.x[:, :, :V - 1] = 0.25 * torch.rand(n, 1, V - 1, generator=g)
    c.x[:, :, V - 2] = 41.0
    c.noise[:] = 2.0 ** 81 * (1 + 0.01 * torch.rand(n, V, generator=g))
    c.noise[:, V - 2] = INF
    c.run(z)


@pytest.mark.parametrize("small", [0.0, 1e-42])
def test_negative_zero_beside_a_negative_residual(z, small):  # noqa: F811
    """The draft's token is above the target's, its noise -0: minus by minus is no plus."""
    for n, V in ((4, 40), (4, 3001), (320, 500)):
        c = Case(n, 1, V, "f32", "f32", seed=46)
        c.x[:], c.y[:] = 0.0, 0.0
        c.y[:, :, 2] = 3.0
        c.ids[:], c.u[:] = 2, 0.9
        c.noise[:] = INF
        c.noise[:, 2] = -0.0
        c.noise[:, 5] = small
        got = c.run(z)
        assert (got[0] == 0).all() and (got[1][:, 0] == 5).all()
