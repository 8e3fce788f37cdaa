"""Close decisions about tokens hundreds of powers of two below their row's largest, in the
target, the draft, or both: where the weights of 31 bits end."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_verify import Case, z  # noqa: E402, F401

pytestmark = pytest.mark.gpu
LN2 = float(np.log(2.0))
DEPTHS = torch.arange(900.0, 1064.0)  # powers of two, one sequence each


@pytest.mark.parametrize("apart", [0.0, 0.4, -0.4, 30.0, -30.0])
def test_acceptance_far_below(z, apart):  # noqa: F811
    """p and q of the drafted token 2^-900 to 2^-1063 of their rows' largest, `apart` from
    each other (in powers of two); u = 0.9."""
    n = DEPTHS.numel()
    c = Case(n, 1, 300, "f32", "f32", seed=60, spread=0.0, likeness=0.0)
    c.ids[:, 0], c.u[:] = 17, 0.9
    c.x[:, 0, 17] = -LN2 * DEPTHS
    c.y[:, 0, 17] = -LN2 * (DEPTHS - apart)
    got = c.run(z)
    # q = 2^apart p
    assert (got[0] == (1 if 0.9 * 2.0 ** apart < 1 else 0)).all()


@pytest.mark.parametrize("k", [1, 3])
def test_residuals_beside_a_far_draft(z, k):  # noqa: F811
    """Two tokens in a close race, one of which the draft gives 2^-900 to 2^-1063 of its
    largest probability, and hardly any of the other."""
    n, V = DEPTHS.numel(), 90
    c = Case(n, k, V, "f32", "f32", seed=61, spread=0.0, likeness=0.0)
    c.ids[:], c.u[:] = 5, 0.99
    c.x[:, :, 5] = -30.0
    c.y[:, :, 5] = 0.0
    c.y[:, :, :5], c.y[:, :, 6:] = -800.0, -800.0
    c.y[:, :, 40] = -LN2 * DEPTHS[:, None]
    c.noise[:] = 50.0
    c.noise[:, 30] = 1.0
    c.noise[:, 40] = float(np.nextafter(np.float32(1.0), np.float32(0)))
    got = c.run(z)
    assert (got[0] == 0).all() and (got[1][:, 0] == 40).all()
