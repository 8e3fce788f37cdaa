"""What the 64-bit definition of the draw leaves out: tokens below 2^-126 of the row's
largest probability, and negative noise, -0 among it."""
import numpy as np
import pytest

from oracle import verify_oracle as VO

INF = float("inf")


def draw(logits, noise):
    _, t, l = VO.verify(np.array([[logits]], np.float64), None, np.zeros((1, 0)), np.zeros((1, 0)),
                        np.array([noise], np.float64))
    return int(t[0, 0]), l[0, 0]


@pytest.mark.parametrize("noise,token", [((INF, 1.0), -1), ((1.0, 0.0), 0), ((-1.0, 0.0), -1), ((0.0, 0.0), 0)])
def test_tokens_below_the_range_are_not_drawn(noise, token):
    got = draw((0.0, -200.0), noise)
    assert got[0] == token and got[1] == (0.0 if token == 0 else -INF)


def test_tokens_inside_the_range_are():
    assert draw((0.0, -87.0), (INF, 1.0))[0] == 1  # 2^-125.5


def test_acceptance_has_no_such_bound():
    z, y = np.array([[[0.0, -200.0], [0.0, 0.0]]]), np.array([[[0.0, -201.0]]])
    a, t, _ = VO.verify(z, y, np.array([[1]]), np.array([[0.5]]), np.ones((1, 2)))
    assert a[0] == 1 and t[0].tolist() == [1, 0]


@pytest.mark.parametrize("noise", [(-0.0, -0.0), (-0.0, float("nan"))])
def test_negative_zero_is_negative(noise):
    assert draw((0.0, 1.0), noise)[0] == -1
    assert draw((0.0, 1.0, 0.5), noise + (3.0,))[0] == 2
