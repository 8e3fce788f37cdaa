"""Norms of lists so long that a thread adds thousands of squares: its binary32
sums are taken into binary64 every 16 batches.

One-sided rounding errors do not cancel here (equal numbers): a square sum is off by
at most d * 2^-24 of itself, d the longest chain of binary32 roundings: 16 batches
of 4 (bf16) or 2 (binary32) squares per accumulator, 3 additions of the
accumulators, 5 of a warp, one of a last element."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_clip import norm, z  # noqa: E402, F401

pytestmark = pytest.mark.gpu
CHAIN = {torch.bfloat16: 16 * 4 + 9, torch.float32: 16 * 2 + 9}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("times", [1, 7, 64])
def test_equal_numbers(z, dtype, times):  # noqa: F811
    """A tensor of 2^28 + 5 equal numbers, listed up to 64 times (1.7e10 elements)."""
    value = 0.54296875  # its square has 16 bits: a sum of thousands is rounded down most of the time
    x = torch.full((2 ** 28 + 5,), value, device="cuda", dtype=dtype)
    n = x.numel()
    tn, sq, total, _ = norm(z, z.TensorList([x.data_ptr()] * times, [n] * times, z.BF16 if dtype == torch.bfloat16
                                            else z.F32), 1.0)
    one = value * value * n  # exact in 64 bits
    tol = CHAIN[dtype] * 2.0 ** -24
    assert abs(sq - one * times) <= tol * one * times
    assert abs(total - (one * times) ** 0.5) <= (tol / 2 + 2.0 ** -24) * total
    assert all(abs(float(t) - one ** 0.5) <= (tol / 2 + 2.0 ** -24) * one ** 0.5 for t in tn)


@pytest.mark.parametrize("where", [0, 12345, 2 ** 27 + 1, 2 ** 28 - 1])
@pytest.mark.parametrize("bad", [1e25, 3e38, float("inf"), float("nan")])
def test_one_number_beyond_the_range_of_squares(z, bad, where):  # noqa: F811
    """In a sum that has been taken to binary64 before and after it."""
    x = torch.full((2 ** 28,), 2.0 ** -10, device="cuda")
    x[where] = bad
    times = 12
    _, sq, total, _ = norm(z, z.TensorList([x.data_ptr()] * times, [x.numel()] * times, z.F32), 1.0, tensor_norms=False)
    v = float(x[where])
    want = times * (v * v + (2.0 ** 28 - 1) * 2.0 ** -20)
    if want != want:
        assert sq != sq and total != total
    else:
        assert sq == want or abs(sq - want) <= CHAIN[torch.float32] * 2.0 ** -24 * want
        assert total == pytest.approx(want ** 0.5, rel=2.0 ** -18) or total == float("inf")


@pytest.mark.parametrize("scale", [2.0 ** 70, 2.0 ** -60])
def test_equal_numbers_beyond_the_range_of_squares(z, scale):  # noqa: F811
    """The numbers that are read again, eight squares to a binary32 sum."""
    x = torch.full((2 ** 28 + 5,), 0.54296875 * scale, device="cuda", dtype=torch.bfloat16)
    _, sq, _, _ = norm(z, z.TensorList([x.data_ptr()] * 16, [x.numel()] * 16, z.BF16), 1.0, tensor_norms=False)
    want = 16 * x.numel() * (0.54296875 * scale) ** 2
    assert abs(sq - want) <= 9 * 2.0 ** -24 * want


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", [2.0 ** 62, 1.5 * 2.0 ** 62, 2.0 ** 63, 1.25 * 2.0 ** 63, 2.0 ** -75])
@pytest.mark.parametrize("n", [1, 2, 3, 5, 7, 8, 11, 40, 263])
def test_few_numbers_whose_squares_fit_alone(z, n, value, dtype):  # noqa: F811
    """A square of 2^124 to 2^127.3 is a binary32 number, as is 2^-150's neighbour; a warp's
    sum of them is none.  Small integers times a power of two: sums are exact in 64 bits."""
    x = torch.full((n + 3,), value, device="cuda", dtype=dtype)
    t = [x[1:1 + n], x[:n], x[3:3 + n]]
    tn, sq, total, _ = norm(z, z.TensorList([v.data_ptr() for v in t], [n] * 3, z.BF16 if dtype == torch.bfloat16
                                            else z.F32), 1.0)
    assert sq == 3 * n * value * value
    assert abs(total - (3 * n) ** 0.5 * value) <= 2.0 ** -23 * total
    assert all(abs(float(v) - n ** 0.5 * value) <= 2.0 ** -23 * value * n ** 0.5 for v in tn)
