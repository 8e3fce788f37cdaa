"""A distillation list that names a token more than once: the loss takes the
entries one by one, the gradient adds up a token's."""
import numpy as np
import pytest

from oracle import vocab_oracle as V

# students (1, 2, 5) / 8 and (1, 0, 1) / 2; the teacher gives token 2 a quarter twice
# and token 0 a half
STUDENTS = np.array([[0.0, np.log(2.0), np.log(5.0)], [0.0, -np.inf, 0.0]])
IDS = np.array([[2, 0, 2]] * 2)
TEACHER = np.array([[0.0, np.log(2.0), 0.0]] * 2)
LOSS = [0.5 * np.log(0.25 / (5 / 8)) + 0.5 * np.log(0.5 / (1 / 8)), -0.5 * np.log(2.0)]
GRAD = [[1 / 8 - 1 / 2, 2 / 8, 5 / 8 - 1 / 2], [0.0, 0.0, 0.0]]


def test_definition():
    loss, dx, _, _ = V.distill(STUDENTS, TEACHER, IDS, 1.0)
    assert loss == pytest.approx(LOSS) and dx == pytest.approx(np.array(GRAD), abs=1e-15)


@pytest.mark.gpu
def test_kernel(lib):
    torch = pytest.importorskip("torch")
    from zero_sharded_optimizer_shard_gb300 import zero3 as Z
    dev = lambda a, dt: torch.as_tensor(a, device="cuda", dtype=dt).contiguous()  # noqa: E731
    x, t = dev(STUDENTS, torch.float32), dev(TEACHER, torch.float32)
    ids, loss, dx = dev(IDS, torch.int64), torch.empty(2, device="cuda"), torch.empty(2, 3, device="cuda")
    Z.zero3_distill_loss(x.data_ptr(), Z.F32, 2, 3, 3, t.data_ptr(), Z.F32, ids.data_ptr(), Z.I64, 3, 3,
                         1.0, None, loss.data_ptr(), None, dx.data_ptr(), 3,
                         torch.cuda.current_stream().cuda_stream)
    # logits rounded to binary32, a few operations on values of order one
    assert loss.tolist() == pytest.approx(LOSS, abs=32 * 2.0 ** -24)
    assert dx.cpu().numpy() == pytest.approx(np.array(GRAD), abs=32 * 2.0 ** -24)
