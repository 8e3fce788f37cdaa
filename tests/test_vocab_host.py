"""Refusals of the vocabulary operators: every call below carries one invalid
argument, which the library rejects before it touches the GPU."""
import ctypes as C

import pytest

A = 1 << 20  # a plausible, aligned address that is never read


@pytest.fixture(scope="module")
def z(lib):
    from zero_sharded_optimizer_shard_gb300 import zero3
    return zero3


GOOD = {
    "zero3_embedding_forward": dict(table=A, table_dtype=0, vocab=100, dim=16, table_stride=16,
                                    ids=A, id_type=0, n=4, scale=1.0, out=A, out_dtype=0,
                                    out_stride=16, stream=None),
    "zero3_embedding_backward": dict(dout=A, dout_dtype=0, dout_stride=16, ids=A, id_type=1, n=4,
                                     scale=1.0, accumulate=0, grad=A, grad_dtype=0, vocab=100,
                                     dim=16, grad_stride=16, workspace=A, workspace_bytes=1 << 20,
                                     stream=None),
    "zero3_token_logprobs": dict(logits=A, dtype=0, n=4, vocab=100, stride=100, targets=A,
                                 id_type=0, inv_temperature=1.0, k=3, logprob=A, lse=A, entropy=A,
                                 top_ids=A, top_logprobs=A, stream=None),
    "zero3_token_logprobs_backward": dict(logits=A, dtype=0, n=4, vocab=100, stride=100, targets=A,
                                          id_type=0, inv_temperature=1.0, lse=A, entropy=A,
                                          dlogprob=A, dentropy=A, dlogits=2 * A,
                                          dlogits_stride=100, stream=None),
    "zero3_distill_loss": dict(logits=A, dtype=0, n=4, vocab=100, stride=100, teacher_logits=A,
                               teacher_dtype=1, teacher_ids=A, id_type=1, k=8, teacher_stride=8,
                               inv_temperature=1.0, row_weight=A, loss=A, lse=A, dlogits=2 * A,
                               dlogits_stride=100, stream=None),
    "zero3_distill_backward": dict(logits=A, dtype=0, n=4, vocab=100, stride=100, teacher_logits=A,
                                   teacher_dtype=1, teacher_ids=A, id_type=1, k=8,
                                   teacher_stride=8, inv_temperature=1.0, lse=A, dloss=A,
                                   dlogits=2 * A, dlogits_stride=100, stream=None),
}
NAN, INF = float("nan"), float("inf")
LOGITS = [("logits", None), ("logits", A + 1), ("dtype", 2), ("dtype", -1), ("n", -1),
          ("n", 1 << 28), ("vocab", 0), ("vocab", (1 << 30) + 1), ("stride", 99), ("id_type", 2),
          ("inv_temperature", 0.0), ("inv_temperature", -1.0), ("inv_temperature", NAN),
          ("inv_temperature", INF)]
DISTILL = LOGITS + [("teacher_logits", None), ("teacher_logits", A + 2), ("teacher_dtype", 3),
                    ("teacher_ids", None), ("teacher_ids", A + 4), ("k", 0), ("k", 1025),
                    ("teacher_stride", 7), ("dlogits_stride", 99), ("dlogits", 2 * A + 1)]
BAD = {
    "zero3_embedding_forward": [
        ("table", None), ("table", A + 1), ("table_dtype", 2), ("vocab", 0), ("vocab", 1 << 31),
        ("dim", 0), ("dim", 1 << 40), ("table_stride", 15), ("ids", None), ("ids", A + 2),
        ("id_type", 5), ("n", -1), ("n", 1 << 31), ("scale", NAN), ("scale", INF), ("out", None),
        ("out", A + 1), ("out_dtype", -1), ("out_stride", 15)],
    "zero3_embedding_backward": [
        ("dout", None), ("dout", A + 1), ("dout_dtype", 2), ("dout_stride", 15), ("ids", None),
        ("ids", A + 4), ("id_type", 2), ("n", -1), ("n", 1 << 31), ("scale", NAN), ("grad", None),
        ("grad", A + 1), ("grad_dtype", 4), ("vocab", 0), ("dim", 0), ("grad_stride", 15),
        ("workspace", None), ("workspace", A + 8), ("workspace_bytes", 100)],
    "zero3_token_logprobs": LOGITS + [
        ("targets", None), ("targets", A + 2), ("k", -1), ("k", 65), ("vocab", 2), ("logprob", None),
        ("logprob", A + 2), ("lse", A + 1), ("entropy", A + 1), ("top_ids", None),
        ("top_logprobs", None)],
    "zero3_token_logprobs_backward": LOGITS + [
        ("targets", None), ("lse", None), ("entropy", None), ("dlogits", None),
        ("dlogits", 2 * A + 1), ("dlogits_stride", 99), ("dlogprob", A + 2), ("dentropy", A + 3)],
    "zero3_distill_loss": DISTILL + [("loss", None), ("loss", A + 1), ("lse", A + 2),
                                     ("row_weight", A + 2)],
    "zero3_distill_backward": DISTILL + [("lse", None), ("dloss", A + 2), ("dlogits", None)],
}


@pytest.mark.parametrize("name,arg,value", [(f, a, v) for f, bad in BAD.items() for a, v in bad])
def test_refused(z, name, arg, value):
    args = dict(GOOD[name])
    assert arg in args
    args[arg] = value
    assert z.raw_status(name, *args.values()) == z.EINVAL


def test_both_gradients_absent_is_refused(z):
    args = dict(GOOD["zero3_token_logprobs_backward"], dlogprob=None, dentropy=None)
    assert z.raw_status("zero3_token_logprobs_backward", *args.values()) == z.EINVAL


@pytest.mark.parametrize("name", ["zero3_token_logprobs_backward", "zero3_distill_loss",
                                  "zero3_distill_backward"])
def test_in_place_needs_equal_strides(z, name):
    args = dict(GOOD[name], dlogits=A, dlogits_stride=101)
    assert z.raw_status(name, *args.values()) == z.EINVAL


@pytest.mark.parametrize("name", list(GOOD))
def test_empty_call_is_accepted(z, name):
    args = dict(GOOD[name], n=0)
    if name == "zero3_embedding_backward":
        args["accumulate"] = 1  # nothing to add: nothing is written
    for a in ("table", "ids", "logits", "targets"):
        if a in args:
            args[a] = None
    assert z.raw_status(name, *args.values()) == z.OK


def test_refusal_raises_in_the_binding(z):
    with pytest.raises(z.Zero3Error) as e:
        z.zero3_token_logprobs(A, z.BF16, 4, 100, 99, A, z.I64, 1.0, 0, A)
    assert e.value.status == z.EINVAL


def test_workspace(z):
    for n, V, d in [(0, 1, 1), (1, 50257, 2048), (32768, 50257, 2048), (5, 3, 7)]:
        b = z.zero3_embedding_workspace(n, V, d)
        assert 4 * (V + 1) + 4 * n <= b
        assert b <= 4 * (V + 600) + 16 * n + (n // 16 + 1) * (8 * (d + 3) + 4 * (d // 256 + 1)) + 80
    out = C.c_int64()
    for bad in [(-1, 5, 5), (1, 0, 5), (1, 5, 0), (1 << 31, 5, 5), (1, 5, 1 << 42),
                (1, 1, (1 << 27) + 1)]:
        assert z.raw_status("zero3_embedding_workspace", *bad, C.byref(out)) == z.EINVAL
    assert z.raw_status("zero3_embedding_workspace", 1, 1, 1, None) == z.EINVAL
