"""Refusals at the size limits of the vocabulary operators: each call is valid but
for one limit, which it exceeds by the least; just inside a limit, empty calls and
workspace queries, which touch no GPU, are accepted."""
import ctypes as C

import pytest

from test_vocab_host import GOOD, z  # noqa: F401

LOGITS = ["zero3_token_logprobs", "zero3_token_logprobs_backward", "zero3_distill_loss",
          "zero3_distill_backward"]
EMBED = ["zero3_embedding_forward", "zero3_embedding_backward"]
VOCAB, ROWS, TOKENS, DIM, ELEMS = 1 << 30, 1 << 27, (1 << 31) - 1, 1 << 27, 1 << 41


def sized(name, n, vocab=None, dim=None):
    """A call of these sizes with its strides to match."""
    args = dict(GOOD[name], n=n)
    if vocab is not None:
        args["vocab"] = vocab
    cols = dim if name in EMBED else args["vocab"]
    if dim is not None:
        args["dim"] = dim
    for a in ("stride", "dlogits_stride", "table_stride", "out_stride", "dout_stride", "grad_stride"):
        if a in args:
            args[a] = cols
    if "workspace_bytes" in args:
        args["workspace_bytes"] = 1 << 62
    return args


def status(z, name, args):  # noqa: F811
    return z.raw_status(name, *args.values())


@pytest.mark.parametrize("name", LOGITS)
@pytest.mark.parametrize("n,vocab", [(1, VOCAB + 1), (ROWS + 1, 100), (ROWS, ELEMS // ROWS + 1),
                                     ((1 << 21) + 1, 1 << 20)])
def test_logits_beyond_one_limit(z, name, n, vocab):  # noqa: F811
    assert status(z, name, sized(name, n, vocab)) == z.EINVAL


@pytest.mark.parametrize("name", LOGITS)
def test_logits_inside_the_limit(z, name):  # noqa: F811
    assert status(z, name, sized(name, 0, VOCAB)) == z.OK
    assert status(z, name, sized(name, 0, VOCAB + 1)) == z.EINVAL


@pytest.mark.parametrize("name", EMBED)
@pytest.mark.parametrize("n,vocab,dim", [
    (1, VOCAB + 1, 1), (TOKENS + 1, 100, 1), (1, 1, DIM + 1), (TOKENS, 1, ELEMS // TOKENS + 1),
    (1, VOCAB, ELEMS // VOCAB + 1)])
def test_embedding_beyond_one_limit(z, name, n, vocab, dim):  # noqa: F811
    assert status(z, name, sized(name, n, vocab, dim)) == z.EINVAL
    out = C.c_int64()
    assert z.raw_status("zero3_embedding_workspace", n, vocab, dim, C.byref(out)) == z.EINVAL


@pytest.mark.parametrize("n,vocab,dim", [(1, VOCAB, 1), (TOKENS, 100, 1), (1, 1, DIM),
                                         (TOKENS, 1, ELEMS // TOKENS), (1, VOCAB, ELEMS // VOCAB)])
def test_embedding_inside_the_limit(z, n, vocab, dim):  # noqa: F811
    assert z.zero3_embedding_workspace(n, vocab, dim) >= 4 * vocab + 16 * n
    args = sized("zero3_embedding_forward", 0, vocab, dim)
    assert status(z, "zero3_embedding_forward", args) == z.OK


def test_workspace_one_byte_short(z):  # noqa: F811
    need = z.zero3_embedding_workspace(4, 100, 16)
    args = dict(GOOD["zero3_embedding_backward"], workspace_bytes=need - 1)
    assert status(z, "zero3_embedding_backward", args) == z.EINVAL
