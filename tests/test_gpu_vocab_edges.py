"""The vocabulary operators on the GPU at the edges of their kernels: rows of
every kind side by side, lists that overflow, sizes at the limits.  Tolerances
as in test_gpu_vocab.py, from binary32 arithmetic.
"""
import ctypes as C

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import vocab_oracle as V  # noqa: E402
from test_gpu_vocab import (DT, U, Mat, close, code, grad_case, grad_tol, ids_tensor,  # noqa: E402
                            logits, rounding, stream, sum_tol, zipf)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def Z(lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from zero_sharded_optimizer_shard_gb300 import zero3
    return zero3


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,vocab,K", [
    (6, 500, 7), (160, 3001, 40), (40, 8193, 130), (6, 9000, 33), (160, 9001, 3), (6, 50257, 64),
    (160, 21003, 300), (80, 40007, 5),
])
def test_distill_rows_of_every_kind_side_by_side(Z, n, vocab, K, dtype):
    """Rows whose list is full, repeated or empty and rows without any student
    token in one call: the warp of the list and the warps of the logits meet
    wherever a row's kind leads them, in place and not, for every number of threads
    per row and of blocks per row."""
    rng = np.random.default_rng(n + vocab + K)
    xs = logits(rng, n, vocab)
    ids = np.stack([rng.choice(vocab, K, replace=False) for _ in range(n)])
    kind = np.arange(n) % 5
    ids[kind == 1] = ids[kind == 1] % 3  # a few tokens, again and again
    ids[kind == 2] = -1
    xs[kind == 3] = -np.inf
    xs[kind == 4, : vocab // 2] = -np.inf
    ids[kind == 4] = vocab // 2 + ids[kind == 4] % (vocab - vocab // 2)
    x = Mat(xs, DT[dtype])
    tm = Mat(rng.normal(size=(n, K)) * 3, DT[dtype])
    idt = ids_tensor(ids, "i64")
    wt = torch.as_tensor(rng.normal(size=n), dtype=torch.float32, device="cuda")
    w, scale = wt.cpu().double().numpy(), 0.75
    loss, lse = torch.full((n,), 9.0, device="cuda"), torch.full((n,), 9.0, device="cuda")
    out = Mat(np.full((n, vocab), 3.0), DT[dtype])
    head = (code(Z, dtype), n, vocab, x.stride, tm.ptr, code(Z, dtype), idt.data_ptr(), Z.I64, K, K, scale)
    rl, rdx, rlse, mag = V.distill(x.host(), tm.host(), ids, scale, w)
    st, qe = sum_tol(vocab), U * (2 * K + 32)
    with np.errstate(invalid="ignore"):
        logp, _ = V._log_softmax(x.host() * scale)
    d, p = np.where(np.isfinite(logp), np.abs(logp), 0), np.exp(logp)
    q = np.zeros_like(p)
    qk = V.teacher_probabilities(tm.host(), ids, scale, vocab)[0]
    for i in range(n):
        np.add.at(q[i], np.where(ids[i] >= 0, ids[i], 0), qk[i])
    big = np.where(np.isfinite(rlse), np.abs(rlse), 0)
    ltol = (qe + st) * (mag + 1 / scale ** 2) + 16 * U * mag + 1e-30
    wa = np.abs(w / scale)[:, None]
    gtol = wa * (p * (2 * st + U * (16 + 6 * d)) + 2 * q * qe) + rounding(dtype, rdx) + 1e-37
    alone = gtol + wa * p * (st + 4 * U * (1 + big))[:, None]

    Z.zero3_distill_loss(x.ptr, *head, wt.data_ptr(), loss.data_ptr(), lse.data_ptr(), out.ptr, vocab,
                         stream())
    close(loss.cpu(), rl, ltol)
    close(lse.cpu(), rlse, st + 2 * U * (1 + big))
    close(out.host(), rdx, gtol)
    both = out.t.clone()
    out.t.fill_(4.0)
    Z.zero3_distill_backward(x.ptr, *head, lse.data_ptr(), wt.data_ptr(), out.ptr, vocab, stream())
    close(out.host(), rdx, alone)
    grad, keep = out.t.clone(), x.t.clone()
    Z.zero3_distill_backward(x.ptr, *head, lse.data_ptr(), wt.data_ptr(), x.ptr, vocab, stream())
    assert torch.equal(x.t, grad)
    x.t.copy_(keep)
    Z.zero3_distill_loss(x.ptr, *head, wt.data_ptr(), loss.data_ptr(), lse.data_ptr(), x.ptr, vocab,
                         stream())
    assert torch.equal(x.t, both)
    assert x.intact() and out.intact() and tm.intact()
    quiet = (kind == 2) | (kind == 3)
    assert not both[quiet].any() and not grad[quiet].any() and not loss[quiet].any()


@pytest.mark.parametrize("accumulate,tail", [(False, 0), (True, 100)])
@pytest.mark.parametrize("dim", [1, 8])
def test_embedding_backward_largest_batch(Z, dim, accumulate, tail):
    """2^31 - 1 positions, all of one token but the last `tail`, of another: the
    indices of the last pieces, and the counts, lie next to 2^31.  Every sum of
    ones is exact: pieces hold 128 rows, and a multiple of 128 below 2^31
    has 24 bits."""
    n = 2 ** 31 - 1
    ids = torch.zeros(n, device="cuda", dtype=torch.int32)
    if tail:
        ids[-tail:] = 1
    dout = torch.ones(n, dim, device="cuda", dtype=torch.bfloat16)
    grad = torch.full((3, dim), 0.5, device="cuda")
    nb = Z.zero3_embedding_workspace(n, 3, dim)
    ws = torch.empty(nb, device="cuda", dtype=torch.uint8)
    Z.zero3_embedding_backward(dout.data_ptr(), Z.BF16, dim, ids.data_ptr(), Z.I32, n, 1.0,
                               int(accumulate), grad.data_ptr(), Z.F32, 3, dim, dim, ws.data_ptr(), nb,
                               stream())
    base = 0.5 if accumulate else 0.0
    want = np.float32([n - tail + base, tail + base if tail else 0.0, base])
    assert np.array_equal(grad.cpu().numpy(), np.repeat(want[:, None], dim, 1))
    del ids, dout, ws
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("weight", [1e6, -1e9, 1e20, -1e36])
@pytest.mark.parametrize("vocab,pad", [(40, 0), (1001, 0), (1001, 1), (9001, 0)])
def test_entropy_gradient_of_large_weights(Z, dtype, weight, vocab, pad):
    """Masked tokens have no gradient however large the entropy's weight is, by the
    wide path and by single elements."""
    n, scale = 5, 0.75
    rng = np.random.default_rng(vocab)
    xs = logits(rng, n, vocab, "masked")
    xs[2, 1::2] = -3.3895313892515355e38  # finite, and without weight all the same
    x, t = Mat(xs, DT[dtype], vocab + pad), rng.integers(0, vocab, n)
    it = ids_tensor(t, "i64")
    lp, lse, ent = (torch.empty(n, device="cuda") for _ in range(3))
    Z.zero3_token_logprobs(x.ptr, code(Z, dtype), n, vocab, x.stride, it.data_ptr(), Z.I64, scale, 0,
                           lp.data_ptr(), lse.data_ptr(), ent.data_ptr(), stream=stream())
    g = torch.as_tensor(rng.normal(size=n), dtype=torch.float32, device="cuda")
    h = torch.as_tensor(rng.uniform(0.5, 1, size=n) * weight, dtype=torch.float32, device="cuda")
    dx = Mat(np.full((n, vocab), 3.0), DT[dtype])
    Z.zero3_token_logprobs_backward(x.ptr, code(Z, dtype), n, vocab, x.stride, it.data_ptr(), Z.I64,
                                    scale, lse.data_ptr(), ent.data_ptr(), g.data_ptr(), h.data_ptr(),
                                    dx.ptr, dx.stride, stream())
    g, h = g.cpu().double().numpy(), h.cpu().double().numpy()
    want = V.token_logprobs_backward(x.host(), t, scale, g, h)
    ref = V.token_logprobs(x.host(), t, scale)
    with np.errstate(invalid="ignore"):
        logp, _ = V._log_softmax(V.scaled(x.host(), scale))
    p, H = np.exp(logp), ref["entropy"]
    eps = sum_tol(vocab) + 2 * U * (1 + np.where(np.isfinite(ref["lse"]), np.abs(ref["lse"]), 0))
    size = np.where(p > 0, np.abs(np.where(p > 0, logp, 0)), 0)
    w = np.abs(g)[:, None] + np.abs(h)[:, None] * (size + H[:, None] + 1)
    tol = grad_tol(dtype, want, p, np.where(p > 0, logp, 0), g, h, H, scale) + \
        scale * p * w * (4 + H[:, None]) * eps[:, None]
    close(dx.host(), want, tol)
    masked = p == 0
    masked[np.arange(n), t] = False
    assert not dx.host()[masked].any()
    assert x.intact() and dx.intact()


def test_an_earlier_calls_error_is_not_this_calls(Z):
    """A synchronisation refused because its stream is being captured leaves an error
    code behind in the runtime; the launches after it succeed and do their work."""
    from examples.tied_lm import TiedLM
    lm = TiedLM(vocab=64, dim=16, hidden=16)
    table = torch.randn(8, 16, device="cuda")
    ids = torch.arange(8, device="cuda").flip(0)
    out, grad = torch.zeros(8, 16, device="cuda"), torch.zeros(8, 16, device="cuda")
    ws = torch.empty(Z.zero3_embedding_workspace(8, 8, 16), device="cuda", dtype=torch.uint8)
    x, lp, loss = torch.randn(8, 8, device="cuda"), torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda")
    tl, full, s = torch.zeros(8, 1, device="cuda"), torch.zeros_like(lm.full), stream()
    torch.cuda.synchronize()
    rt = C.CDLL("libcudart.so.%s" % torch.version.cuda.split(".")[0])

    def refused():
        st, graph = C.c_void_p(), C.c_void_p()
        assert rt.cudaStreamCreate(C.byref(st)) == 0
        assert rt.cudaStreamBeginCapture(st, 2) == 0
        assert Z.raw_status("zero3_sync", st) == Z.ECUDA
        assert rt.cudaStreamEndCapture(st, C.byref(graph)) != 0 and not graph.value
        assert rt.cudaStreamDestroy(st) == 0
        rt.cudaGetLastError()  # the caller's own runtime is clean

    refused()
    Z.zero3_embedding_forward(table.data_ptr(), Z.F32, 8, 16, 16, ids.data_ptr(), Z.I64, 8, 1.0,
                              out.data_ptr(), Z.F32, 16, s)
    refused()
    Z.zero3_embedding_backward(table.data_ptr(), Z.F32, 16, ids.data_ptr(), Z.I64, 8, 1.0, 0,
                               grad.data_ptr(), Z.F32, 8, 16, 16, ws.data_ptr(), ws.numel(), s)
    refused()
    Z.zero3_token_logprobs(x.data_ptr(), Z.F32, 8, 8, 8, ids.data_ptr(), Z.I64, 1.0, 0, lp.data_ptr(),
                           stream=s)
    refused()
    Z.zero3_distill_loss(x.data_ptr(), Z.F32, 8, 8, 8, tl.data_ptr(), Z.F32, ids.data_ptr(), Z.I64, 1, 1,
                         1.0, None, loss.data_ptr(), stream=s)
    refused()  # the library's other launches
    Z.zero3_cast_params(lm.plan, lm._ptrs(lm.master), lm._ptrs(lm.sparam), full.data_ptr(), None, 0,
                        lm.plan.info.psi_pad, s)
    refused()
    wte = lm.gather()[0]
    torch.cuda.synchronize()
    assert torch.equal(out, table[ids]) and torch.equal(grad, out)
    assert torch.equal(full, lm.full) and torch.equal(wte.flatten(), full[:64 * 16])
    want = torch.log_softmax(x, 1)[torch.arange(8), ids]
    assert torch.allclose(lp, want, atol=1e-5) and torch.allclose(loss, -want, atol=1e-5)
    lm.release()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,vocab,pad", [(5, 300, 0), (5, 300, 1), (7, 9001, 0), (170, 50001, 0), (5, 50001, 3)])
def test_distill_not_finite_rows(Z, dtype, n, vocab, pad):
    """Which of an empty list, a list that is not finite, a row without any student
    token and logits that are not finite decides: the loss and every form of
    the gradient agree."""
    K, rng = 6, np.random.default_rng(vocab)
    xs, ts = rng.normal(size=(n, vocab)), rng.normal(size=(n, K))
    ids = np.stack([rng.choice(vocab, K, replace=False) for _ in range(n)])
    xs[0], ts[0, 3] = -np.inf, np.nan  # a NaN in the list, no student token
    xs[1], ts[1, 0] = -np.inf, np.inf
    xs[2, vocab // 2], ids[2] = np.nan, -1  # a NaN in the logits, no entry
    xs[3, vocab - 1] = np.inf
    ts[4, 1], ids[4, 1] = np.nan, vocab  # an entry that does not count
    x, tm, it = Mat(xs, DT[dtype], vocab + pad), Mat(ts, DT[dtype]), ids_tensor(ids, "i32")
    loss, lse = torch.full((n,), 9.0, device="cuda"), torch.full((n,), 9.0, device="cuda")
    head = (code(Z, dtype), n, vocab, x.stride, tm.ptr, code(Z, dtype), it.data_ptr(), Z.I32, K, K, 1.0)
    dx = Mat(np.full((n, vocab), 3.0), DT[dtype])

    def check():
        bad = torch.isnan(dx.t)
        assert bad[[0, 1, 3]].all() and not bad[[2, 4]].any() and not bad[5:].any()
        assert not dx.t[2].any() and dx.t[4].any()
        assert x.intact() and dx.intact()
        dx.t.fill_(4.0)
    Z.zero3_distill_loss(x.ptr, *head, None, loss.data_ptr(), lse.data_ptr(), dx.ptr, dx.stride, stream())
    check()
    assert torch.isnan(loss[[0, 1, 3]]).all() and loss[2] == 0 and torch.isfinite(loss[4:]).all()
    assert torch.isneginf(lse[:2]).all() and torch.isnan(lse[2:4]).all()
    Z.zero3_distill_backward(x.ptr, *head, lse.data_ptr(), None, dx.ptr, dx.stride, stream())
    check()
    alone = torch.full((n,), 9.0, device="cuda")
    Z.zero3_distill_loss(x.ptr, *head, None, alone.data_ptr(), None, None, 0, stream())
    assert torch.isnan(alone[[0, 1, 3]]).all() and alone[2] == 0
    keep = x.t.clone()
    Z.zero3_distill_backward(x.ptr, *head, lse.data_ptr(), None, x.ptr, x.stride, stream())
    dx.t.copy_(x.t)
    check()
    x.t.copy_(keep)
    Z.zero3_distill_loss(x.ptr, *head, None, loss.data_ptr(), None, x.ptr, x.stride, stream())
    dx.t.copy_(x.t)
    check()


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dim", [8, 13])
@pytest.mark.parametrize("n,vocab,share", [(20000, 50, 1.0), (33000, 3000, 0.95), (65536, 70000, 0.9)])
def test_embedding_backward_one_token_fills_the_batch(Z, n, vocab, share, dim, accumulate):
    """More positions of one token (padding inside the vocabulary, say) than a sorting
    warp lists: it reads the ids again, next to warps that need not."""
    rng = np.random.default_rng(n)
    ids = zipf(rng, n, vocab)
    ids[rng.random(n) < share] = 7
    assert (ids[: n // 32] == 7).sum() > 512
    ids[n - n // 16:] = rng.integers(0, vocab, n // 16)  # the last warps' lists do not overflow
    grad_case(Z, n, vocab, dim, "f32", "f32", "i64", ids, accumulate=accumulate)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n", [700, 3001, 9000])
@pytest.mark.parametrize("vocab", [65536, 65537, 131073, 300007])
def test_embedding_backward_large_vocabularies(Z, vocab, n, accumulate):
    """128 sorting blocks, 256, 512 and 1024."""
    rng = np.random.default_rng(vocab + n)
    ids = np.where(rng.random(n) < 0.5, zipf(rng, n, vocab), rng.integers(vocab - 600, vocab + 2, n))
    grad_case(Z, n, vocab, 8 if n % 2 else 11, "bf16", "f32", "i32", ids, accumulate=accumulate)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("gd", ["bf16", "f32"])
@pytest.mark.parametrize("n,dim", [(8192, 2048), (8192, 2056), (7300, 2312), (32769, 512), (16400, 1024)])
def test_embedding_backward_two_groups_per_lane(Z, n, dim, gd, accumulate):
    """Batches of at least 2^24 elements, rows of any multiple of 8 from 2048 on: the
    last columns' second group lies in the row, partly in it, or past its end."""
    assert n * dim >= 1 << 24
    grad_case(Z, n, 300, dim, "bf16", gd, "i64", zipf(np.random.default_rng(dim), n, 300), accumulate=accumulate,
              scale=0.5)


@pytest.mark.parametrize("dim", [1, 8])
def test_embedding_backward_long_shares(Z, dim):
    """A sorting warp's share of more than 65536 positions, which its list cannot
    number."""
    n, vocab = 32 * 65536 + 77, 1009
    rng = np.random.default_rng(dim)
    ids = rng.integers(-1, vocab + 1, n)
    d = Mat(rng.normal(size=(n, dim)), torch.bfloat16)
    grad, it = torch.full((vocab, dim), 3.0, device="cuda"), ids_tensor(ids, "i32")
    nb = Z.zero3_embedding_workspace(n, vocab, dim)
    ws = torch.empty(nb, device="cuda", dtype=torch.uint8)
    Z.zero3_embedding_backward(d.ptr, Z.BF16, dim, it.data_ptr(), Z.I32, n, 0.5, 0, grad.data_ptr(), Z.F32,
                               vocab, dim, dim, ws.data_ptr(), nb, stream())
    keep = (ids >= 0) & (ids < vocab)
    x, t = 0.5 * d.host()[keep], ids[keep]
    ref = np.stack([np.bincount(t, x[:, c], vocab) for c in range(dim)], 1)
    mag = np.stack([np.bincount(t, np.abs(x[:, c]), vocab) for c in range(dim)], 1)
    close(grad.cpu(), ref, (np.bincount(t, minlength=vocab)[:, None] + 4) * U * mag + U * np.abs(ref))
