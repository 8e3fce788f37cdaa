"""The vocabulary operators on the GPU against their 64-bit definitions.

Tolerances follow from binary32 arithmetic (unit roundoff u = 2^-24) and one
rounding at the end:
 - a row's sum S of positive terms has relative error at most u times the
   longest chain of additions, below V / 1024 + 64 with the join of a block,
   plus a few u for the exponentials (2 ulp) and their arguments; log S has
   that error absolutely;
 - a probability exp(d), d = z - lse, carries 4 u |d| from its argument
   and 8 u of its own;
 - a bf16 result is within half an ulp, 2^-8 relative, of the binary32 one.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import vocab_oracle as V  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def Z(lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from zero_sharded_optimizer_shard_gb300 import zero3
    return zero3


class Mat:
    """A row-major matrix inside a larger buffer of sentinels: `offset`
    elements from its start, rows `stride` apart."""

    def __init__(self, data, dtype, stride=None, offset=0):
        rows, cols = data.shape
        self.stride = stride or cols
        self.buf = torch.full((offset + rows * self.stride + 16,), 777.0, device="cuda",
                              dtype=dtype)
        self.t = torch.as_strided(self.buf, (rows, cols), (self.stride, 1), offset)
        self.t.copy_(torch.as_tensor(data))
        self.ptr = self.buf.data_ptr() + offset * self.buf.element_size()
        self.mask = torch.ones_like(self.buf, dtype=torch.bool)
        torch.as_strided(self.mask, (rows, cols), (self.stride, 1), offset).fill_(False)

    def host(self):
        return self.t.double().cpu().numpy()

    def intact(self):
        return bool((self.buf[self.mask] == 777.0).all())


def code(Z, name):
    return Z.BF16 if name == "bf16" else Z.F32


def rounding(name, ref):
    """Error of storing a value: half an ulp."""
    return (2.0 ** -8 if name == "bf16" else U) * np.abs(ref)


def close(got, ref, tol):
    """Equal infinities and NaNs, and within tol elsewhere."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    tol = np.broadcast_to(tol, ref.shape)
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf])
    assert np.isfinite(got[fin]).all()
    bad = np.abs(got - ref)[fin] > tol[fin]
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - ref)[fin] / np.maximum(tol[fin], 1e-300)).max()))


def stream():
    return torch.cuda.current_stream().cuda_stream


def ids_tensor(ids, kind):
    return torch.as_tensor(np.asarray(ids), device="cuda",
                           dtype=torch.int32 if kind == "i32" else torch.int64)


def id_code(Z, kind):
    return Z.I32 if kind == "i32" else Z.I64


# ------------------------------------------------------------------ embedding
EMBED = [  # n, vocab, dim, table dtype, out dtype, ids, strides beyond dim, offsets
    (1, 1, 1, "f32", "f32", "i32", 0, 0), (1, 50257, 2048, "bf16", "bf16", "i64", 0, 0),
    (5, 7, 8, "bf16", "bf16", "i32", 0, 0), (5, 7, 8, "bf16", "f32", "i64", 8, 8),
    (33, 100, 767, "bf16", "bf16", "i64", 0, 0), (33, 100, 768, "bf16", "bf16", "i64", 0, 1),
    (33, 100, 768, "f32", "bf16", "i32", 3, 0), (2500, 1000, 256, "bf16", "bf16", "i64", 8, 16),
    (701, 300, 1021, "f32", "f32", "i32", 0, 3), (300, 50, 4104, "f32", "f32", "i64", 0, 4),
]


@pytest.mark.parametrize("n,vocab,dim,td,od,kind,pad,off", EMBED)
def test_embedding_forward(Z, n, vocab, dim, td, od, kind, pad, off):
    rng = np.random.default_rng(n + dim)
    ids = rng.integers(0, vocab, n)
    if n > 4:
        ids[[0, 2, n - 1]] = [-1, vocab, -(1 << 31)]
    if kind == "i64" and n > 4:
        ids[3] = (1 << 32) + 1  # not token 1
    table = Mat(rng.normal(size=(vocab, dim)), DT[td], dim + pad, off)
    out = Mat(np.full((n, dim), 5.0), DT[od], dim + pad, off)
    it = ids_tensor(ids, kind)
    for scale in (1.0, 27.5):
        Z.zero3_embedding_forward(table.ptr, code(Z, td), vocab, dim, table.stride, it.data_ptr(),
                                  id_code(Z, kind), n, scale, out.ptr, code(Z, od), out.stride,
                                  stream())
        ref = V.embedding_forward(table.host(), ids, scale)
        close(out.host(), ref, rounding(od, ref) + U * np.abs(ref))
        assert out.intact() and table.intact()


@pytest.mark.parametrize("off", [0, 1, 2, 3, 5, 7])
@pytest.mark.parametrize("td,od", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_embedding_forward_any_alignment(Z, td, od, off):
    """Rows that start anywhere between two 16-byte boundaries, down to tables
    smaller than the words that a row is read by."""
    for dim in list(range(1, 19)) + [31, 71]:
        for vocab, pad in ((1, 0), (3, 0), (40, 5)):
            n = 9
            rng = np.random.default_rng(dim)
            ids = rng.integers(0, vocab, n)
            ids[4] = vocab
            table = Mat(rng.normal(size=(vocab, dim)), DT[td], dim + pad, off)
            out = Mat(np.full((n, dim), 5.0), DT[od], dim + (dim + pad) % 3, (3 * off) % 8)
            it = ids_tensor(ids, "i64")
            Z.zero3_embedding_forward(table.ptr, code(Z, td), vocab, dim, table.stride, it.data_ptr(),
                                      Z.I64, n, 0.75, out.ptr, code(Z, od), out.stride, stream())
            ref = V.embedding_forward(table.host(), ids, 0.75)
            close(out.host(), ref, rounding(od, ref) + U * np.abs(ref))
            assert out.intact() and table.intact()


def grad_case(Z, n, vocab, dim, dd, gd, kind, ids, pad=0, off=0, accumulate=False, scale=1.0):
    rng = np.random.default_rng(n + dim + vocab)
    d = Mat(rng.normal(size=(n, dim)), DT[dd], dim + pad, off)
    base = rng.normal(size=(vocab, dim))
    g = Mat(base, DT[gd], dim + pad, off)
    base = g.host()
    it = ids_tensor(ids, kind)
    nb = Z.zero3_embedding_workspace(n, vocab, dim)
    ws = torch.full((nb + 64,), 0xA5, device="cuda", dtype=torch.uint8)

    def call():
        Z.zero3_embedding_backward(d.ptr, code(Z, dd), d.stride, it.data_ptr(), id_code(Z, kind), n,
                                   scale, int(accumulate), g.ptr, code(Z, gd), vocab, dim, g.stride,
                                   ws.data_ptr(), nb, stream())
    call()
    got = g.host()
    ref, mag, count = V.embedding_backward(d.host(), ids, scale, vocab, base if accumulate else None)
    tol = (count[:, None] + 4) * U * (mag + (np.abs(base) if accumulate else 0)) + rounding(gd, ref)
    close(got, ref, tol)
    assert g.intact() and d.intact() and bool((ws[nb:] == 0xA5).all())
    untouched = count == 0
    want = base[untouched] if accumulate else 0.0
    assert np.array_equal(got[untouched], np.broadcast_to(want, got[untouched].shape))
    if not accumulate:  # the same bits again
        call()
        assert np.array_equal(g.host(), got)


def zipf(rng, n, vocab):
    w = 1.0 / (np.arange(vocab) + 2.7)
    ids = rng.choice(vocab, n, p=w / w.sum())
    ids[rng.random(n) < 0.02] = -1
    return ids


@pytest.mark.parametrize("off", [0, 1, 3, 6])
@pytest.mark.parametrize("dd,gd", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
def test_embedding_backward_any_alignment(Z, dd, gd, off):
    """Rows that start anywhere between two 16-byte boundaries, next to other
    rows, gaps and the matrix's ends, with single and repeated tokens."""
    rng = np.random.default_rng(off)
    for dim in [1, 2, 3, 5, 7, 9, 15, 17, 63, 71, 255, 257, 263, 521]:
        for n, vocab, pad in ((1, 1, 0), (5, 3, 0), (90, 40, 0), (90, 4, 5)):
            grad_case(Z, n, vocab, dim, dd, gd, "i32", rng.integers(-1, vocab, n), pad, off,
                      (dim + n) % 2 == 0, 0.75)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,vocab,dim,dd,gd,kind,pad,off", [
    (1, 1, 1, "f32", "f32", "i32", 0, 0), (1, 50257, 768, "bf16", "bf16", "i64", 0, 0),
    (64, 9, 8, "bf16", "f32", "i64", 8, 8), (65, 352, 40, "bf16", "bf16", "i32", 0, 0),
    (1000, 353, 257, "f32", "f32", "i32", 0, 0), (3000, 1000, 264, "bf16", "bf16", "i64", 0, 1),
    (3000, 1000, 512, "f32", "bf16", "i64", 4, 4), (2047, 5000, 1032, "bf16", "bf16", "i32", 0, 0),
    (4100, 1000, 771, "bf16", "f32", "i64", 5, 3), (20000, 60000, 16, "f32", "f32", "i64", 0, 0),
    (40001, 3000, 24, "bf16", "bf16", "i32", 0, 0),
])
def test_embedding_backward(Z, n, vocab, dim, dd, gd, kind, pad, off, accumulate):
    ids = zipf(np.random.default_rng(n), n, vocab)
    grad_case(Z, n, vocab, dim, dd, gd, kind, ids, pad, off, accumulate, 1.0 if n % 2 else 0.37)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("counts", [
    [64], [65], [256], [257], [512], [513, 64, 65, 1], [1, 64, 65, 64, 321, 2, 1023],
    [63, 66, 63, 130], [5000], [0, 0, 700, 0, 3],
])
@pytest.mark.parametrize("dim", [8, 13, 1040])
def test_embedding_backward_counts(Z, counts, dim, accumulate):
    """Tokens whose positions end at and around the tiles' edges, in a
    shuffled order."""
    ids = np.concatenate([np.full(c, 3 + v) for v, c in enumerate(counts)])
    np.random.default_rng(len(ids)).shuffle(ids)
    grad_case(Z, len(ids), 3 + len(counts), dim, "bf16", "f32", "i64", ids, accumulate=accumulate)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("ids", [[-1] * 70, [], [5] * 3 + [-7] * 100, [99, 0]])
def test_embedding_backward_sparse(Z, ids, accumulate):
    grad_case(Z, len(ids), 100, 32, "f32", "f32", "i32", np.asarray(ids, np.int64),
              accumulate=accumulate)


@pytest.mark.parametrize("dim", [24, 27])
@pytest.mark.parametrize("n", [1024, 1025, 4096, 4097, 32768, 32769])
def test_embedding_backward_batch_sizes(Z, n, dim):
    """Frequent tokens in batches at the edges of the sizes that are sorted and
    summed differently."""
    grad_case(Z, n, 300, dim, "f32", "f32", "i32", zipf(np.random.default_rng(n), n, 300))


@pytest.mark.parametrize("n", [8191, 8192, 32769])
def test_embedding_backward_wide_rows(Z, n):
    grad_case(Z, n, 700, 2048 if n < 10000 else 512, "bf16", "bf16", "i64",
              zipf(np.random.default_rng(n), n, 700), accumulate=True, scale=0.5)


@pytest.mark.parametrize("dim", [16, 19])
@pytest.mark.parametrize("accumulate", [False, True])
def test_embedding_backward_pieces(Z, dim, accumulate):
    """Tokens with as many positions as fill pieces of every length exactly, or
    one more or less."""
    counts = [7, 8, 9, 15, 16, 17, 31, 32, 33, 511, 512, 513, 2047, 2048, 2049, 8191, 8192, 8193]
    ids = np.concatenate([np.full(c, 5 * v + 2) for v, c in enumerate(counts)])
    np.random.default_rng(1).shuffle(ids)
    grad_case(Z, len(ids), 100, dim, "bf16", "f32", "i32", ids, accumulate=accumulate)



# ------------------------------------------------------------ log probabilities
def logits(rng, n, vocab, kind="normal"):
    x = rng.normal(size=(n, vocab)) * 3
    if kind == "ties":
        x = np.round(x)
    if kind == "constant":
        x[:] = -4.25
    if kind == "masked":
        for i in range(n):
            keep = rng.random(vocab) < (0.0 if i % 4 == 0 else 6.0 / vocab if i % 4 == 1 else 0.3)
            x[i, ~keep] = -np.inf
    if kind == "lowest":  # the type's lowest value as a mask
        x[rng.random((n, vocab)) < 0.7] = -3.3895313892515355e38
        x[0] = -3.3895313892515355e38
    if kind == "sorted":
        x = -np.sort(-x, axis=1)
    if kind == "large":
        x = x * 300 + 5000
    return x


def sum_tol(vocab):
    return U * (vocab / 1024 + 64)


def logprob_case(Z, n, vocab, dtype, kind, k, pad=0, off=0, ids="i64", scale=1.0, entropy=True):
    rng = np.random.default_rng(n * 7 + vocab + k)
    x = Mat(logits(rng, n, vocab, kind), DT[dtype], vocab + pad, off)
    t = rng.integers(0, vocab, n)
    if n > 2:
        t[1] = -100
        t[2] = vocab
    it = ids_tensor(t, ids)
    f = lambda *s: torch.full(s, 9.0, device="cuda")  # noqa: E731
    lp, lse, ent, tl = f(n), f(n), f(n), f(n, max(k, 1))
    ti = torch.full((n, max(k, 1)), -5, device="cuda", dtype=torch.int32)
    p = lambda y, on=True: y.data_ptr() if on else None  # noqa: E731
    Z.zero3_token_logprobs(x.ptr, code(Z, dtype), n, vocab, x.stride, it.data_ptr(), id_code(Z, ids),
                           scale, k, p(lp), p(lse), p(ent, entropy), p(ti, k > 0), p(tl, k > 0),
                           stream())
    scale = float(np.float32(scale))
    xs = x.host()
    ref = V.token_logprobs(xs, t, scale, k)
    st = sum_tol(vocab)
    big = np.where(np.isfinite(ref["lse"]), np.abs(ref["lse"]), 0)
    # z - mz is formed exactly before its rounding: u times its size; the
    # largest z is rounded once (u |z|), in the sum's exponents as in z - mz
    def lp_tol(v):
        return st + 4 * U * (1 + np.where(np.isfinite(v), np.abs(v), 0))
    close(lse.cpu(), ref["lse"], st + 2 * U * (1 + big))
    close(lp.cpu(), ref["logprob"], lp_tol(ref["logprob"]))
    if entropy:
        h = ref["entropy"]
        close(ent.cpu(), h, st * (2 + 2 * h) + 8 * U * (1 + h))
    else:
        assert bool((ent == 9.0).all())
    if k:
        assert np.array_equal(ti.cpu().numpy(), ref["top_ids"])
        close(tl.cpu(), ref["top_logprobs"], lp_tol(ref["top_logprobs"]))
    assert x.intact()
    return x, t, it, lse, ent, ref


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,vocab,k", [
    (1, 1, 1), (3, 2, 2), (4, 7, 7), (5, 9, 3), (3, 31, 31), (3, 64, 64), (3, 65, 64), (9, 257, 5),
    (2, 600, 64), (7, 1000, 20), (400, 1000, 1), (1, 4099, 64), (3, 8191, 20), (1, 50257, 20),
    (2, 50257, 0), (5, 50257, 64), (170, 9001, 5), (330, 16400, 5), (1, 131077, 64),
])
def test_logprobs(Z, n, vocab, k, dtype):
    logprob_case(Z, n, vocab, dtype, "normal", k, scale=1.0 if n % 2 else 0.7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,vocab,k", [(700, 1003, 0), (607, 1003, 0), (1823, 8193, 2), (1824, 8193, 2),
                                       (1824, 8193, 0), (80, 25001, 3), (38, 12345, 7)])
def test_logprobs_rows_per_warp_block_and_cluster(Z, n, vocab, k, dtype):
    logprob_case(Z, n, vocab, dtype, "masked", k, ids="i32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["ties", "constant", "masked", "lowest", "sorted", "large"])
@pytest.mark.parametrize("n,vocab,k", [(6, 40, 20), (6, 1000, 64), (5, 5000, 20), (4, 50257, 64),
                                       (310, 5003, 6)])
def test_logprobs_distributions(Z, n, vocab, k, dtype, kind):
    logprob_case(Z, n, vocab, dtype, kind, k, ids="i32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pad,off", [(0, 1), (0, 5), (3, 0), (8, 8), (1, 7)])
def test_logprobs_layouts(Z, dtype, pad, off):
    logprob_case(Z, 9, 3001, dtype, "normal", 10, pad, off, scale=1.9)
    logprob_case(Z, 4, 33, dtype, "normal", 0, pad, off, entropy=False)


def test_logprobs_top_in_one_threads_share(Z):
    """The largest logits at a regular distance: any fixed split of a row
    gives them to few threads."""
    for step in (8 * 256, 8 * 128, 8 * 1024, 16384):
        vocab, n = 100003, 2
        x = np.random.default_rng(step).normal(size=(n, vocab))
        x[:, ::step] += 1000
        x[1] = np.round(x[1])
        for shift in range(8):
            x[:, shift::step] += 1000
        xm = Mat(x, torch.float32)
        k = 64
        lp = torch.empty(n, device="cuda")
        ti = torch.empty(n, k, device="cuda", dtype=torch.int32)
        tl = torch.empty(n, k, device="cuda")
        t = ids_tensor([0, 1], "i64")
        Z.zero3_token_logprobs(xm.ptr, Z.F32, n, vocab, vocab, t.data_ptr(), Z.I64, 1.0, k,
                               lp.data_ptr(), None, None, ti.data_ptr(), tl.data_ptr(), stream())
        assert np.array_equal(ti.cpu().numpy(), V.token_logprobs(xm.host(), [0, 1], 1.0, k)["top_ids"])


@pytest.mark.parametrize("vocab", [300, 50257])
def test_logprobs_not_finite(Z, vocab):
    x = np.random.default_rng(0).normal(size=(4, vocab))
    x[0, 5] = np.nan
    x[1, vocab - 1] = np.inf
    x[2, :] = np.nan
    xm = Mat(x, torch.bfloat16)
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    lp, lse, ent, tl = f(4), f(4), f(4), f(4, 3)
    ti = torch.zeros(4, 3, device="cuda", dtype=torch.int32)
    t = ids_tensor([1, 2, -1, 4], "i64")
    Z.zero3_token_logprobs(xm.ptr, Z.BF16, 4, vocab, vocab, t.data_ptr(), Z.I64, 1.0, 3,
                           lp.data_ptr(), lse.data_ptr(), ent.data_ptr(), ti.data_ptr(),
                           tl.data_ptr(), stream())
    assert torch.isnan(lse[:3]).all() and torch.isnan(ent[:3]).all() and torch.isnan(tl[:3]).all()
    assert torch.isnan(lp[:2]).all() and lp[2] == 0 and bool((ti[:3] == -1).all())
    assert torch.isfinite(lp[3]) and bool((ti[3] >= 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [30, 9001])
def test_products_that_overflow_count_as_infinite(Z, vocab, dtype):
    """Masks of the lowest value under a temperature below one: the masked
    tokens have no weight, and a row of them alone is an empty one; logits that
    overflow upwards are infinite."""
    n, K, low = 4, 5, -3.3895313892515355e38
    rng = np.random.default_rng(vocab)
    x = rng.normal(size=(n, vocab))
    x[0] = low
    x[1, 3:] = low
    x[2, 7] = 3e38
    xm = Mat(x, DT[dtype])
    t = [1, 1, 1, 1]
    it = ids_tensor(t, "i64")
    lp, lse, ent = (torch.empty(n, device="cuda") for _ in range(3))
    ti, tl = torch.empty(n, 4, device="cuda", dtype=torch.int32), torch.empty(n, 4, device="cuda")
    Z.zero3_token_logprobs(xm.ptr, code(Z, dtype), n, vocab, vocab, it.data_ptr(), Z.I64, 1.5, 4,
                           lp.data_ptr(), lse.data_ptr(), ent.data_ptr(), ti.data_ptr(),
                           tl.data_ptr(), stream())
    ref = V.token_logprobs(xm.host(), t, 1.5, 4)
    tol = sum_tol(vocab) + 64 * U
    for got, name in ((lp, "logprob"), (lse, "lse"), (tl, "top_logprobs")):
        close(got.cpu(), ref[name], tol)
    h = np.where(np.isnan(ref["lse"]), np.nan, ref["entropy"])
    close(ent.cpu(), h, tol * (2 + 2 * np.where(np.isnan(h), 0, h)))
    assert bool((ti[2] == -1).all())
    keep = [0, 1, 3]
    assert np.array_equal(ti.cpu().numpy()[keep], ref["top_ids"][keep])

    tt = rng.normal(size=(n, K))
    tt[1, 1:] = low
    tt[3] = low  # an empty list
    ids = np.stack([rng.choice(vocab, K, replace=False) for _ in range(n)])
    ids[1] = np.arange(K)
    ids[1, 0] = 2  # a token that the student has not masked
    ids[1, 2] = 0
    tm, idt = Mat(tt, DT[dtype]), ids_tensor(ids, "i32")
    loss, dx = torch.empty(n, device="cuda"), Mat(np.zeros((n, vocab)), DT[dtype])
    Z.zero3_distill_loss(xm.ptr, code(Z, dtype), n, vocab, vocab, tm.ptr, code(Z, dtype), idt.data_ptr(),
                         Z.I32, K, K, 1.5, None, loss.data_ptr(), None, dx.ptr, vocab, stream())
    rl, rdx, _, mag = V.distill(xm.host(), tm.host(), ids, 1.5)
    close(loss.cpu(), rl, np.where(np.isnan(rl), 0, (tol + 64 * U) * (mag + 1)))
    close(dx.host(), rdx, np.where(np.isnan(rdx), 0, 4 * tol + rounding(dtype, rdx)))
    assert loss[0] == 0 and loss[3] == 0 and not dx.host()[[0, 3]].any()


def grad_tol(dtype, ref, p, d, g, h, H, scale):
    """Bound of a logit gradient's error (per element); d = log p."""
    d = np.where(np.isfinite(d), np.abs(d), 0)
    w = np.abs(g)[:, None] + np.abs(h)[:, None] * (d + H[:, None])
    return scale * (p * w * U * (16 + 6 * d) + U * np.abs(g)[:, None] * (p > 0.01)) + \
        rounding(dtype, ref) + 2 * U * np.abs(ref) + 1e-37


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["normal", "masked", "constant"])
@pytest.mark.parametrize("n,vocab,pads,off,which", [
    (1, 1, (0, 0), 0, "both"), (5, 7, (0, 0), 0, "both"), (5, 9, (1, 0), 0, "lp"),
    (7, 1000, (0, 0), 0, "h"), (7, 1001, (0, 0), 3, "both"), (5, 1001, (3, 8), 0, "both"),
    (3, 8193, (0, 0), 0, "lp"), (4, 50257, (0, 0), 0, "both"), (3, 50257, (7, 0), 1, "lp"),
])
def test_logprobs_backward(Z, n, vocab, pads, off, which, dtype, kind):
    scale = 0.7
    x, t, it, lse, ent, ref = logprob_case(Z, n, vocab, dtype, kind, 0, pads[0], off, scale=scale)
    scale = float(np.float32(scale))
    rng = np.random.default_rng(5)
    g, h = rng.normal(size=n), rng.normal(size=n)
    dev = lambda y: torch.as_tensor(y, dtype=torch.float32, device="cuda")  # noqa: E731
    gt, ht = dev(g), dev(h)
    g, h = gt.cpu().double().numpy(), ht.cpu().double().numpy()
    xs = x.host()
    want = V.token_logprobs_backward(xs, t, scale, g if which != "h" else None,
                                     h if which != "lp" else None)
    with np.errstate(invalid="ignore", divide="ignore"):
        logp, _ = V._log_softmax(xs * scale)
        p = np.exp(logp)
    gi = np.where((t >= 0) & (t < vocab), g, 0) * (which != "h")
    tol = grad_tol(dtype, want, p, logp, gi, h * (which != "lp"), ref["entropy"], scale)
    # lse and entropy are inputs here, each with its own error
    eps = sum_tol(vocab) + 2 * U * (1 + np.where(np.isfinite(ref["lse"]), np.abs(ref["lse"]), 0))
    H = ref["entropy"]
    w = np.abs(gi)[:, None] + np.abs(h * (which != "lp"))[:, None] * (
        np.where(np.isfinite(logp), np.abs(logp), 0) + H[:, None] + 1)
    tol = tol + scale * p * w * (4 + H[:, None]) * eps[:, None]
    dp = lambda y, on: y.data_ptr() if on else None  # noqa: E731

    def call(out):
        Z.zero3_token_logprobs_backward(x.ptr, code(Z, dtype), n, vocab, x.stride, it.data_ptr(),
                                        Z.I64, scale, lse.data_ptr(), dp(ent, which != "lp"),
                                        dp(gt, which != "h"), dp(ht, which != "lp"), out.ptr,
                                        out.stride, stream())
    out = Mat(np.full((n, vocab), 3.0), DT[dtype], vocab + pads[1], 0)
    call(out)
    close(out.host(), want, tol)
    assert out.intact() and x.intact()
    first = out.host()
    call(x)  # in place
    assert np.array_equal(x.host(), first) or x.stride % 8 != out.stride % 8 or off % 8 != 0
    close(x.host(), want, tol)
    assert x.intact()


# ------------------------------------------------------------------ distillation
def teacher(rng, n, vocab, K, kind):
    ids = np.stack([rng.choice(vocab, K, replace=K > vocab) for _ in range(n)])
    t = -np.sort(-rng.normal(size=(n, K)) * 4, axis=1)
    if kind == "ragged":
        for i in range(n):
            length = [K, 0, 1, K // 2][i % 4]
            ids[i, length:] = -1
        t[0, K // 2:] = -np.inf
        ids[min(3, n - 1), 0] = vocab
    if kind == "repeated":
        ids = ids % max(1, min(vocab, 3))
    return ids, t


def distill_case(Z, n, vocab, K, dtype, td, kind, xkind="normal", pads=(0, 0), off=0, scale=1.0,
                 ids="i64", tpad=0):
    rng = np.random.default_rng(n + vocab * 3 + K)
    x = Mat(logits(rng, n, vocab, xkind), DT[dtype], vocab + pads[0], off)
    tid, tl = teacher(rng, n, vocab, K, kind)
    tm = Mat(tl, DT[td], K + tpad)
    idt = torch.full((n, K + tpad), 1 << 30, device="cuda",
                     dtype=torch.int32 if ids == "i32" else torch.int64)
    idt[:, :K] = ids_tensor(tid, ids)
    wt = torch.as_tensor(rng.normal(size=n), dtype=torch.float32, device="cuda")
    loss, lse = torch.full((n,), 9.0, device="cuda"), torch.full((n,), 9.0, device="cuda")
    out = Mat(np.full((n, vocab), 3.0), DT[dtype], vocab + pads[1])
    head = (code(Z, dtype), n, vocab, x.stride, tm.ptr, code(Z, td), idt.data_ptr(),
            id_code(Z, ids), K, K + tpad, scale)
    Z.zero3_distill_loss(x.ptr, *head, wt.data_ptr(), loss.data_ptr(), lse.data_ptr(), out.ptr,
                         out.stride, stream())
    scale = float(np.float32(scale))
    w = wt.cpu().double().numpy()
    xs, ts = x.host(), tm.host()
    rl, rdx, rlse, mag = V.distill(xs, ts, tid, scale, w)
    st = sum_tol(vocab)
    with np.errstate(invalid="ignore", divide="ignore"):
        logp, _ = V._log_softmax(xs * scale)
        p = np.exp(logp)
    d = np.where(np.isfinite(logp), np.abs(logp), 0)
    big = np.where(np.isfinite(rlse), np.abs(rlse), 0)
    # q: its sum (K additions at most), exponentials, one division
    qe = U * (2 * K + 32)
    ltol = (qe + st) * (mag + 1 / scale ** 2) + 16 * U * mag + 1e-30
    close(loss.cpu(), rl, np.where(np.isfinite(ltol), ltol, 0))
    close(lse.cpu(), rlse, st + 2 * U * (1 + big))
    q = np.zeros_like(xs)
    qk, _, _ = V.teacher_probabilities(ts, tid, scale, vocab)
    for i in range(n):
        for k in range(K):
            if qk[i, k] > 0:
                q[i, tid[i, k]] += qk[i, k]
    wa = np.abs(w / scale)[:, None]
    gtol = wa * (p * (2 * st + U * (16 + 6 * d)) + q * qe * 2) + rounding(dtype, rdx) + 1e-37
    close(out.host(), rdx, gtol)
    assert out.intact() and x.intact()
    first = out.host()

    # the loss alone, and without the optional output
    l2 = torch.empty(n, device="cuda")
    Z.zero3_distill_loss(x.ptr, *head, None, l2.data_ptr(), None, None, 0, stream())
    close(l2.cpu(), rl, np.where(np.isfinite(ltol), ltol, 0))
    # the gradient alone
    gtol = gtol + wa * p * (st + 4 * U * (1 + big))[:, None]
    out.t.fill_(4.0)
    Z.zero3_distill_backward(x.ptr, *head, lse.data_ptr(), wt.data_ptr(), out.ptr, out.stride,
                             stream())
    close(out.host(), rdx, gtol)
    assert out.intact()
    # unit weights
    out.t.fill_(4.0)
    Z.zero3_distill_backward(x.ptr, *head, lse.data_ptr(), None, out.ptr, out.stride, stream())
    r1 = V.distill(xs, ts, tid, scale)[1]
    close(out.host(), r1, (gtol - rounding(dtype, rdx)) / np.maximum(np.abs(w)[:, None], 1e-9) +
          rounding(dtype, r1) + 1e-37)
    # in place: the gradient alone, then both
    keep = x.t.clone()
    Z.zero3_distill_backward(x.ptr, *head, lse.data_ptr(), wt.data_ptr(), x.ptr, x.stride, stream())
    close(x.host(), rdx, gtol)
    x.t.copy_(keep)
    Z.zero3_distill_loss(x.ptr, *head, wt.data_ptr(), loss.data_ptr(), lse.data_ptr(), x.ptr,
                         x.stride, stream())
    close(x.host(), rdx, gtol)
    assert x.intact()
    if off % 8 == 0 and (n == 1 or (pads[0] - pads[1]) % 8 == 0):
        assert np.array_equal(x.host(), first)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,vocab,K,kind", [
    (1, 1, 1, "plain"), (3, 2, 2, "plain"), (4, 7, 3, "ragged"), (5, 9, 9, "repeated"),
    (4, 1000, 20, "ragged"), (4, 1001, 64, "repeated"), (3, 5000, 300, "plain"),
    (2, 3000, 1024, "repeated"), (1, 50257, 64, "plain"), (4, 50257, 100, "ragged"),
    (320, 2003, 8, "ragged"), (1, 131077, 32, "repeated"),
])
def test_distill(Z, n, vocab, K, kind, dtype):
    distill_case(Z, n, vocab, K, dtype, "f32" if K % 2 else dtype, kind,
                 scale=1.0 if n % 2 else 0.5, ids="i32" if n % 3 else "i64", tpad=n % 4)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,vocab,K,kind", [
    (3, 4096, 33, "repeated"), (3, 8192, 5, "ragged"), (37, 8193, 40, "plain"), (2, 12001, 64, "repeated"),
    (150, 10240, 9, "ragged"), (160, 10241, 9, "plain"), (3, 20480, 31, "plain"), (2, 20481, 70, "ragged"),
])
def test_distill_rows_per_block_and_cluster(Z, n, vocab, K, kind, dtype):
    distill_case(Z, n, vocab, K, dtype, dtype, kind, "masked", scale=0.9)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("xkind", ["constant", "masked", "lowest", "large", "ties"])
def test_distill_distributions(Z, dtype, xkind):
    distill_case(Z, 5, 1003, 16, dtype, "bf16", "ragged", xkind)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pads,off", [((0, 0), 1), ((3, 0), 0), ((8, 16), 8), ((1, 1), 0), ((5, 2), 3)])
def test_distill_layouts(Z, dtype, pads, off):
    distill_case(Z, 5, 3001, 10, dtype, "f32", "ragged", pads=pads, off=off, scale=0.8)


def test_distill_nan_stays_in_its_row(Z):
    n, vocab, K = 4, 500, 6
    rng = np.random.default_rng(3)
    x, t = rng.normal(size=(n, vocab)), rng.normal(size=(n, K))
    x[0, 77] = np.nan
    t[1, 2] = np.nan
    ids = np.stack([rng.choice(vocab, K, replace=False) for _ in range(n)])
    xm, tm, it = Mat(x, torch.float32), Mat(t, torch.float32), ids_tensor(ids, "i64")
    loss, lse = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    dx = torch.zeros(n, vocab, device="cuda")
    head = (Z.F32, n, vocab, vocab, tm.ptr, Z.F32, it.data_ptr(), Z.I64, K, K, 1.0)
    Z.zero3_distill_loss(xm.ptr, *head, None, loss.data_ptr(), lse.data_ptr(), dx.data_ptr(), vocab,
                         stream())
    assert torch.isnan(loss[:2]).all() and torch.isfinite(loss[2:]).all()
    assert torch.isnan(dx[:2]).all() and torch.isfinite(dx[2:]).all()
    dx.zero_()
    Z.zero3_distill_backward(xm.ptr, *head, lse.data_ptr(), None, dx.data_ptr(), vocab, stream())
    assert torch.isnan(dx[:2]).all() and torch.isfinite(dx[2:]).all()


# ------------------------------------------------------- streams, graphs, sizes
def test_streams_and_graph(Z):
    """Every call on a side stream, behind and ahead of other kernels without
    synchronisation, then replayed from a graph with new inputs."""
    n, vocab, dim, K = 64, 5003, 256, 8
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(0)
    ids = torch.randint(0, vocab, (n,), generator=g, device=dev)
    table = torch.empty(vocab, dim, device=dev)
    x = torch.empty(n, vocab, device=dev)
    tid = torch.randint(0, vocab, (n, K), generator=g, device=dev)
    tl = torch.randn(n, K, generator=g, device=dev)
    emb, gt = torch.empty(n, dim, device=dev), torch.empty(vocab, dim, device=dev)
    lp, lse, ent, loss = (torch.empty(n, device=dev) for _ in range(4))
    dx1, dx2 = torch.empty_like(x), torch.empty_like(x)
    ti = torch.empty(n, 4, device=dev, dtype=torch.int32)
    tp = torch.empty(n, 4, device=dev)
    ws = torch.empty(Z.zero3_embedding_workspace(n, vocab, dim), device=dev, dtype=torch.uint8)
    src_t, src_x = torch.empty_like(table), torch.empty_like(x)
    outs = [emb, gt, lp, lse, ent, ti, tp, loss, dx1, dx2]
    copies = [torch.empty_like(o) for o in outs]

    def calls():
        s = stream()
        table.copy_(src_t)
        x.copy_(src_x)
        Z.zero3_embedding_forward(table.data_ptr(), Z.F32, vocab, dim, dim, ids.data_ptr(), Z.I64, n,
                                  2.0, emb.data_ptr(), Z.F32, dim, s)
        Z.zero3_embedding_backward(emb.data_ptr(), Z.F32, dim, ids.data_ptr(), Z.I64, n, 1.0, 0,
                                   gt.data_ptr(), Z.F32, vocab, dim, dim, ws.data_ptr(), ws.numel(), s)
        Z.zero3_token_logprobs(x.data_ptr(), Z.F32, n, vocab, vocab, ids.data_ptr(), Z.I64, 1.0, 4,
                               lp.data_ptr(), lse.data_ptr(), ent.data_ptr(), ti.data_ptr(),
                               tp.data_ptr(), s)
        Z.zero3_token_logprobs_backward(x.data_ptr(), Z.F32, n, vocab, vocab, ids.data_ptr(), Z.I64,
                                        1.0, lse.data_ptr(), ent.data_ptr(), lp.data_ptr(),
                                        ent.data_ptr(), dx1.data_ptr(), vocab, s)
        Z.zero3_distill_loss(x.data_ptr(), Z.F32, n, vocab, vocab, tl.data_ptr(), Z.F32,
                             tid.data_ptr(), Z.I64, K, K, 1.0, lse.data_ptr(), loss.data_ptr(), None,
                             dx2.data_ptr(), vocab, s)
        for c, o in zip(copies, outs):
            c.copy_(o)

    def fill(seed):
        h = torch.Generator(dev).manual_seed(seed)
        src_t.copy_(torch.randn(vocab, dim, generator=h, device=dev))
        src_x.copy_(torch.randn(n, vocab, generator=h, device=dev))

    def expect(seed):
        fill(seed)
        torch.cuda.synchronize()
        calls()
        torch.cuda.synchronize()
        return [c.clone() for c in copies]

    want = {s: expect(s) for s in (1, 2, 3)}
    xs = src_x.double().cpu().numpy()
    ref = V.token_logprobs(xs, ids.cpu().numpy(), 1.0)
    close(want[3][2].cpu(), ref["logprob"], sum_tol(vocab) + 4 * U * (1 + np.abs(ref["logprob"])))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fill(1)
        calls()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want[1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed in (2, 3):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(copies, want[seed]))


def test_rows_beyond_32_bit_offsets(Z):
    """Logits and tables of more than 2^32 elements: the last rows are
    addressed with 64-bit offsets."""
    vocab, stride = 1003, 1 << 22
    n = 1100  # 4.6e9 elements of bf16
    buf = torch.zeros(n * stride, device="cuda", dtype=torch.bfloat16)
    x = torch.as_strided(buf, (n, vocab), (stride, 1))
    g = torch.Generator("cuda").manual_seed(1)
    x.copy_(torch.randn(n, vocab, generator=g, device="cuda"))
    rows = [0, 1, 1023, 1024, n - 1]
    xs = x[rows].double().cpu().numpy()
    t = torch.randint(0, vocab, (n,), generator=g, device="cuda")
    lp, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    Z.zero3_token_logprobs(buf.data_ptr(), Z.BF16, n, vocab, stride, t.data_ptr(), Z.I64, 1.0, 0,
                           lp.data_ptr(), lse.data_ptr(), stream=stream())
    ref = V.token_logprobs(xs, t[rows].cpu().numpy(), 1.0)
    close(lp[rows].cpu(), ref["logprob"], sum_tol(vocab) + 4 * U * (1 + np.abs(ref["logprob"])))
    one = torch.ones(n, device="cuda")
    Z.zero3_token_logprobs_backward(buf.data_ptr(), Z.BF16, n, vocab, stride, t.data_ptr(), Z.I64,
                                    1.0, lse.data_ptr(), 0, one.data_ptr(), 0, buf.data_ptr(),
                                    stride, stream())
    want = V.token_logprobs_backward(xs, t[rows].cpu().numpy(), 1.0, np.ones(len(rows)))
    close(x[rows].double().cpu().numpy(), want, 2.0 ** -8 * np.abs(want) + 40 * U)
    # the same memory as a table: rows 0 and n - 1 looked up and updated
    ids = torch.tensor([n - 1, 0, n - 1], device="cuda")
    out = torch.empty(3, vocab, device="cuda")
    x.copy_(torch.randn(n, vocab, generator=g, device="cuda"))
    Z.zero3_embedding_forward(buf.data_ptr(), Z.BF16, n, vocab, stride, ids.data_ptr(), Z.I64, 3, 1.0,
                              out.data_ptr(), Z.F32, vocab, stream())
    assert torch.equal(out, x[ids].float())
    old = x[[n - 1, 0, 5]].float()
    ws = torch.empty(Z.zero3_embedding_workspace(3, n, vocab), device="cuda", dtype=torch.uint8)
    Z.zero3_embedding_backward(out.data_ptr(), Z.F32, vocab, ids.data_ptr(), Z.I64, 3, 1.0, 1,
                               buf.data_ptr(), Z.BF16, n, vocab, stride, ws.data_ptr(), ws.numel(),
                               stream())
    assert torch.equal(x[n - 1].float(), (old[0] + (out[0] + out[2])).bfloat16().float())
    assert torch.equal(x[0].float(), (old[1] + out[1]).bfloat16().float())
    assert torch.equal(x[5].float(), old[2])
    assert bool((buf.view(n, stride)[:, vocab:] == 0).all())
