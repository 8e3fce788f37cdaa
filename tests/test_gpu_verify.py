"""Verification of drafted tokens on the GPU against the 64-bit definition.

Accepted counts and tokens have to be equal: the library decides as exact
arithmetic on the given numbers does, to about 1e-9 relative.  Log probabilities:
z - max rounds once (2^-24 of it), the logarithm of the sum is off by 2^-23 of
itself and by the sum's relative error, which 2^-17 + (chain of additions) * 2^-24
bounds: below 1.3e-5 at these sizes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import verify_oracle as VO  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def z(lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from zero_sharded_optimizer_shard_gb300 import zero3
    return zero3


def rows(x, dt, pad=0, shift=0):
    """Device rows of x [..., V] with `pad` elements between them, `shift` elements
    behind a 16-byte boundary; (tensor view [rows, V], stride)."""
    r = torch.as_tensor(x).reshape(-1, x.shape[-1])
    V = r.shape[1]
    base = torch.full((shift + r.shape[0] * (V + pad) + 8,), float("nan"), dtype=dt, device="cuda")
    v = base[shift:shift + r.shape[0] * (V + pad)].view(r.shape[0], V + pad)[:, :V]
    v.copy_(r.to(dt))
    return v, V + pad


class Case:
    def __init__(self, n, k, V, dtype="f32", draft="f32", ids=torch.int64, scale=1.0, draft_scale=1.0,
                 pad=0, shift=0, seed=0, spread=2.5, likeness=0.6):
        g = torch.Generator().manual_seed(seed * 7919 + V * 31 + k)
        r = lambda *a: torch.randn(*a, generator=g)  # noqa: E731
        self.n, self.k, self.V, self.ids_type = n, k, V, ids
        self.scale, self.draft_scale, self.pad, self.shift = scale, draft_scale, pad, shift
        self.x = (r(n, k + 1, V) * spread).to(DT[dtype])
        near = self.x[:, :k].float() + likeness * r(n, k, V)
        self.y = near.to(DT[draft]) if draft else None
        e = torch.empty(n, k, V).exponential_(generator=g)
        self.ids = (near * draft_scale - torch.log(e)).argmax(2) if k else torch.zeros(n, 0, dtype=torch.int64)
        self.u = torch.rand(n, k, generator=g)
        self.noise = torch.empty(n, V).exponential_(generator=g)

    def run(self, z, check=True, tol=1.3e-5):
        n, k, V = self.n, self.k, self.V
        x, sx = rows(self.x, self.x.dtype, self.pad, self.shift)
        y, sy = rows(self.y, self.y.dtype, self.pad, self.shift) if self.y is not None and k else (None, V)
        e, se = rows(self.noise, torch.float32, self.pad, self.shift)
        ids, u = self.ids.to(self.ids_type).cuda(), self.u.cuda()
        out = torch.full((2, n + 2, k + 1), -7, dtype=torch.int32, device="cuda")
        acc, tok = out[0].view(-1)[1:n + 1], out[1].view(-1)[k + 1:k + 1 + n * (k + 1)]
        lps = torch.full((n * (k + 1) + 2,), -7.0, device="cuda")
        code = lambda t: z.BF16 if t.dtype == torch.bfloat16 else z.F32  # noqa: E731
        z.zero3_verify_draft(x.data_ptr(), code(x), n, k, V, sx, y.data_ptr() if y is not None else 0,
                             code(y) if y is not None else 0, sy, ids.data_ptr() if k else 0,
                             z.I64 if self.ids_type == torch.int64 else z.I32, self.scale,
                             self.draft_scale, u.data_ptr() if k else 0, e.data_ptr(), se,
                             acc.data_ptr(), tok.data_ptr(), lps[1:].data_ptr(),
                             torch.cuda.current_stream().cuda_stream)
        got = acc.cpu().numpy(), tok.view(n, k + 1).cpu().numpy(), lps[1:-1].view(n, k + 1).cpu().numpy()
        assert float(lps[0]) == -7 and float(lps[-1]) == -7
        assert int((out[0] != -7).sum()) <= n
        if check:
            want = self.want()
            np.testing.assert_array_equal(got[0], want[0])
            np.testing.assert_array_equal(got[1], want[1])
            w = want[2]
            fin = np.isfinite(w)
            np.testing.assert_array_equal(got[2][~fin], w[~fin].astype(np.float32))
            assert np.all(np.abs(got[2][fin] - w[fin]) <= tol + 2.0 ** -21 * np.abs(w[fin]))
        return got

    def want(self):
        f = lambda t: t.double().numpy()  # noqa: E731
        s = lambda v: float(np.float32(v))  # noqa: E731
        return VO.verify(f(self.x), f(self.y) if self.y is not None else None, self.ids.numpy(), f(self.u),
                         f(self.noise), s(self.scale), s(self.draft_scale))


@pytest.mark.parametrize("draft", ["same", None])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k,V", [(1, 0, 1), (1, 1, 1), (3, 2, 2), (2, 3, 7), (5, 4, 33), (40, 1, 257),
                                   (1, 4, 50257), (7, 8, 4097), (2, 17, 1000), (20, 5, 3001),
                                   (80, 2, 1031), (160, 3, 999), (400, 2, 131)])
def test_against_the_definition(z, n, k, V, dtype, draft):
    """Every cluster size (1 to 8 blocks) and number of positions per round."""
    Case(n, k, V, dtype, dtype if draft else None, scale=1.25 if n % 2 else 1.0,
         draft_scale=1.25 if n % 2 else 0.8).run(z)


@pytest.mark.parametrize("dtype,draft", [("bf16", "f32"), ("f32", "bf16")])
def test_types_that_differ(z, dtype, draft):
    Case(9, 3, 2049, dtype, draft, ids=torch.int32, seed=1).run(z)


@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1), (3, 5), (8, 7)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_alignment(z, pad, shift, dtype):
    for n, draft in ((3, dtype), (50, dtype), (3, None)):
        Case(n, 3, 1500, dtype, draft, pad=pad, shift=shift, seed=2).run(z)


def test_long_drafts(z):
    """The longest draft, accepted to the end, to the middle, and not at all."""
    c = Case(6, 256, 40, "f32", "f32", seed=3, likeness=0.0)
    c.u.mul_(0.999)
    c.u[1, 100], c.ids[1, 100] = 1.0, 5
    c.x[1, 100, 5] = -30.0
    c.ids[2, 0] = -1
    c.ids[3, 31], c.ids[4, 32], c.ids[5, 255] = 40, -9, 1 << 40
    got = c.run(z)
    assert got[0].tolist() == [256, 100, 0, 31, 32, 255]


@pytest.mark.parametrize("draft", ["f32", None])
def test_acceptance_at_the_border(z, draft):
    """Uniform numbers next to p / q, on both sides of it, at a distance that
    binary32 sums do not resolve."""
    n, V = 200, 2003
    c = Case(n, 1, V, "f32", draft, seed=4)
    p = np.stack([VO._row(c.x[s, 0].double().numpy()) for s in range(n)])
    d = c.ids[:, 0].numpy()
    lp = p[np.arange(n), d]
    if draft:
        q = np.stack([VO._row(c.y[s, 0].double().numpy()) for s in range(n)])
        lp = lp - q[np.arange(n), d]
    ratio = np.exp(lp)
    below = ratio.astype(np.float32)
    below = np.where(below.astype(np.float64) >= ratio, np.nextafter(below, np.float32(0)), below)
    above = np.nextafter(below, np.float32(2))
    u = np.where(np.arange(n) % 2 == 0, below, above)
    far = np.abs(u.astype(np.float64) / ratio - 1) > 4e-9
    assert far.sum() > 150
    u = np.where(far, u, np.float32(0.5))
    c.u[:, 0] = torch.from_numpy(u)
    got = c.run(z)
    np.testing.assert_array_equal(got[0][far], u[far].astype(np.float64) < ratio[far])


@pytest.mark.parametrize("k,draft", [(0, None), (1, "f32"), (1, None)])
@pytest.mark.parametrize("V", [300, 20011])
def test_races_that_are_nearly_tied(z, V, k, draft):
    """The noise of one more token is set so that its score lies one binary32 step
    of the noise beside the winner's, on either side."""
    n = 48
    c = Case(n, k, V, "f32", draft, seed=5)
    if k:
        c.u[:] = 0.99999994
        c.ids[:, 0] = c.ids[:, 0]
        at = torch.arange(n)
        c.x[at, 0, c.ids[:, 0]] = -20.0  # refused
    for s in range(n):
        p = np.exp(VO._row(c.x[s, 0].double().numpy()))
        r = p
        if k and draft:
            r = p - np.exp(VO._row(c.y[s, 0].double().numpy()))
        elif k:
            r = np.where(np.arange(V) == int(c.ids[s, 0]), 0, p)
        e = c.noise[s].double().numpy()
        win = int(np.argmax(np.where(r > 0, r / e, 0)))
        order = np.argsort(-r)
        other = int(order[1] if order[0] == win else order[0])
        tie = r[other] * e[win] / r[win]
        f = np.float32(tie)
        c.noise[s, other] = float(np.nextafter(f, np.float32(0)) if s % 2 else np.nextafter(f, np.float32(1e30)))
        gap = abs(r[other] / float(c.noise[s, other]) / (r[win] / e[win]) - 1)
        if gap < 4e-9 * (1 + p[other] / r[other] + p[win] / r[win]):
            c.noise[s, other] = 100.0
    c.run(z)


def test_equal_scores_go_to_the_lowest_token(z):
    for n in (2, 200):
        c = Case(n, 1, 999, "f32", "f32", seed=6)
        c.x[:] = 0.0
        c.y[:] = 0.0
        c.x[:, 0, ::3] = 1.0
        c.y[:, 0, ::3] = 0.5
        c.ids[:, 0] = 1
        c.u[:] = 0.999
        c.noise[:] = 2.0
        got = c.run(z)
        assert (got[0] == 0).all() and (got[1][:, 0] == 0).all()
        c.noise[:, :500] = 4.0
        assert (c.run(z)[1][:, 0] == 501).all()
        c.noise[:, 700] = 0.0   # no residual there
        c.noise[:, 702] = 0.0
        c.noise[:, 705] = 0.0
        assert (c.run(z)[1][:, 0] == 702).all()


def test_noise_that_excludes(z):
    c = Case(12, 0, 500, "bf16", None, seed=7)
    c.noise[0] = -1.0
    c.noise[1] = float("nan")
    c.noise[2] = float("inf")
    c.noise[3, :499] = float("nan")
    c.noise[4] = 3e38
    c.noise[5] = 1e-40
    c.noise[6, 77] = 1e-44
    c.noise[7, ::2] = -0.0
    c.noise[8, 100:] = float("inf")
    got = c.run(z)
    assert got[1][:3, 0].tolist() == [-1, -1, -1] and got[1][3, 0] == 499


@pytest.mark.parametrize("n", [6, 330])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masks_and_rows_without_tokens(z, n, dtype):
    c = Case(n, 3, 1201, dtype, dtype, seed=8)
    inf = float("inf")
    keep = torch.rand(n, 4, 1201, generator=torch.Generator().manual_seed(1)) < 0.02
    c.x[::2] = torch.where(keep[::2], c.x[::2].float(), torch.tensor(-inf)).to(c.x.dtype)
    c.x[1, 0] = -inf
    c.x[3, 1] = -inf
    c.y[4, 0] = -inf
    c.y[5, 1] = torch.finfo(c.y.dtype).min
    c.x[5, 2] = torch.finfo(c.x.dtype).min  # finite, all equal
    c.ids[5, 0] = -1
    c.run(z)


def test_rows_that_are_not_finite(z):
    inf, nan = float("inf"), float("nan")
    for n in (8, 330):
        c = Case(n, 2, 777, "f32", "f32", seed=9)
        c.u[:] = 0.0   # everything that can be accepted is
        c.x[0, 0, 5] = nan
        c.x[1, 1, 776] = inf
        c.x[2, 2, 0] = nan
        c.y[3, 0, 3] = nan
        c.y[4, 1, 700] = inf
        c.x[5, 0, 9] = 3e38
        c.u[6, 0] = nan
        got = c.run(z, check=False)
        want = c.want()
        keep = np.arange(n) != 6
        for a, b in zip(got[:2], want[:2]):
            np.testing.assert_array_equal(a[keep], b[keep])
        np.testing.assert_array_equal(np.isnan(got[2][keep]), np.isnan(want[2][keep]))
        assert got[0][:5].tolist() == [0, 1, 2, 0, 1] and got[0][6] == 0 and got[1][6, 0] >= 0


def test_probabilities_far_below_binary32(z):
    """Tokens thousands of units below the row's largest, in both rows: the
    logarithms decide."""
    c = Case(40, 1, 300, "f32", "f32", seed=12)
    at = torch.arange(40)
    c.ids[:, 0] = 17
    c.x[:, 0, 17] = -4000.0 - 0.125 * at
    c.y[:, 0, 17] = -4002.0
    c.x[30:, 0, 3] = 3e38
    c.y[30:, 0, 3] = 3e38
    c.x[30:35, 0, 17] = -3e37
    got = c.run(z)
    assert 0 < got[0].sum() < 40


@pytest.mark.parametrize("unit", [1e-35, 1e30])
@pytest.mark.parametrize("draft", ["f32", None])
def test_logits_in_other_units(z, unit, draft):
    """Tiny logits under a huge inverse temperature, and the other way round."""
    c = Case(30, 2, 1200, "f32", draft, seed=13, scale=1 / unit, draft_scale=1 / unit)
    c.x = (c.x.double() * unit).float()
    c.ids = c.ids % 1200
    if draft:
        c.y = (c.y.double() * unit).float()
        c.ids[:] = c.y.argmax(2)
    c.run(z)


def test_a_draft_equal_to_the_target(z):
    """Accepted at every u below 1; at u = 1 there is no residual and the draw is
    from the target."""
    for n in (4, 320):
        c = Case(n, 2, 1500, "bf16", "bf16", seed=10, likeness=0.0)
        c.y.copy_(c.x[:, :2])
        c.u[:] = 0.99999994
        assert (c.run(z)[0] == 2).all()
        c.u[:] = 1.0
        got = c.run(z)
        assert (got[0] == 0).all() and (got[1][:, 0] >= 0).all()


def test_the_same_draw_over_again_and_in_a_graph(z):
    c = Case(64, 4, 5003, "bf16", "bf16", seed=11)
    first = c.run(z)
    x, sx = rows(c.x, c.x.dtype)
    y, sy = rows(c.y, c.y.dtype)
    e, se = rows(c.noise, torch.float32)
    ids, u = c.ids.cuda(), c.u.cuda()
    acc = torch.empty(64, dtype=torch.int32, device="cuda")
    tok = torch.empty(64, 5, dtype=torch.int32, device="cuda")
    call = lambda: z.zero3_verify_draft(  # noqa: E731
        x.data_ptr(), z.BF16, 64, 4, 5003, sx, y.data_ptr(), z.BF16, sy, ids.data_ptr(), z.I64, 1.0, 1.0,
        u.data_ptr(), e.data_ptr(), se, acc.data_ptr(), tok.data_ptr(), 0,
        torch.cuda.current_stream().cuda_stream)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(2):
        acc.fill_(-3)
        tok.fill_(-3)
        g.replay()
        np.testing.assert_array_equal(acc.cpu().numpy(), first[0])
        np.testing.assert_array_equal(tok.cpu().numpy(), first[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,V", [(1, 1), (2, 7), (3, 9), (1, 50257), (5, 4099), (33, 1025), (70, 2050),
                                 (140, 8191), (300, 1537), (700, 515)])
def test_sampling(z, n, V, dtype):
    """Without a draft, at every cluster size."""
    Case(n, 0, V, dtype, None, scale=1.25 if n % 2 else 0.8, seed=20).run(z)


@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1), (3, 5), (8, 7), (2, 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sampling_strides_and_alignment(z, pad, shift, dtype):
    for n in (3, 40, 310):
        Case(n, 0, 2500, dtype, None, pad=pad, shift=shift, seed=21).run(z)


@pytest.mark.parametrize("n", [1, 20, 320])
def test_sampling_where_the_largest_logits_come_late(z, n):
    """Rows that rise by 200, 60 and 30 over the row, that rise at the last element, that
    begin with masked tokens or hold one token only."""
    c = Case(n, 0, 20011, "f32", None, seed=22)
    at = torch.arange(20011) / 20010.0
    for s in range(n):
        c.x[s, 0] += at * (200.0, 60.0, 30.0, 0.0, -60.0, -200.0)[s % 6]
        if s % 7 == 1:
            c.x[s, 0, -1] += 150.0
        if s % 5 == 2:
            c.x[s, 0, :19000] = -float("inf")
        if s % 11 == 3:
            c.x[s, 0, torch.arange(20011) != 20010 - s] = -float("inf")
    c.run(z)


def test_sampling_against_noise_of_all_sizes(z):
    """Noise from 1e-37 to 1e38, which moves the winner to unlikely tokens."""
    c = Case(64, 0, 3001, "f32", None, seed=23)
    g = torch.Generator().manual_seed(24)
    c.noise = torch.exp2(torch.rand(64, 3001, generator=g) * 250 - 123)
    c.run(z)


def test_sampling_of_equal_scores(z):
    c = Case(50, 0, 4001, "bf16", None, seed=25)
    c.x[:, 0] = 1.0
    c.noise[:] = 0.5
    c.noise[:, :100] = 2.0
    assert (c.run(z)[1][:, 0] == 100).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sampling_rows_that_are_not_finite(z, dtype):
    c = Case(8, 0, 5000, dtype, None, seed=26)
    c.x[0, 0, 4999] = float("nan")
    c.x[1, 0, 0] = float("inf")
    c.x[2, 0] = float("nan")
    c.x[3, 0] = -float("inf")
    c.x[4, 0] = torch.finfo(c.x.dtype).min
    c.x[5, 0, 1::2] = torch.finfo(c.x.dtype).min
    c.run(z)
