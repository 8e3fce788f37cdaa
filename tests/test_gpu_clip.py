"""Gradient norms, clipping and the clipped step on the GPU, against 64-bit sums
and the oracle's step.

Norms: a sum of m squares whose longest chain of binary32 roundings has d of them
is off by at most d * 2^-24 of itself (all terms are positive), its root by half
of that, plus 2^-24 where it is stored.  Lists: a thread adds at most per / 256
products (per = 1024 chunks up to 4864 * 8192 elements), then 4 + 5 sums: d <= 16
here.  Reduced gradients: 8 squares, 5 sums: d <= 13, on top of the reduced
gradient itself, which the oracle gives bit for bit."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle as O  # noqa: E402
from oracle import clip_oracle as CO  # noqa: E402
from tests._oracle_runs import bits, f32, host_grads, host_master, host_pgrads, u16  # noqa: E402
from zero_sharded_optimizer_shard_gb300 import workloads as W  # noqa: E402

pytestmark = pytest.mark.gpu
NORM_TOL = 9 * 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def z(lib):
    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for -m gpu tests")
    from zero_sharded_optimizer_shard_gb300 import zero3
    return zero3


def code(z, dt):
    return z.BF16 if dt == torch.bfloat16 else z.F32


def sid():
    return torch.cuda.current_stream().cuda_stream


class Buffers:
    """Tensors of the given sizes at the given element offsets from 16-byte
    boundaries in one guarded buffer (gaps hold a sentinel)."""
    SENTINEL = 7.0

    def __init__(self, sizes, offsets, dtype):
        starts, at = [], 16
        for n, o in zip(sizes, offsets):
            at = (at + 7) // 8 * 8 + o
            starts.append(at)
            at += n
        self.base = torch.full((at + 16,), self.SENTINEL, dtype=dtype, device="cuda")
        self.tensors = [self.base[s:s + n] for s, n in zip(starts, sizes)]
        self.mask = torch.ones(at + 16, dtype=torch.bool, device="cuda")
        for s, n in zip(starts, sizes):
            self.mask[s:s + n] = False

    def list(self, z):
        return z.TensorList([t.data_ptr() if t.numel() else 0 for t in self.tensors],
                            [t.numel() for t in self.tensors], code(z, self.base.dtype))

    def untouched(self):
        return bool((self.base[self.mask] == self.SENTINEL).all())


def fill(b, seed, scale=1e-3):
    g = torch.Generator().manual_seed(seed)
    for t in b.tensors:
        t.copy_(torch.randn(t.numel(), generator=g) * scale)
    return b


def norm(z, tl, max_norm, tensor_norms=True):
    ws = torch.empty(z.zero3_grad_norm_workspace(tl), dtype=torch.uint8, device="cuda")
    tn = torch.full((max(tl.n, 1),), -1.0, device="cuda") if tensor_norms else None
    sq = torch.full((1,), -1.0, dtype=torch.float64, device="cuda")
    out = torch.full((2,), -1.0, device="cuda")
    z.zero3_grad_norm(tl, max_norm, tn.data_ptr() if tn is not None else 0, sq.data_ptr(),
                      out.data_ptr(), out[1:].data_ptr(), ws.data_ptr(), ws.numel(), sid())
    return (tn[:tl.n].cpu().numpy() if tn is not None else None), float(sq), *out.cpu().tolist()


def want(b, max_norm):
    xs = [t.double().cpu().numpy() for t in b.tensors]
    s = CO.square_sum(xs)
    return [np.sqrt(CO.square_sum([x])) for x in xs], s, np.sqrt(s), CO.clip_coefficient(s, max_norm)


SIZES = {
    "one": [1],
    "empty": [0, 5, 0, 0, 8191, 0],
    "odd": [1, 7, 8, 9, 15, 17, 8192, 8193, 16384 + 5, 100_003, 262_144 + 3],
    "many": [(i * 37) % 41 for i in range(2100)],          # three launches
    "tiles": [40_000, 1, 1_000_001, 65_537],
}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("sizes", list(SIZES))
def test_norms_of_lists(z, sizes, dtype):
    n = SIZES[sizes]
    b = fill(Buffers(n, [(3 * i + 1) % 8 for i in range(len(n))], DT[dtype]), 1)
    tn, sq, total, coef = norm(z, b.list(z), 0.01)
    wtn, wsq, wtotal, wcoef = want(b, 0.01)
    assert np.all(np.abs(tn - wtn) <= NORM_TOL * np.asarray(wtn))
    assert abs(sq - wsq) <= 2 * NORM_TOL * wsq
    assert abs(total - wtotal) <= NORM_TOL * wtotal
    assert abs(coef - wcoef) <= NORM_TOL * wcoef
    assert b.untouched()


def test_norm_of_twenty_thousand_tensors(z):
    """More blocks than one block joins: the sums are folded first."""
    n = [1 + i % 3 for i in range(20_000)]
    x = torch.randn(sum(n), generator=torch.Generator().manual_seed(2)).cuda()
    ts = list(x.split(n))
    tl = z.TensorList([t.data_ptr() for t in ts], n, z.F32)
    tn, sq, total, _ = norm(z, tl, 1.0)
    ref = x.double().cpu().numpy() ** 2
    each = np.sqrt(np.add.reduceat(ref, np.cumsum([0] + n[:-1])))
    assert np.all(np.abs(tn - each) <= NORM_TOL * each)
    assert abs(total - np.sqrt(ref.sum())) <= NORM_TOL * total


def test_norm_of_a_large_tensor(z):
    """Blocks of more than 1024 chunks: 60e6 elements give two units per block,
    8 more products in a thread's chain."""
    x = torch.randn(60_000_001, generator=torch.Generator("cuda").manual_seed(3), device="cuda") \
        .to(torch.bfloat16)
    tl = z.TensorList([x[1:].data_ptr()], [x.numel() - 1], z.BF16)
    ref = float(x[1:].double().square().sum().sqrt())
    for _ in range(2):
        _, _, total, coef = norm(z, tl, 1.0, tensor_norms=False)
        assert abs(total - ref) <= 2 * NORM_TOL * ref
    assert abs(coef - 1.0 / (ref + 1e-6)) <= 2 * NORM_TOL


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [1e30, 1e19, 3e-20, 1e-30, 1e-39])
def test_norm_beyond_the_range_of_squares(z, dtype, value):
    b = Buffers([5000, 33], [0, 3], DT[dtype])
    g = torch.Generator().manual_seed(4)
    for t in b.tensors:  # near `value`: small integers times it, exact enough in 64 bits
        t.copy_(torch.randn(t.numel(), generator=g).double() * value)
    b.tensors[0][:100] = 0
    tn, sq, total, coef = norm(z, b.list(z), 1.0)
    wtn, wsq, wtotal, wcoef = want(b, 1.0)
    assert wtotal > 0
    tol = NORM_TOL + (2.0 ** -149 / wtotal)  # the stored norm may be subnormal
    assert np.all(np.abs(tn - wtn) <= NORM_TOL * np.asarray(wtn) + 2.0 ** -149)
    assert abs(sq - wsq) <= 2 * NORM_TOL * wsq
    assert abs(total - wtotal) <= tol * wtotal
    assert abs(coef - wcoef) <= NORM_TOL * wcoef + 2.0 ** -149


@pytest.mark.parametrize("value", [2.0 ** 60, 2.0 ** 50, 2.0 ** -40])
def test_norm_of_a_large_tensor_beyond_the_range_of_squares(z, value):
    """2^30 equal numbers: a thread's 8 * 108 squares, and all other sums, are small
    integers times a power of two, which binary32 holds exactly."""
    x = torch.full((2 ** 30,), value, device="cuda", dtype=torch.bfloat16)
    _, sq, total, coef = norm(z, z.TensorList([x.data_ptr()], [x.numel()], z.BF16), 1.0, tensor_norms=False)
    assert sq == value * value * 2.0 ** 30
    assert total == value * 2.0 ** 15
    assert coef == min(1.0, float(np.float32(1.0 / (value * 2.0 ** 15 + 1e-6))))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_over_mixed_magnitudes(z, dtype):
    """Large and small numbers in one thread's share."""
    b = fill(Buffers([4096, 9], [0, 1], DT[dtype]), 5, 1e-25)
    b.tensors[0][1000] = 1e25
    b.tensors[1][0] = 3.0
    tn, sq, total, _ = norm(z, b.list(z), 1.0)
    wtn, wsq, wtotal, _ = want(b, 1.0)
    assert np.all(np.abs(tn - wtn) <= NORM_TOL * np.asarray(wtn))
    assert abs(total - wtotal) <= NORM_TOL * wtotal


def test_norms_that_are_not_finite(z):
    inf, nan = float("inf"), float("nan")
    for bad, n_want, c_want in ((inf, inf, 0.0), (-inf, inf, 0.0), (nan, nan, nan)):
        b = fill(Buffers([9000, 20], [0, 5], torch.float32), 6)
        b.tensors[1][7] = bad
        tn, sq, total, coef = norm(z, b.list(z), 1.0)
        np.testing.assert_equal([tn[1], sq, total, coef], [n_want, n_want, n_want, c_want])
        assert np.isfinite(tn[0])
        assert norm(z, b.list(z), inf)[3] == 1.0
    # a finite sum of squares whose norm binary32 does not hold
    big = torch.full((64,), 3e38, device="cuda")
    _, sq, total, coef = norm(z, z.TensorList([big.data_ptr()], [64], z.F32), 3e38)
    assert total == inf and abs(coef - 0.125) <= 2.0 ** -24 and np.isfinite(sq)


def test_empty_list_and_zero_gradients(z):
    tn, sq, total, coef = norm(z, z.TensorList([], [], z.F32), 1.0)
    assert (sq, total, coef) == (0.0, 0.0, 1.0)
    x = torch.zeros(1000, dtype=torch.bfloat16, device="cuda")
    x[::3] = -0.0
    tn, sq, total, coef = norm(z, z.TensorList([x.data_ptr(), 0], [1000, 0], z.BF16), 0.5)
    assert tn.tolist() == [0.0, 0.0] and (sq, total, coef) == (0.0, 0.0, 1.0)


# ------------------------------------------------------------------ clipping
@pytest.mark.parametrize("src,dst", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("shift", [0, 1, 2, 4, 5, 7])
def test_clip_into_other_buffers(z, src, dst, shift):
    n = [1, 6, 8, 23, 0, 5000, 16_500, 70_001]
    a = fill(Buffers(n, [i % 8 for i in range(len(n))], DT[src]), 7)
    o = Buffers(n, [(i + shift) % 8 for i in range(len(n))], DT[dst])
    coef = torch.tensor([0.37], device="cuda")
    z.zero3_clip_grads(a.list(z), coef.data_ptr(), o.list(z), sid())
    for x, y in zip(a.tensors, o.tensors):
        assert torch.equal(y, (x.float() * coef).to(DT[dst]))
    assert a.untouched() and o.untouched()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_clip_in_place(z, dtype):
    n = [3, 8, 0, 4097, 30_011]
    a = fill(Buffers(n, [1, 3, 0, 5, 7], DT[dtype]), 8, 1.0)
    before = [t.clone() for t in a.tensors]
    tl = a.list(z)
    ws = torch.empty(z.zero3_grad_norm_workspace(tl), dtype=torch.uint8, device="cuda")
    nc = torch.empty(2, device="cuda")
    for max_norm in (1e9, 2.5):  # nothing to clip, then clipping
        z.zero3_grad_norm(tl, max_norm, 0, 0, nc.data_ptr(), nc[1:].data_ptr(), ws.data_ptr(),
                          ws.numel(), sid())
        z.zero3_clip_grads(tl, nc[1:].data_ptr(), None, sid())
        c = float(nc[1])
        assert (c == 1.0) == (max_norm > 1e6)
        for x, y in zip(before, a.tensors):
            assert torch.equal(y, (x.float() * nc[1]).to(DT[dtype]))
        assert a.untouched()
    assert abs(float(torch.cat([t.float() for t in a.tensors]).norm()) - 2.5) < 2.5 * 2.0 ** -8


def test_clip_many_tensors(z):
    n = [1 + (i * 53) % 97 for i in range(1500)]
    x = torch.randn(sum(n), device="cuda")
    y = torch.zeros(sum(n), dtype=torch.bfloat16, device="cuda")
    coef = torch.tensor([0.25], device="cuda")
    z.zero3_clip_grads(z.TensorList([t.data_ptr() for t in x.split(n)], n, z.F32), coef.data_ptr(),
                       z.TensorList([t.data_ptr() for t in y.split(n)], n, z.BF16), sid())
    assert torch.equal(y, (x * 0.25).to(torch.bfloat16))


# ----------------------------------------------------------- the sharded step
def emulation(w, **kw):
    from zero_sharded_optimizer_shard_gb300.emulation import Emulation
    e = Emulation(w, **kw)
    e.init_params()
    return e


def oracle_state(w):
    plan = O.partition(w.numels, w.submodule_of, w.n_ranks, w.threshold, w.bucket)
    return plan, *O.init_state(plan, *host_master(w, plan))


def assert_state(e, st, full, ps):
    for r in e.state_ranks:
        for name in ("master", "m", "v"):
            assert np.array_equal(bits(f32(getattr(e, name)[r])), bits(getattr(st, name)[r])), (name, r)
        assert np.array_equal(u16(e.sparam[r]), st.sparam[r])
    assert np.array_equal(u16(e.full), full)
    for got, ref in ((e.pmaster, ps.master), (e.pm, ps.m), (e.pv, ps.v)):
        assert np.array_equal(bits(f32(got)), bits(ref))
    assert np.array_equal(u16(e.pparam), ps.param)


def check_coefficient(w, plan, t, max_norm, got_norm, got_coef):
    G, P = host_grads(w, plan, t), host_pgrads(w, plan, t)
    inv = np.float32(1.0 / plan.n_ranks)
    s = CO.square_sum([g for g in CO.reduced(plan, G) if g is not None] + [O.reduce_sum(P, inv)])
    ref = np.sqrt(s)
    assert abs(got_norm - ref) <= NORM_TOL * ref
    assert abs(got_coef - CO.clip_coefficient(s, max_norm)) <= NORM_TOL
    return G, P


WORKLOADS = {"toy": W.toy_mlp, "mini1": lambda: W.mini_gpt(1), "mini4": lambda: W.mini_gpt(4),
             "mini8": lambda: W.mini_gpt(8), "ragged3": lambda: W.ragged_small(3),
             "ragged7": lambda: W.ragged_small(7), "mini33": lambda: W.mini_gpt(33)}


@pytest.mark.parametrize("name", list(WORKLOADS))
@pytest.mark.parametrize("keep", [False, True])
def test_clipped_step(z, name, keep):
    """Two steps, clipped and not; either workspace; the coefficient is read back
    from the parts, and the step has to be the oracle's with it, bit for bit."""
    w = WORKLOADS[name]()
    plan, st, full, ps = oracle_state(w)
    e = emulation(w, guard=64)
    least, best = z.zero3_step_clipped_workspace(e.plan, 0, e.psi_pad)
    assert (best > least) == (w.n_ranks > 4)
    ws = e.alloc(best if keep else least, torch.int8)
    out = torch.full((2,), -1.0, device="cuda")
    sq = torch.empty(1, dtype=torch.float64, device="cuda")
    for t, max_norm in ((1, 0.05), (2, 1e6)):
        e.fill_grads(t)
        G = e.ptrs(e.grads[0])
        z.zero3_grad_square_sum(e.plan, G, 0, e.ptrs(e.pgrads), 0, e.psi_pad, 0, sq.data_ptr(),
                                ws.data_ptr(), least, sid())
        z.zero3_clip_coefficient(sq.data_ptr(), max_norm, 0, out[1:].data_ptr(), sid())
        z.zero3_step_clipped(e.plan, e.hp, t, G, 0, e.ptrs(e.master), e.ptrs(e.m), e.ptrs(e.v),
                             e.ptrs(e.sparam), e.full.data_ptr(), e.persist, 0, e.psi_pad, max_norm,
                             out.data_ptr(), ws.data_ptr(), ws.numel(), sid())
        n, c = out.cpu().tolist()
        hG, hP = check_coefficient(w, plan, t, max_norm, n, c)
        assert (c == 1.0) == (max_norm == 1e6)
        CO.scaled_step(plan, w.hparams, t, hG, st, full, hP, ps, c)
        assert_state(e, st, full, ps)
    assert e.check_guards() == []


@pytest.mark.parametrize("name,bucketed", [("mini3", True), ("mini4", False), ("ragged7", True)])
def test_emulation_steps_with_clipping(z, name, bucketed):
    """Buckets: square sums, one coefficient, scaled steps; one chunk: one call."""
    w = {"mini3": lambda: W.mini_gpt(3), "mini4": lambda: W.mini_gpt(4),
         "ragged7": lambda: W.ragged_small(7)}[name]()
    w.bucket = 100_003
    plan, st, full, ps = oracle_state(w)
    e = emulation(w, bucketed=bucketed, guard=64)
    assert (len(e.chunks) > 3) == bucketed
    for t, max_norm in ((1, 0.04), (2, 0.07), (3, 1e9)):
        e.fill_grads(t)
        e.step(t, max_norm=max_norm)
        n = float(e.norm)
        G, P = host_grads(w, plan, t), host_pgrads(w, plan, t)
        s = CO.square_sum([g for g in CO.reduced(plan, G) if g is not None] +
                          [O.reduce_sum(P, np.float32(1.0 / plan.n_ranks))])
        assert abs(n - np.sqrt(s)) <= NORM_TOL * n
        # the coefficient lies within its tolerance of the 64-bit one: find it
        want = CO.clip_coefficient(s, max_norm)
        tried = [np.float32(want)]
        for _ in range(8):
            tried += [np.nextafter(tried[0], np.float32(0)), np.nextafter(tried[-1], np.float32(2))]
            tried.sort()
        import copy
        for c in tried:
            st2, full2, ps2 = copy.deepcopy(st), full.copy(), copy.deepcopy(ps)
            CO.scaled_step(plan, w.hparams, t, G, st2, full2, P, ps2, c)
            if np.array_equal(bits(f32(e.m[0])), bits(st2.m[0])):
                break
        st, full, ps = st2, full2, ps2
        assert_state(e, st, full, ps)
    assert e.check_guards() == []


@pytest.mark.parametrize("nd", [1, 2, 5, 8, 9])
def test_scaled_replicated_step(z, nd):
    """ZeRO-1/2: every rank's full copy and the shards' states, twice."""
    w = W.mini_gpt(nd)
    plan, st, full, ps = oracle_state(w)
    e = emulation(w)
    reps = [e.full.clone() for _ in range(nd)]
    scale = torch.tensor([0.0], device="cuda")
    for t, c in ((1, 0.3125), (2, 0.7)):
        e.fill_grads(t)
        scale.fill_(c)
        z.zero3_step_stage12_scaled(e.plan, e.hp, t, e.ptrs(e.grads[0]), 0, e.ptrs(e.master), e.ptrs(e.m),
                                    e.ptrs(e.v), e.ptrs(reps), 0, e.psi_pad, scale.data_ptr(), sid())
        CO.scaled_step(plan, w.hparams, t, host_grads(w, plan, t), st, full, host_pgrads(w, plan, t), ps,
                       np.float32(c))
        for r in range(nd):
            for name in ("master", "m", "v"):
                assert np.array_equal(bits(f32(getattr(e, name)[r])), bits(getattr(st, name)[r]))
            assert np.array_equal(u16(reps[r]), full)


@pytest.mark.parametrize("bits_", [8, 4])
@pytest.mark.parametrize("nd", [3, 8])
def test_scaled_quantizing_step(z, nd, bits_):
    w = W.ragged_small(nd)
    plan, st, full, ps = oracle_state(w)
    e = emulation(w)
    n = (e.S + 255) // 256
    codes = [torch.zeros(n * 256, dtype=torch.int8, device="cuda") for _ in range(nd)]
    scales = [torch.zeros(n, device="cuda") for _ in range(nd)]
    scale = torch.tensor([0.21], device="cuda")
    e.fill_grads(1)
    z.zero3_step_qwz_scaled(e.plan, e.hp, 1, e.ptrs(e.grads[0]), 0, e.ptrs(e.master), e.ptrs(e.m),
                            e.ptrs(e.v), e.ptrs(e.sparam), e.ptrs(codes), e.ptrs(scales), e.persist, 0,
                            e.psi_pad, scale.data_ptr(), sid(), bits=bits_)
    CO.scaled_step(plan, w.hparams, 1, host_grads(w, plan, 1), st, full, host_pgrads(w, plan, 1), ps,
                   np.float32(0.21))
    for r in range(nd):
        assert np.array_equal(bits(f32(e.master[r])), bits(st.master[r]))
        c, s = O.qwz_quantize(st.sparam[r], bits=bits_)
        packed = O.qwz_pack(c, bits_)
        assert np.array_equal(codes[r].cpu().numpy().view(np.uint8)[:packed.size], packed.view(np.uint8))
        assert np.array_equal(bits(f32(scales[r])), bits(s))
    assert np.array_equal(bits(f32(e.pmaster)), bits(ps.master))


def test_persistent_gradients_apart(z):
    """Persistent gradients that are no common offset away: a launch of their own."""
    w = W.mini_gpt(5)
    plan, st, full, ps = oracle_state(w)
    e = emulation(w)
    e.fill_grads(1)
    apart = [torch.zeros(e.psi_s + 64 * q + 8, dtype=torch.bfloat16, device="cuda") for q in range(5)]
    for a, g in zip(apart, e.pgrads):
        a[:e.psi_s] = g
    persist = z.persist_state(e.ptrs(apart), e.pmaster.data_ptr(), e.pm.data_ptr(), e.pv.data_ptr(),
                              e.pparam.data_ptr())
    best = z.zero3_step_clipped_workspace(e.plan, 0, e.psi_pad)[1]
    ws = torch.empty(best, dtype=torch.uint8, device="cuda")
    nc = torch.empty(2, device="cuda")
    sq = torch.zeros(1, dtype=torch.float64, device="cuda")
    G = e.ptrs(e.grads[0])
    z.zero3_grad_square_sum(e.plan, G, 0, e.ptrs(apart), 0, e.psi_pad, 0, sq.data_ptr(), ws.data_ptr(), best,
                            sid())
    z.zero3_clip_coefficient(sq.data_ptr(), 0.03, nc.data_ptr(), nc[1:].data_ptr(), sid())
    z.zero3_step_clipped(e.plan, e.hp, 1, G, 0, e.ptrs(e.master), e.ptrs(e.m), e.ptrs(e.v),
                         e.ptrs(e.sparam), e.full.data_ptr(), persist, 0, e.psi_pad, 0.03, nc.data_ptr(),
                         ws.data_ptr(), best, sid())
    hG, hP = check_coefficient(w, plan, 1, 0.03, *nc.cpu().tolist())
    CO.scaled_step(plan, w.hparams, 1, hG, st, full, hP, ps, float(nc[1]))
    assert_state(e, st, full, ps)


def test_clipped_steps_in_a_graph(z):
    """Captured once, replayed twice, with new gradients each time."""
    w = W.ragged_small(7)
    plan, st, full, ps = oracle_state(w)
    e = emulation(w)
    e.fill_grads(1)
    e.step(1, max_norm=0.03)  # makes the workspace
    e.init_params()
    for x in [*e.m, *e.v, e.pm, e.pv]:
        x.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        e.step(1, max_norm=0.03)
    coef = torch.empty(2, device="cuda")
    for t in (1, 2):
        e.fill_grads(t)
        z.zero3_grad_square_sum(e.plan, e.ptrs(e.grads[0]), 0, e.ptrs(e.pgrads), 0, e.psi_pad, 0,
                                e.square_sum.data_ptr(), e.clip_ws.data_ptr(), e.clip_ws.numel(), sid())
        z.zero3_clip_coefficient(e.square_sum.data_ptr(), 0.03, coef.data_ptr(), coef[1:].data_ptr(), sid())
        g.replay()
        assert float(coef[0]) == float(e.norm)
        CO.scaled_step(plan, w.hparams, 1, host_grads(w, plan, t), st, full, host_pgrads(w, plan, t), ps,
                       float(coef[1]))
        assert_state(e, st, full, ps)


def test_gradients_that_are_not_finite(z):
    """An infinite gradient: norm inf, coefficient 0; the other elements take a step
    with zero gradient, its own becomes NaN.  A NaN reaches every element."""
    w = W.mini_gpt(2)
    for bad in (float("inf"), float("nan")):
        e = emulation(w)
        e.fill_grads(1)
        e.grads[0][1][12345] = bad
        e.step(1, max_norm=1.0)
        assert np.isnan(float(e.norm)) if np.isnan(bad) else np.isinf(float(e.norm))
        n = sum(int(torch.isnan(x).sum()) for x in e.m) + int(torch.isnan(e.pm).sum())
        assert n == (2 * e.S + e.psi_s if np.isnan(bad) else 1)
