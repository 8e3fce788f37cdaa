"""Refusals of clipping and of drafted tokens' verification: every call carries one
invalid argument, which the library rejects before it touches the GPU."""
import ctypes as C

import pytest

A = 1 << 20  # a plausible, aligned address that is never read
B = 1 << 30  # and one for outputs
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def z(lib):
    from zero_sharded_optimizer_shard_gb300 import zero3
    return zero3


def ptrs(*p):
    return (C.c_void_p * len(p))(*p)


def i64(*v):
    return (C.c_int64 * len(v))(*v)


VERIFY = dict(logits=A, dtype=0, n=4, k=3, vocab=100, stride=100, draft_logits=A, draft_dtype=1,
              draft_stride=100, draft_ids=A, id_type=1, inv_temperature=1.0, draft_inv_temperature=1.0,
              uniform=A, noise=A, noise_stride=100, accepted=B, tokens=B, logprobs=B, stream=None)


@pytest.mark.parametrize("name,value", [
    ("logits", None), ("logits", A + 1), ("dtype", 2), ("dtype", -1), ("n", -1), ("n", 1 << 26), ("k", -1),
    ("k", 257), ("vocab", 0), ("vocab", (1 << 30) + 1), ("stride", 99), ("draft_logits", A + 2),
    ("draft_dtype", 2), ("draft_stride", 99), ("draft_ids", None), ("draft_ids", A + 4), ("id_type", 2),
    ("inv_temperature", 0.0), ("inv_temperature", NAN), ("inv_temperature", INF),
    ("draft_inv_temperature", -1.0), ("draft_inv_temperature", NAN), ("uniform", None), ("uniform", A + 2),
    ("noise", None), ("noise", A + 1), ("noise_stride", 99), ("accepted", None), ("accepted", B + 2),
    ("tokens", None), ("tokens", B + 1), ("logprobs", B + 3)])
def test_verify_refuses(z, name, value):
    assert z.raw_status("zero3_verify_draft", *dict(VERIFY, **{name: value}).values()) == z.EINVAL


@pytest.mark.parametrize("output,bytes_", [("accepted", 4 * 4), ("tokens", 4 * 4 * 4), ("logprobs", 4 * 4 * 4)])
@pytest.mark.parametrize("name,size", [("logits", 2 * 16 * 100), ("draft_logits", 4 * 12 * 100),
                                       ("draft_ids", 8 * 12), ("uniform", 4 * 12), ("noise", 4 * 4 * 100)])
def test_verify_refuses_outputs_over_inputs(z, output, bytes_, name, size):
    """The first and the last place where they share 4 bytes."""
    for at in (B + 4 - bytes_, B + size - 4):
        args = dict(VERIFY, accepted=2 * B, tokens=2 * B, logprobs=2 * B)
        args.update({name: B, output: at})
        assert z.raw_status("zero3_verify_draft", *args.values()) == z.EINVAL


def test_verify_of_no_sequence(z):
    args = dict(VERIFY, n=0, logits=None, draft_ids=None, noise=None, accepted=None, tokens=None, uniform=None)
    assert z.raw_status("zero3_verify_draft", *args.values()) == z.OK


NORM = dict(tensors=ptrs(A, A + 2), numels=i64(10, 20), n=2, dtype=0, max_norm=1.0, tensor_norms=A,
            square_sum=A, norm=A, coef=A, workspace=A, bytes=1 << 20, stream=None)


@pytest.mark.parametrize("name,value", [
    ("tensors", None), ("tensors", ptrs(A, None)), ("tensors", ptrs(A, A + 1)), ("numels", None),
    ("numels", i64(10, -1)), ("numels", i64(1 << 40, (1 << 40) + 1)), ("n", -1), ("n", (1 << 24) + 1),
    ("dtype", 2), ("max_norm", 0.0), ("max_norm", -1.0), ("max_norm", NAN), ("tensor_norms", A + 2),
    ("square_sum", A + 4), ("norm", A + 1), ("coef", A + 2), ("workspace", None), ("workspace", A + 8),
    ("bytes", 100)])
def test_norm_refuses(z, name, value):
    assert z.raw_status("zero3_grad_norm", *dict(NORM, **{name: value}).values()) == z.EINVAL


def test_norm_without_an_output_is_refused(z):
    args = dict(NORM, tensor_norms=None, square_sum=None, norm=None, coef=None)
    assert z.raw_status("zero3_grad_norm", *args.values()) == z.EINVAL


def test_norm_workspace(z):
    def need(*sizes):
        b = C.c_int64()
        assert z.raw_status("zero3_grad_norm_workspace", i64(*sizes), len(sizes), C.byref(b)) == z.OK
        return b.value
    assert 0 < need(1) <= need(1, 1) <= need(1 << 30, 1, 0)
    assert need(1 << 40) < 1 << 20  # blocks grow instead
    assert z.raw_status("zero3_grad_norm_workspace", i64(1), 1, None) == z.EINVAL


CLIP = dict(tensors=ptrs(A, A + 2), numels=i64(10, 20), n=2, dtype=0, coef=A, out=ptrs(A, 2 * A),
            out_dtype=0, stream=None)


@pytest.mark.parametrize("change", [
    dict(tensors=None), dict(numels=None), dict(numels=i64(-1, 2)), dict(dtype=3), dict(out_dtype=3),
    dict(coef=None), dict(coef=A + 2), dict(out=ptrs(A, None)), dict(out=ptrs(A, 2 * A + 1)),
    dict(out=None, out_dtype=1), dict(out_dtype=1), dict(n=-1)])
def test_clip_refuses(z, change):
    assert z.raw_status("zero3_clip_grads", *dict(CLIP, **change).values()) == z.EINVAL


@pytest.mark.parametrize("change", [dict(square_sum=None), dict(square_sum=A + 4), dict(max_norm=0.0),
                                    dict(max_norm=NAN), dict(norm=A + 1), dict(coef=A + 1),
                                    dict(norm=None, coef=None)])
def test_coefficient_refuses(z, change):
    args = dict(dict(square_sum=A, max_norm=1.0, norm=A, coef=A, stream=None), **change)
    assert z.raw_status("zero3_clip_coefficient", *args.values()) == z.EINVAL


@pytest.fixture(scope="module")
def step(z):
    """Arguments of a clipped step of a plan with a persistent tensor, two ranks."""
    plan = z.Plan([100_000, 10], None, 2, threshold=100)
    hp = z.hparams(lr=1e-3)
    ps = z.persist_state([A + 32, A + 32], A, A, A, A)
    two = ptrs(A, A)
    return plan, dict(plan=plan.handle, hp=C.byref(hp), t=1, grads=two, origin=0, master=two, m=two, v=two,
                      sparam=two, full=A, persist=C.byref(ps), lo=0, hi=100_000, max_norm=1.0, norm=A,
                      workspace=A, bytes=1 << 30, stream=None), (hp, ps)


@pytest.mark.parametrize("change", [
    dict(plan=None), dict(hp=None), dict(t=0), dict(grads=None), dict(grads=ptrs(A, None)),
    dict(grads=ptrs(A, A + 2)), dict(origin=1), dict(master=None), dict(m=ptrs(A, None)),
    dict(v=ptrs(A + 4, A)), dict(sparam=None), dict(full=None), dict(full=A + 2), dict(lo=-1),
    dict(hi=100_001), dict(lo=2, hi=1), dict(max_norm=0.0), dict(max_norm=NAN), dict(norm=A + 2),
    dict(workspace=None), dict(workspace=A + 8), dict(bytes=64)])
def test_clipped_step_refuses(z, step, change):
    assert z.raw_status("zero3_step_clipped", *dict(step[1], **change).values()) == z.EINVAL


@pytest.mark.parametrize("field,value", [("master", None), ("m", A + 4), ("v", None), ("param", A + 2)])
def test_clipped_step_refuses_persistent_states(z, step, field, value):
    ps = z.persist_state([A + 32, A + 32], A, A, A, A)
    setattr(ps, field, value)
    assert z.raw_status("zero3_step_clipped", *dict(step[1], persist=C.byref(ps)).values()) == z.EINVAL
    apart = z.persist_state([A + 32, A + 34], A, A, A, A)  # a launch of its own: 16 bytes
    assert z.raw_status("zero3_step_clipped", *dict(step[1], persist=C.byref(apart)).values()) == z.EINVAL


@pytest.mark.parametrize("name", ["zero3_step_scaled", "zero3_step_stage12_scaled", "zero3_step_qwz_scaled"])
@pytest.mark.parametrize("scale", [None, A + 2])
def test_scaled_steps_refuse(z, step, name, scale):
    a, two = step[1], ptrs(A, A)
    head = [a["plan"], a["hp"], 1, two, 0, two, two, two, two]
    more = {"zero3_step_scaled": [A, a["persist"]], "zero3_step_stage12_scaled": [],
            "zero3_step_qwz_scaled": [8, two, two, a["persist"]]}[name]
    assert z.raw_status(name, *head, *more, 0, 100_000, scale, None) == z.EINVAL


@pytest.mark.parametrize("change", [
    dict(plan=None), dict(grads=None), dict(origin=1), dict(pgrads=ptrs(A, None)), dict(lo=-1),
    dict(hi=100_001), dict(square_sum=None), dict(square_sum=A + 4), dict(workspace=None),
    dict(workspace=A + 8), dict(bytes=64)])
def test_square_sum_refuses(z, step, change):
    a = dict(plan=step[0].handle, grads=ptrs(A, A), origin=0, pgrads=ptrs(A, A), lo=0, hi=100_000,
             accumulate=0, square_sum=A, workspace=A, bytes=1 << 20, stream=None)
    assert z.raw_status("zero3_grad_square_sum", *dict(a, **change).values()) == z.EINVAL
