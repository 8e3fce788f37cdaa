"""The oracle of clipping: its sums against numpy's norm, the scaled step with a
scale of 1 against the plain step, and a clipped gradient's norm."""
import copy

import numpy as np
import pytest

import oracle as O
from oracle import clip_oracle as CO
from tests._oracle_runs import host_grads, host_master, host_pgrads
from zero_sharded_optimizer_shard_gb300 import workloads as W


def test_sums_and_coefficients():
    rng = np.random.default_rng(0)
    xs = [rng.normal(size=n).astype(np.float32) for n in (1, 7, 1000)]
    s = CO.square_sum(xs)
    assert s == pytest.approx(np.linalg.norm(np.concatenate(xs).astype(np.float64)) ** 2, rel=1e-14)
    assert CO.clip_coefficient(4.0, 1.0) == pytest.approx(1.0 / (2.0 + 1e-6), rel=1e-15)
    assert CO.clip_coefficient(4.0, 3.0) == 1.0
    assert CO.clip_coefficient(np.inf, 3.0) == 0.0
    assert np.isnan(CO.clip_coefficient(np.nan, 3.0))
    assert CO.clip_coefficient(np.nan, np.inf) == 1.0


@pytest.mark.parametrize("nd", [1, 3])
def test_scale_of_one_is_the_plain_step(nd):
    w = W.ragged_small(nd)
    plan = O.partition(w.numels, w.submodule_of, nd, w.threshold, w.bucket)
    st, full, ps = O.init_state(plan, *host_master(w, plan))
    a, b = copy.deepcopy((st, full, ps)), (st, full, ps)
    G, P = host_grads(w, plan, 1), host_pgrads(w, plan, 1)
    CO.scaled_step(plan, w.hparams, 1, G, a[0], a[1], P, a[2], 1.0)
    O.sharded_step(plan, w.hparams, 1, G, b[0], b[1])
    O.persistent_step(plan, w.hparams, 1, P, b[2])
    for r in range(nd):
        for k in ("master", "m", "v"):
            assert np.array_equal(getattr(a[0], k)[r], getattr(b[0], k)[r])
    assert np.array_equal(a[1], b[1]) and np.array_equal(a[2].master, b[2].master)


def test_clipped_moments_have_the_clipped_norm():
    """After one step m = (1 - beta1) g', so its norm is (1 - beta1) max_norm; the
    binary32 roundings (g', the product, 1 - beta1) move it by 2^-22 at most."""
    w = W.ragged_small(2)
    plan = O.partition(w.numels, w.submodule_of, 2, w.threshold, w.bucket)
    st, full, ps = O.init_state(plan, *host_master(w, plan))
    G, P = host_grads(w, plan, 1), host_pgrads(w, plan, 1)
    s = CO.square_sum(CO.reduced(plan, G) + [O.reduce_sum(P, np.float32(0.5))])
    c = CO.clip_coefficient(s, 0.25)
    assert c < 1
    CO.scaled_step(plan, w.hparams, 1, G, st, full, P, ps, c)
    norm = np.sqrt(CO.square_sum(st.m + [ps.m]))
    want = (1 - w.hparams["beta1"]) * 0.25 * np.sqrt(s) / (np.sqrt(s) + 1e-6)
    assert abs(norm - want) <= 2.0 ** -22 * want
