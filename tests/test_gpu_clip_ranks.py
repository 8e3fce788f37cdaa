"""The rank-per-process step with clipping, its CUDA parts on one GPU: every rank's
square sum of its received slices, the coefficient of their total, the scaled step;
the collectives are device copies and a sum, one phase for all ranks before the
next."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle as O  # noqa: E402
from oracle import clip_oracle as CO  # noqa: E402
from tests._oracle_runs import bits, f32, host_grads, host_master, host_pgrads, u16  # noqa: E402
from tests.test_gpu_dist import _bf, _init  # noqa: E402
from zero_sharded_optimizer_shard_gb300 import workloads as W  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nd,wname", [(2, "ragged"), (3, "mini"), (7, "ragged")])
def test_every_rank_clips_by_the_total(lib, nd, wname):
    from zero_sharded_optimizer_shard_gb300 import zero3
    from zero_sharded_optimizer_shard_gb300.distributed import ShardedRank
    w = {"ragged": lambda: W.ragged_small(nd), "mini": lambda: W.mini_gpt(nd)}[wname]()
    plan = zero3.Plan(w.numels, w.submodule_of, nd, w.threshold, w.bucket)
    oplan = O.partition(w.numels, w.submodule_of, nd, w.threshold, w.bucket)
    ranks = [ShardedRank(plan, zero3.hparams(**w.hparams), r, device="cuda") for r in range(nd)]
    S, pad = ranks[0].S, ranks[0].psi_pad
    for rk in ranks:
        _init(rk, w, oplan)
        rk.clipping = True
    st, full, ps = O.init_state(oplan, *host_master(w, oplan))
    for t, max_norm in ((1, 0.02), (2, 1e6)):
        hG, hP = host_grads(w, oplan, t), host_pgrads(w, oplan, t)
        G = [_bf(np.concatenate([g, pg])).cuda() for g, pg in zip(hG, hP)]
        for rk in ranks:
            for q in range(nd):
                rk.slice_of(q).copy_(G[q][rk.rank * S:(rk.rank + 1) * S])
                rk.persist_of(q).copy_(G[q][pad:])
        for rk in ranks:
            rk.sum_squares()
        total = sum(rk.square_sum.clone() for rk in ranks)  # the all-reduce
        for rk in ranks:
            rk.square_sum.copy_(total)
            rk.clip_coefficient(max_norm)
        for rk in ranks:
            rk.fused_step(t)
        s = CO.square_sum([g for g in CO.reduced(oplan, hG) if g is not None] +
                          [O.reduce_sum(hP, np.float32(1.0 / nd))])
        # 8 squares and 5 sums in binary32 per warp: 13 roundings of a sum of squares
        assert abs(float(ranks[0].norm) - np.sqrt(s)) <= 9 * 2.0 ** -24 * np.sqrt(s)
        assert (float(ranks[0].coef) < 1) == (max_norm < 1)
        CO.scaled_step(oplan, w.hparams, t, hG, st, full, hP, ps, float(ranks[0].coef))
        for rk in ranks:
            r = rk.rank
            for k in ("master", "m", "v"):
                assert np.array_equal(bits(f32(getattr(rk, k))), bits(getattr(st, k)[r])), (r, k)
            assert np.array_equal(u16(rk.sparam), st.sparam[r])
            assert np.array_equal(bits(f32(rk.pmaster)), bits(ps.master))
            assert np.array_equal(u16(rk.pparam), ps.param)
