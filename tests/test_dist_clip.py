"""Clipping across ranks, one per process (gloo, CPU): square sums of the slices,
one all-reduce, the same coefficient everywhere.  The local arithmetic is the
oracle's; what is pinned is who counts what, and the flow around it."""
import os
import sys

import numpy as np
import pytest
import torch
import torch.multiprocessing as mp

from tests.test_dist_sharded import ROOT, _bf, _free_port, _np_u16

MAX_NORMS = (0.02, 1e6, 0.03)


def square_sum(rk):
    import oracle as O
    inv = np.float32(1.0 / rk.nd)
    parts = [O.reduce_sum([_np_u16(rk.slice_of(q)) for q in range(rk.nd)], inv)]
    if rk.rank == 0:
        parts.append(O.reduce_sum([_np_u16(rk.persist_of(q)) for q in range(rk.nd)], inv))
    from oracle import clip_oracle as CO
    rk.square_sum[0] = CO.square_sum(parts)


def coefficient(rk, max_norm):
    from oracle import clip_oracle as CO
    rk.norm[0] = float(np.sqrt(float(rk.square_sum)))
    rk.coef[0] = CO.clip_coefficient(float(rk.square_sum), max_norm)


def local_step(rk, t):
    import oracle as O
    sc = O.adamw_scalars(rk.w.hparams, t, rk.nd)
    c = np.float32(float(rk.coef)) if rk.clipping else np.float32(1)
    for names, grads in ((("master", "m", "v", "sparam"), [rk.slice_of(q) for q in range(rk.nd)]),
                         (("pmaster", "pm", "pv", "pparam"), [rk.persist_of(q) for q in range(rk.nd)])):
        p, m, v, h = (getattr(rk, k) for k in names)
        g = O.reduce_sum([_np_u16(x) for x in grads], sc["inv_nd"]) * c
        new = O.adamw_update(g, p.numpy().copy(), m.numpy().copy(), v.numpy().copy(), sc)
        for x, y in zip((p, m, v), new):
            x.copy_(torch.from_numpy(y))
        h.copy_(_bf(O.cast_bf16(new[0])))


def _worker(rank, world, port, out):
    sys.path.insert(0, ROOT)
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    import torch.distributed as dist
    import oracle as O
    from tests._oracle_runs import host_grads, host_master, host_pgrads
    from zero_sharded_optimizer_shard_gb300 import workloads as W, zero3
    from zero_sharded_optimizer_shard_gb300.distributed import ShardedRank
    dist.init_process_group("gloo", rank=rank, world_size=world)
    w = W.ragged_small(world)
    plan = zero3.Plan(w.numels, w.submodule_of, world, w.threshold, w.bucket)
    oplan = O.partition(w.numels, w.submodule_of, world, w.threshold, w.bucket)
    rk = ShardedRank(plan, zero3.hparams(**w.hparams), rank, device="cpu", local_step=local_step,
                     local_clip=(square_sum, coefficient))
    rk.w = w
    S = rk.S
    mf, mp_ = host_master(w, oplan)
    rk.master.copy_(torch.from_numpy(mf[rank * S:(rank + 1) * S].copy()))
    rk.pmaster.copy_(torch.from_numpy(mp_))
    coefs = []
    for t, max_norm in enumerate(MAX_NORMS, 1):
        rk.grad.copy_(_bf(np.concatenate([host_grads(w, oplan, t)[rank], host_pgrads(w, oplan, t)[rank]])))
        rk.step(t, max_norm=max_norm)
        coefs.append((float(rk.norm), float(rk.coef)))
    out[rank] = (coefs, rk.master.numpy().copy(), _np_u16(rk.full), rk.pmaster.numpy().copy())
    dist.barrier()
    dist.destroy_process_group()


@pytest.mark.parametrize("world", [2, 3])
def test_every_rank_clips_by_the_same_norm(world, lib):
    import oracle as O
    from oracle import clip_oracle as CO
    from tests._oracle_runs import host_grads, host_master, host_pgrads
    from zero_sharded_optimizer_shard_gb300 import workloads as W
    ctx = mp.get_context("spawn")
    out = ctx.Manager().dict()
    mp.start_processes(_worker, args=(world, _free_port(), out), nprocs=world, join=True,
                       start_method="spawn")
    w = W.ragged_small(world)
    plan = O.partition(w.numels, w.submodule_of, world, w.threshold, w.bucket)
    st, full, ps = O.init_state(plan, *host_master(w, plan))
    for t, max_norm in enumerate(MAX_NORMS, 1):
        G, P = host_grads(w, plan, t), host_pgrads(w, plan, t)
        s = CO.square_sum(CO.reduced(plan, G) + [O.reduce_sum(P, np.float32(1.0 / world))])
        # the ranks' sums are added in another order: 64-bit roundings
        norm, c = out[0][0][t - 1]
        assert abs(norm - np.sqrt(s)) <= 2.0 ** -23 * norm
        assert abs(c - CO.clip_coefficient(s, max_norm)) <= 2.0 ** -23
        assert (c < 1) == (max_norm < 1)
        assert all(out[r][0][t - 1] == (norm, c) for r in range(world))
        CO.scaled_step(plan, w.hparams, t, G, st, full, P, ps, c)
    for r in range(world):
        assert np.array_equal(out[r][1].view(np.uint32), st.master[r].view(np.uint32))
        assert np.array_equal(out[r][2], full)
        assert np.array_equal(out[r][3].view(np.uint32), ps.master.view(np.uint32))
