"""Clipping where the global norm, or the clipping itself, is not at hand: such
calls are refused before anything runs (no GPU: nothing is launched)."""
import pytest
import torch

from zero_sharded_optimizer_shard_gb300 import workloads as W


@pytest.fixture
def calls(lib, monkeypatch):
    """The names of the library's steps that are called, none of which run."""
    from zero_sharded_optimizer_shard_gb300 import zero3
    seen = []
    for name in ("zero3_step", "zero3_step_clipped", "zero3_grad_square_sum", "zero3_clip_coefficient",
                 "zero3_step_scaled", "zero3_persistent_step"):
        monkeypatch.setattr(zero3, name, lambda *a, name=name, **k: seen.append(name))
    return seen


def emulation(monkeypatch, **kw):
    from zero_sharded_optimizer_shard_gb300.emulation import Emulation
    monkeypatch.setattr(Emulation, "sid", property(lambda self: 0))
    return Emulation(W.mini_gpt(4), device="cpu", **kw)


@pytest.mark.parametrize("bucketed", [False, True])
@pytest.mark.parametrize("ranks", [[0], [1, 2], [0, 1, 2]])
def test_a_subset_of_the_ranks_has_no_global_norm(calls, monkeypatch, ranks, bucketed):
    e = emulation(monkeypatch, state_ranks=ranks, bucketed=bucketed)
    with pytest.raises(ValueError, match="all 4 ranks"):
        e.step(1, max_norm=1.0)
    assert calls == [] and e.norm is None
    e.step(1)
    assert set(calls) == {"zero3_step"}


@pytest.mark.parametrize("bucketed", [False, True])
@pytest.mark.parametrize("ranks", [None, [0, 1, 2, 3]])
def test_all_ranks_clip(calls, monkeypatch, ranks, bucketed):
    e = emulation(monkeypatch, state_ranks=ranks, bucketed=bucketed)
    e.step(1, max_norm=1.0)
    assert "zero3_step" not in calls
    assert ("zero3_step_clipped" in calls) == (len(e.chunks) == 1)


@pytest.mark.parametrize("own_clip", [False, True])
def test_a_local_step_that_does_not_clip_is_refused_a_norm(lib, monkeypatch, own_clip):
    """A caller's local step alone would take an unclipped step beside a reported norm."""
    from zero_sharded_optimizer_shard_gb300 import distributed, zero3
    ran = []
    monkeypatch.setattr(distributed.ShardedRank, "exchange", lambda self: ran.append("exchange"))
    monkeypatch.setattr(distributed.ShardedRank, "gather", lambda self: ran.append("gather"))
    monkeypatch.setattr(distributed.dist, "all_reduce", lambda *a, **k: ran.append("all_reduce"))
    w = W.mini_gpt(2)
    plan = zero3.Plan(w.numels, w.submodule_of, 2, w.threshold, w.bucket)
    clip = (lambda rk: ran.append("squares"), lambda rk, max_norm: ran.append("coefficient"))
    rk = distributed.ShardedRank(plan, zero3.hparams(**w.hparams), 0, device="cpu",
                                 local_step=lambda rk, t: ran.append(rk.clipping),
                                 local_clip=clip if own_clip else None)
    if own_clip:
        rk.step(1, max_norm=1.0)
        assert ran == ["exchange", "squares", "all_reduce", "coefficient", True, "gather"]
    else:
        with pytest.raises(ValueError, match="local_clip"):
            rk.step(1, max_norm=1.0)
        assert ran == []
    ran.clear()
    rk.step(2)
    assert ran == ["exchange", False, "gather"]
