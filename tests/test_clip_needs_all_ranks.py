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
