"""Gradient norms and clipping in 64 bits, and the sharded step with a scaled
gradient (the step itself in the fixed binary32 order of zero3_oracle)."""
from __future__ import annotations

from typing import Sequence

import numpy as np

from . import zero3_oracle as Z


def square_sum(tensors: Sequence[np.ndarray]) -> float:
    return float(sum(np.sum(np.square(np.asarray(x, np.float64))) for x in tensors))


def clip_coefficient(squares: float, max_norm: float) -> float:
    """min(1, max_norm / (N + 1e-6)); 1 for an infinite max_norm."""
    if np.isinf(max_norm):
        return 1.0
    with np.errstate(invalid="ignore"):
        c = max_norm / (np.sqrt(np.float64(squares)) + 1e-6)
    return float(c) if np.isnan(c) else float(min(1.0, c))


def reduced(plan, grads, flat_lo=0, flat_hi=None) -> list:
    """Every owner's reduced binary32 gradient of flat [flat_lo, flat_hi)."""
    hi = plan.psi_pad if flat_hi is None else flat_hi
    inv = np.float32(1.0 / plan.n_ranks)
    return Z.reduce_scatter(plan, grads, inv, flat_lo, hi)


def scaled_step(plan, hp, t, grads, st, full, pgrads, ps, scale) -> None:
    """zero3_oracle's sharded and persistent steps with the reduced gradient times
    binary32 `scale`, one more rounding; in place."""
    sc = Z.adamw_scalars(hp, t, plan.n_ranks)
    scale = np.float32(scale)
    for r, g in enumerate(reduced(plan, grads)):
        if g is None:
            continue
        p, m, v = Z.adamw_update(g * scale, st.master[r], st.m[r], st.v[r], sc)
        st.master[r][:], st.m[r][:], st.v[r][:] = p, m, v
        st.sparam[r][:] = Z.cast_bf16(p)
    full[:] = Z.allgather(plan, st.sparam)
    g = Z.reduce_sum(pgrads, sc["inv_nd"]) * scale
    ps.master[:], ps.m[:], ps.v[:] = Z.adamw_update(g, ps.master, ps.m, ps.v, sc)
    ps.param[:] = Z.cast_bf16(ps.master)
