"""fp64 CPU oracle of the global gradient norm and of clipping at it.

TEST INFRASTRUCTURE ONLY, like the other oracles here.

  norm = sqrt(sum g^2),  c = max_norm / norm if norm > max_norm else 1,  out = c g
"""
from __future__ import annotations

import math

import numpy as np


def grad_norm(grads):
    # scaled by the largest magnitude, so that no square leaves fp64's range
    top = max((float(np.max(np.abs(g))) for g in grads if g.size), default=0.0)
    if not math.isfinite(top) or top == 0.0:
        return top
    return top * math.sqrt(math.fsum(float(np.sum((np.asarray(g, dtype=np.float64) / top) ** 2))
                                     for g in grads))


def grad_clip(grads, max_norm):
    norm = grad_norm(grads)
    c = max_norm / norm if norm > max_norm else 1.0
    return norm, [np.asarray(g, dtype=np.float64) * c for g in grads]
