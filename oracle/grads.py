"""Float64 oracle of the gradient operators: 2-norms and clipping."""

from __future__ import annotations

import math

import numpy as np


def norms(grads):
    """(norm of all, norm of each).  math.hypot scales, so nothing overflows or underflows."""
    each = [math.hypot(*np.asarray(g, np.float64).ravel().tolist()) for g in grads]
    return math.hypot(*each), each


def factor(norm, max_norm):
    """What clipping to max_norm multiplies by."""
    if math.isinf(max_norm):
        return 1.0
    f = 0.0 if math.isinf(norm) else max_norm / (norm + 1e-6)
    return f if math.isnan(f) else min(1.0, f)
