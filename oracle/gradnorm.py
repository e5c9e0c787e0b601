"""The norm of many gradients as one vector, and the factor that clips it (TEST
INFRASTRUCTURE ONLY), in fp64: norm = |s| ||g||, scale = s min(1, max_norm / norm).
"""
import numpy as np


def norm(grads, max_norm=np.inf, s=1.0, kind=2):
    """(norm, scale, each tensor's norm)."""
    def one(flat):
        if flat.size == 0:
            return 0.0
        return np.sqrt(np.sum(flat * flat)) if kind == 2 else np.max(np.abs(flat))
    flats = [np.asarray(g, np.float64).ravel() for g in grads]
    each = np.array([abs(s) * one(f) for f in flats])
    total = abs(s) * one(np.concatenate(flats))
    if np.isnan(total):
        return total, total, each
    return total, s * (max_norm / total if total > max_norm else 1.0), each
