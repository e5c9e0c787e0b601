"""Rank-r updates of several policies beside the projection they share (TEST
INFRASTRUCTURE ONLY).

[LoGRA] Sketch / Sync: a layer's update is W - alpha eta U A with A rebuilt
from a seed.  Applied to the layer's input instead of merged into W:
  out[t] = Y[t] + scale[a] (X[t] A_a^T) U_a^T,  a = adapter[t],
rows with an index outside [0, n) keep Y[t].  All arithmetic is fp64; A holds
the bases as they are (1/sqrt(r) inside).
"""
import numpy as np


def apply(X, Y, adapter, U, A, scale):
    """(out, bound): the result, and sum_i sum_j |X_j| |A_ij| |U_i| |scale| per
    output entry, which scales rounding errors."""
    out = np.array(Y, np.float64)
    bound = np.zeros_like(out)
    X = np.asarray(X, np.float64)
    for a in range(len(U)):
        at = np.flatnonzero(np.asarray(adapter) == a)
        if len(at):
            u, b = np.asarray(U[a], np.float64), np.asarray(A[a], np.float64)
            out[at] += scale[a] * (X[at] @ b.T) @ u.T
            bound[at] = abs(scale[a]) * (np.abs(X[at]) @ np.abs(b).T) @ np.abs(u).T
    return out, bound
