"""One token per row of logits from a given random number, with temperature,
top-k, top-p and min-p (TEST INFRASTRUCTURE ONLY).

The tokens with a logit above -inf in descending order of it, equal ones by
ascending index; kept are the first K = max(1, min(K1, Kp, Km)): K1 = top_k (0:
all), Kp the fewest with mass >= top_p times that of the first K1 (1: no limit),
Km those with p >= min_p max p.  The token is the first whose cumulative mass
exceeds u times the kept mass.  All arithmetic is fp64.
"""
import numpy as np


def row(z, u, tau=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logp, logq, kept) of one row."""
    if not 0 <= u < 1:
        return -1, 0.0, 0.0, 0
    z = np.asarray(z, np.float64)
    legal = 0 < tau < np.inf and 0 < top_p <= 1 and 0 <= min_p <= 1
    if not legal or not np.all(z < np.inf) or not np.any(z > -np.inf):
        return -1, np.nan, np.nan, 0
    order = np.argsort(-z, kind="stable")
    order = order[z[order] > -np.inf]
    gap = (z[order] - z[order[0]]) / tau
    w = np.exp(gap)
    C = np.cumsum(w)
    K = K1 = min(top_k, len(order)) if top_k > 0 else len(order)
    if top_p < 1:
        K = min(K, int(np.argmax(C >= top_p * C[K1 - 1])) + 1)
    if min_p > 0:
        K = min(K, int(np.sum(gap >= np.log(min_p))))
    K = max(K, 1)
    j = int(np.argmax(C > u * C[K - 1]))
    return int(order[j]), gap[j] - np.log(C[-1]), gap[j] - np.log(C[K - 1]), K


def rows(z, u, tau=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logp, logq, kept) arrays; each setting a number or one per row."""
    n = len(z)
    each = [np.broadcast_to(np.asarray(x), (n,)) for x in (u, tau, top_k, top_p, min_p)]
    got = [row(z[t], *(x[t].item() for x in each)) for t in range(n)]
    return [np.array(x) for x in zip(*got)]
