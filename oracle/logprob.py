"""Log probabilities of given tokens, entropy, top alternatives, and their
gradient (TEST INFRASTRUCTURE ONLY).

With a = z / tau and p = softmax(a) per row:
  lse = log sum_j e^a_j,  logp = a[target] - lse,  H = -sum_j p_j log p_j,
  alternatives: descending logits, equal ones by ascending index; tokens with
  a logit of -inf (probability zero) and NaN logits are none.
  dz_j = (g_logp ([j = target] - p_j) - g_H p_j (log p_j + H) + g_lse p_j) / tau
A row whose target lies outside [0, V) is left out (zeros; index -1, -inf).
All arithmetic is fp64.
"""
import numpy as np


def rows(z, target=None, tau=1.0, n_top=0):
    """dict(logp, entropy, lse, top_idx, top_logp); logp None without target."""
    a = np.asarray(z, np.float64) / tau
    n, V = a.shape
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        m = np.max(a, axis=1, keepdims=True)
        m0 = np.where(m == -np.inf, 0.0, m)
        s = np.exp(a - m0).sum(axis=1, keepdims=True)
        lse = (m0 + np.log(s))[:, 0]
        lp = (a - m0) - np.log(s)      # (a - lse would lose log s beside a huge m)
        p = np.exp(lp)
        H = -np.where(a == -np.inf, 0.0, p * lp).sum(axis=1)
        H = np.where(lse == -np.inf, np.nan, H)
    ok = np.ones(n, bool)
    logp = None
    if target is not None:
        t = np.asarray(target)
        ok = (t >= 0) & (t < V)
        with np.errstate(invalid="ignore"):
            logp = np.where(ok, lp[np.arange(n), np.clip(t, 0, V - 1)], 0.0)
    idx = np.full((n, n_top), -1, np.int64)
    top = np.full((n, n_top), -np.inf)
    for i in range(n):
        if not ok[i]:
            continue
        cand = np.flatnonzero(a[i] > -np.inf)          # (False for NaN)
        best = cand[np.argsort(-a[i, cand], kind="stable")][:n_top]
        idx[i, :len(best)] = best
        with np.errstate(invalid="ignore"):
            top[i, :len(best)] = lp[i, best]
    return dict(logp=logp, entropy=np.where(ok, H, 0.0), lse=np.where(ok, lse, 0.0),
                top_idx=idx, top_logp=top)


def gradient(z, target, tau, lse, entropy=None, d_logp=None, d_entropy=None, d_lse=None):
    """dz (fp64) from the given lse and entropy."""
    a = np.asarray(z, np.float64) / tau
    n, V = a.shape
    zero = np.zeros(n)
    g, gh, gl = (zero if x is None else np.asarray(x, np.float64)
                 for x in (d_logp, d_entropy, d_lse))
    H = zero if entropy is None else np.asarray(entropy, np.float64)
    with np.errstate(invalid="ignore"):
        lp = a - np.asarray(lse, np.float64)[:, None]
        p = np.exp(lp)
        plog = np.where(a == -np.inf, 0.0, p * (lp + H[:, None]))
        dz = (gl - g)[:, None] * p - gh[:, None] * plog
    if target is not None:
        t = np.asarray(target)
        ok = (t >= 0) & (t < V)
        dz[np.flatnonzero(ok), t[ok]] += g[ok]
        dz[~ok] = 0.0
    return dz / tau
