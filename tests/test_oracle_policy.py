"""The oracle of the policy-step operators against closed forms, differences
and direct loops (CPU)."""
import numpy as np
import pytest

from oracle import adamw, adapter, logprob


def test_logprob_closed_forms():
    # uniform: logp = -log V, H = log V; two-point: p = (1/4, 3/4)
    r = logprob.rows(np.zeros((1, 8)), [3], 1.0, 3)
    assert np.isclose(r["logp"][0], -np.log(8)) and np.isclose(r["entropy"][0], np.log(8))
    assert r["top_idx"].tolist() == [[0, 1, 2]]            # ties by index
    z = np.array([[0.0, 2 * np.log(3.0), -np.inf]])
    r = logprob.rows(z, [0], 2.0, 3)
    assert np.isclose(r["logp"][0], np.log(0.25))
    assert np.isclose(r["entropy"][0], -(0.25 * np.log(0.25) + 0.75 * np.log(0.75)))
    assert r["top_idx"].tolist() == [[1, 0, -1]] and r["top_logp"][0, 2] == -np.inf
    # left out, no distribution, NaN
    z = np.array([[1.0, 2.0], [-np.inf, -np.inf], [np.nan, 0.0]])
    r = logprob.rows(z, [-100, 0, 1], 1.0, 1)
    assert r["logp"][0] == r["entropy"][0] == r["lse"][0] == 0 and r["top_idx"][0, 0] == -1
    assert np.isnan(r["logp"][1]) and np.isnan(r["entropy"][1]) and r["lse"][1] == -np.inf
    assert np.isnan(r["logp"][2]) and r["top_idx"][2, 0] == 1


@pytest.mark.parametrize("tau", [1.0, 0.6])
def test_logprob_gradient_is_the_difference_quotient(tau):
    rng = np.random.default_rng(5)
    z = rng.normal(size=(3, 7)) * 2
    z[1, 4] = -np.inf
    t = np.array([2, 0, 6])
    g, gh, gl = rng.normal(size=(3, 3))

    def loss(x):
        r = logprob.rows(x, t, tau)
        return g @ r["logp"] + gh @ r["entropy"] + gl @ r["lse"]

    r = logprob.rows(z, t, tau)
    dz = logprob.gradient(z, t, tau, r["lse"], r["entropy"], g, gh, gl)
    for i, j in np.ndindex(z.shape):
        if z[i, j] == -np.inf:
            assert dz[i, j] == 0
            continue
        e = np.zeros_like(z)
        e[i, j] = 1e-5
        assert np.isclose((loss(z + e) - loss(z - e)) / 2e-5, dz[i, j], atol=1e-8)


def test_adamw_first_step_is_the_sign_and_the_decay():
    w, g = np.array([1.0, -2.0, 3.0]), np.array([0.1, -5.0, 0.0])
    new, m, v = adamw.step(w, g, 0 * w, 0 * w, 0.01, 0.9, 0.999, 0.0 + 1e-300, 0.1, 1)
    assert np.allclose(new, w - 0.01 * (np.sign(g) + 0.1 * w))
    assert np.allclose(m, 0.1 * g) and np.allclose(v, 0.001 * g * g)


@pytest.mark.parametrize("which", ["m", "v"])
def test_8bit_form(which):
    keep = adamw.KEEP[which]
    # every code but zero is a value that encodes to itself, whatever the dither
    c = np.arange(1, 128 if which == "m" else 256)
    c = np.concatenate([c, np.zeros(-len(c) % 32, int)])
    c.reshape(-1, 32)[:, 0] = c.max()                 # every block's largest exponent
    E = np.full(len(c) // 32, 120)
    x = adamw.decode(c, E, which)
    for t in (1, 2, 77):
        code, e = adamw.encode(x, t, which)
        assert np.array_equal(code, c) and np.array_equal(e, E)
    # rounding is unbiased over steps, to a spacing over the number of steps
    rng = np.random.default_rng(1)
    x = np.abs(rng.normal(size=320)).astype(np.float32).astype(np.float64) + 0.05
    ys = np.mean([adamw.decode(*adamw.encode(x, t, which), which) for t in range(1, 2001)], axis=0)
    assert np.max(np.abs(ys / x - 1)) < 2.0 ** -keep / 100
    # the zero state, short blocks, small values, non-finite blocks
    code, e = adamw.encode(np.zeros(33), 3, which)
    assert not code.any() and np.array_equal(adamw.decode(code, e, which), np.zeros(33))
    x = np.array([1.0, 2.0 ** -20, 0.0])
    y = adamw.decode(*adamw.encode(x, 3, which), which)
    assert y[0] >= 1 and y[2] == 0
    assert y[1] == (0 if which == "m" else 2.0 ** -15 * (1 + 2.0 ** -keep))
    x = np.concatenate([np.ones(32), [np.nan], np.ones(31)])
    y = adamw.decode(*adamw.encode(x, 3, which), which)
    assert np.isfinite(y[:32]).all() and np.isnan(y[32:]).all()


def test_rounding_to_nearest_would_freeze_the_second_moment():
    """Why the 8-bit form dithers: with beta2 = 0.999 a root changes by at most
    0.05 % a step without a new gradient, far below half a spacing."""
    r, q = 1.0, 2.0 ** -4
    decayed = r * np.sqrt(0.999)
    assert abs(decayed - r) < q / 2 / 4
    # (dithered, 2000 steps without gradients reach the true decay to 10 %)
    x = np.full(32, 1.0)
    for t in range(1, 2001):
        x = adamw.decode(*adamw.encode((x * np.sqrt(0.999)).astype(np.float32), t, "v"), "v")
    assert abs(np.log(x.mean()) / (1000 * np.log(0.999)) - 1) < 0.1


def test_adapter_is_the_merged_weight():
    rng = np.random.default_rng(2)
    T, k, d, r, n = 9, 6, 5, 3, 2
    X, W = rng.normal(size=(T, k)), rng.normal(size=(d, k))
    U, A, s = rng.normal(size=(n, d, r)), rng.normal(size=(n, r, k)), np.array([-0.5, 2.0])
    ids = np.array([0, 1, -1, 0, 1, 1, 2, 0, -7])
    out, _ = adapter.apply(X, X @ W.T, ids, U, A, s)
    for t in range(T):
        Wt = W + (s[ids[t]] * U[ids[t]] @ A[ids[t]] if 0 <= ids[t] < n else 0)
        assert np.allclose(out[t], Wt @ X[t])
