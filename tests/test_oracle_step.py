"""Pins of the oracles of the operators that close a policy step (oracle/sample.py,
linear.py, gradnorm.py): hand-worked cases, closed forms and differences."""
import numpy as np
import pytest

from oracle import gradnorm, linear, sample

LN = np.log


def test_sample_worked_example():
    # p = (1/2, 1/8, 1/4, 1/8): order 0, 2, 1, 3 (equal ones by index)
    z = LN(np.array([4.0, 1.0, 2.0, 1.0]))
    for u, want in ((0.0, 0), (0.49, 0), (0.51, 2), (0.74, 2), (0.76, 1), (0.87, 1), (0.88, 3)):
        token, logp, logq, kept = sample.row(z, u)
        assert token == want and kept == 4
        assert logp == pytest.approx(LN([0.5, 0.125, 0.25, 0.125][want])) and logq == pytest.approx(logp)
    token, logp, logq, kept = sample.row(z, 0.7, top_k=2)       # 2/3, 1/3
    assert (token, kept) == (2, 2) and logq == pytest.approx(LN(1 / 3)) and logp == pytest.approx(LN(0.25))
    assert sample.row(z, 0.6, top_k=2)[0] == 0
    # top-p of the whole: 0.6 needs two tokens, of the first three (7/8) 0.6 * 7/8 = 0.525: two
    assert sample.row(z, 0.0, top_p=0.6)[3] == 2
    assert sample.row(z, 0.0, top_p=0.45)[3] == 1
    assert sample.row(z, 0.0, top_k=3, top_p=0.9)[3] == 3
    assert sample.row(z, 0.0, min_p=0.3)[3] == 2                 # half the largest passes, a quarter not
    assert sample.row(z, 0.0, min_p=1.0)[3] == 1
    # tau = 1/2 squares the odds: 16 : 4 : 1 : 1
    assert sample.row(z, 0.0, tau=0.5)[1] == pytest.approx(LN(16 / 22))


def test_sample_rows_without_a_token():
    z = np.array([0.0, 1.0, -np.inf])
    assert sample.row(z, -1.0) == (-1, 0.0, 0.0, 0) and sample.row(z, 1.0)[0] == -1
    assert sample.row(z, 0.5)[3] == 2
    for bad in (np.full(3, -np.inf), np.array([0, np.nan, 0]), np.array([0, np.inf, 0])):
        token, logp, logq, kept = sample.row(bad, 0.5)
        assert token == -1 and np.isnan(logp) and np.isnan(logq) and kept == 0


def test_sample_frequencies():
    rng = np.random.default_rng(0)
    z = rng.standard_normal(50)
    p = np.exp(z) / np.exp(z).sum()
    n = 20000
    got = sample.rows(np.broadcast_to(z, (n, 50)), (np.arange(n) + 0.5) / n)[0]
    assert np.all(np.abs(np.bincount(got, minlength=50) - n * p) <= 1)


@pytest.mark.parametrize("name", [None, "relu", "silu", "gelu", "gelu_tanh"])
def test_activations(name):
    x = np.linspace(-6, 6, 4001) + 1e-4
    h = 1e-5
    v, s = linear.act(x, name)
    assert np.allclose((linear.act(x + h, name)[0] - linear.act(x - h, name)[0]) / (2 * h), s, atol=1e-8)
    assert linear.act(np.array([0.0]), name)[0][0] == 0
    assert linear.act(np.array([40.0]), name)[0][0] == 40       # all of them are x far out
    if name == "gelu":
        assert linear.act(np.array([1.0]), name)[0][0] == pytest.approx(0.8413447460685429)
    if name == "silu":
        assert linear.act(np.array([1.0]), name)[0][0] == pytest.approx(np.e / (1 + np.e))
    if name == "gelu_tanh":
        assert np.max(np.abs(v - linear.act(x, "gelu")[0])) < 5e-4


def test_linear_worked_example():
    X, W = np.array([[1.0, 2.0]]), np.array([[3.0, -1.0], [0.5, 1.0], [-4.0, 0.0]])
    out, pre = linear.forward(X, W, np.array([0.5, 0, 1]), "relu", np.array([[10.0, 20, 30]]))
    assert pre.tolist() == [[1.5, 2.5, -3.0]] and out.tolist() == [[11.5, 22.5, 30.0]]
    dY, b = linear.backward_act(np.ones((1, 3)), pre, "relu")
    assert dY.tolist() == [[1, 1, 0]] and b.tolist() == [1, 1, 0]


def test_norm_worked_example():
    gs = [np.array([3.0, 0.0]), np.array([[-4.0]]), np.zeros(0)]
    total, scale, each = gradnorm.norm(gs, 2.5)
    assert total == 5 and scale == 0.5 and each.tolist() == [3, 4, 0]
    assert gradnorm.norm(gs, 2.5, s=-0.25)[:2] == (1.25, -0.25)
    assert gradnorm.norm(gs, 2.0, kind="inf")[:2] == (4, 0.5)
    assert np.isnan(gradnorm.norm([np.array([np.nan])], 1.0)[1])
    assert gradnorm.norm([np.array([np.inf])], 1.0)[1] == 0
