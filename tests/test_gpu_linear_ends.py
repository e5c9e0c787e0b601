"""logra_linear's activations at the ends of the range: infinities, NaN, the largest
values, and the far side where the result is a small part of the input.

Through a 1 x 1 weight of one, or through the bias, pre is the given value exactly.
u = 2^-24, half a step of fp32 (a function that is good to one unit errs by 2 u).
"""
import numpy as np
import pytest
import torch

from oracle import linear as olin

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]
INF, NAN = float("inf"), float("nan")
ENDS = [INF, -INF, NAN, 3e38, -3e38, 1e20, -1e20, 200.0, -200.0, 100.5, 100.0, 99.5, -99.5, 88.0,
        -88.0, 13.0, -13.0, 1.0, -1.0, 0.0, -0.0, 1e-30, -1e-30, 1e-40]


@pytest.fixture(scope="module")
def lg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rank_gradient_sketching_amd as m
    return m


def f64(t):
    return t.detach().double().cpu().numpy()


def by_formula(x, act):
    """The oracle's value; where its terms overflow in between, the formula's own."""
    with np.errstate(all="ignore"):
        v = olin.act(x, act)[0]
    v = np.where(x == INF, INF, np.where(np.isnan(x), NAN, v))
    return np.where(x == -INF, {None: -INF, "relu": 0.0}.get(act, NAN), v)


def check(got, x, act):
    want = by_formula(x, act)
    assert np.array_equal(np.isnan(got), np.isnan(want)), (act, x[np.isnan(got) != np.isnan(want)])
    big = np.isinf(want)
    assert np.array_equal(got[big], want[big])
    ok = ~np.isnan(want) & ~big
    # as for any pre: 2^-20 of |pre| + 1, which past 20 is 0 or pre itself to a rounding
    tol = 2.0 ** -20 * (np.minimum(np.abs(x[ok]), 20) + 1) + 2 * U * np.abs(want[ok])
    assert np.all(np.abs(got[ok] - want[ok]) <= tol), (act, x[ok], got[ok], want[ok])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("times", [1, 8, 80])
def test_through_a_weight(lg, act, times):
    """Rows of the few-rows kernel's number and of the tiles'."""
    x = torch.tensor(ENDS, dtype=BF)[None].repeat(times, 1).reshape(-1)[:7 if times == 1 else None]
    X = torch.zeros(len(x), 8, dtype=BF, device="cuda")
    X[:, 0] = x.cuda()
    out = lg.linear(X[:, :1], torch.ones(1, 1, dtype=BF, device="cuda"), act=act, out_dtype=F32)
    check(f64(out)[:, 0], f64(x), act)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [2, 40, 300])
def test_through_the_bias(lg, act, T):
    b = torch.tensor(ENDS)
    X, W = torch.zeros(T, 8, dtype=BF, device="cuda"), torch.ones(len(b), 8, dtype=BF, device="cuda")
    pre = torch.empty(T, len(b), dtype=BF, device="cuda")
    out = lg.linear(X, W, bias=b.cuda(), act=act, pre=pre, out_dtype=F32)
    for t in (0, T - 1):
        check(f64(out)[t], f64(b), act)
        assert torch.equal(pre[t].cpu().nan_to_num(7.0), b.to(BF).nan_to_num(7.0))


# Relative error of the far side.  gelu = x Phi(x), Phi(-z) = e^(-z^2 / 2) g(z): the
# exponential's argument a = z^2 / 2 carries its own rounding, that of log2(e) and that
# of their product, 3 u of a in all, and the exponential 2 u; t = 1 / (1 + 0.3 z) 4 u,
# which g passes on 2.7-fold at most; the polynomial's eight steps 10 u and its fit
# 1.5e-7 = 2.6 u; three products 3 u: below (3 a + 30) u.  silu: 3 u of the argument,
# 2 u exponential, 1 u sum, 2 u reciprocal, 1 u product.  gelu_tanh: y = 2 sqrt(2 / pi)
# (x + 0.044715 x^3) carries 6 u (two constants, four operations), then as silu.
FAR = {"gelu": (12.5, lambda x: 3 * x * x / 2 + 30),
       "silu": (80.0, lambda x: 3 * np.abs(x) + 6),
       "gelu_tanh": (9.0, lambda x: 9 * 2 * np.sqrt(2 / np.pi) * np.abs(x + 0.044715 * x ** 3) + 6)}


@pytest.mark.parametrize("act", FAR)
def test_far_side_keeps_its_digits(lg, act):
    from scipy.special import erfc, expit
    far, units = FAR[act]
    x = -torch.from_numpy(np.random.default_rng(3).random(4000) * far).to(BF)
    X = torch.zeros(len(x), 8, dtype=BF, device="cuda")
    X[:, 0] = x.cuda()
    got = f64(lg.linear(X[:, :1], torch.ones(1, 1, dtype=BF, device="cuda"), act=act, out_dtype=F32))[:, 0]
    x = f64(x)
    want = {"gelu": lambda: x * 0.5 * erfc(-x / np.sqrt(2)), "silu": lambda: x * expit(x),
            "gelu_tanh": lambda: x * expit(2 * np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3))}[act]()
    assert np.all(np.abs(got - want) <= units(x) * U * np.abs(want))


def test_activation_gradient_of_the_widest_row(lg):
    """One row of 2^31 - 1 columns: slopes of 0 and 1, so all values are exact."""
    d = (1 << 31) - 1
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randint(-3, 4, (1, d + 1), device="cuda", generator=g, dtype=torch.int8).to(BF)[:, :d]
    d_bias = torch.full((d,), NAN, device="cuda")
    dY = lg.linear_backward_act(x, x, "relu", d_bias=d_bias)
    for a in range(0, d, 1 << 28):
        want = x[0, a:a + (1 << 28)].clamp(min=0)
        assert torch.equal(dY[0, a:a + (1 << 28)], want)
        assert torch.equal(d_bias[a:a + (1 << 28)], want.float())
