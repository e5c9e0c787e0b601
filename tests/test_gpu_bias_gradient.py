"""linear_backward_act with a bias gradient, on both sides of the rule that picks its kernel
(linear_kernel_shapes.BIAS_SHAPES): one strip of columns and several, whole and ragged, one
chunk of rows and many, against 64 bits.

Whole numbers with slopes of 0 and 1 have to be equal.  Silu: a slope is good to 2^-18 of
1, a sum of T terms errs by at most T u of their magnitudes, u = 2^-24, dY is rounded by
half a step of bf16, 2^-8.
"""
import pytest
import torch

from linear_kernel_shapes import BIAS_SHAPES

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U, H = 2.0 ** -24, 2.0 ** -8
NAN = float("nan")
CASES = [pytest.param(T, d, id=f"{T}x{d}") for T, d, *_ in BIAS_SHAPES]


@pytest.fixture(scope="module")
def lg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rank_gradient_sketching_amd as m
    return m


def padded(t, pad=0):
    n, c = t.shape
    buf = torch.full((n, -(-c // 8) * 8 + 8 * pad), NAN, dtype=t.dtype, device="cuda")
    buf[:, :c] = t
    return buf[:, :c]


def blank(T, d):
    return padded(torch.full((T, d), NAN, dtype=BF, device="cuda"), 1)


def behind_is_nan(t):
    n, c = t.shape
    return bool(t.as_strided((n, t.stride(0)), (t.stride(0), 1))[:, c:].isnan().all())


def nans(d):
    return torch.full((d + 7,), NAN, device="cuda")[:d]


@pytest.mark.parametrize("T,d", CASES)
@pytest.mark.parametrize("d_type", [BF, F32])
def test_exact(lg, T, d, d_type):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    draw = lambda: torch.randint(-4, 5, (T, d), device="cuda", generator=g, dtype=torch.int8)
    D, P = padded(draw().to(d_type), 1), padded(draw().to(BF))
    for act in (None, "relu"):
        pre = None if act is None else P
        want = D.to(F64) * (1.0 if act is None else (P > 0).to(F64))
        dY, db = blank(T, d), nans(d)
        lg.linear_backward_act(D, pre, act, dY=dY, d_bias=db)
        assert torch.equal(dY.to(F64), want) and behind_is_nan(dY)
        assert torch.equal(db.to(F64), want.sum(0))
        if act is None and d_type == BF:        # the sums alone
            db = nans(d)
            assert lg.linear_backward_act(D, d_bias=db) is D
            assert torch.equal(db.to(F64), want.sum(0))
        for over in ([D] if d_type == BF else []) + ([P] if act else []):      # in place
            kept, db = over.clone(), nans(d)
            lg.linear_backward_act(D, pre, act, dY=over, d_bias=db)
            assert torch.equal(over.to(F64), want) and torch.equal(db.to(F64), want.sum(0))
            assert behind_is_nan(over)
            over.copy_(kept)


@pytest.mark.parametrize("T,d", CASES)
@pytest.mark.parametrize("d_type", [BF, F32])
def test_silu(lg, T, d, d_type):
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    N = lambda sig: torch.randn(T, d, device="cuda", generator=g) * sig
    D, P = padded(N(1.0).to(d_type), 1), padded(N(3.0).to(BF))
    p = P.to(F64)
    s = torch.sigmoid(p)
    want = D.to(F64) * s * (1 + p * (1 - s))
    err = 2.0 ** -18 * D.to(F64).abs()
    db = nans(d)
    dY = lg.linear_backward_act(D, P, "silu", dY=blank(T, d), d_bias=db)
    assert bool(((dY.to(F64) - want).abs() <= H * want.abs() + err).all()) and behind_is_nan(dY)
    tol = T * U * want.abs().sum(0) + err.sum(0)
    assert bool(((db.to(F64) - want.sum(0)).abs() <= tol).all())
    again = nans(d)
    lg.linear_backward_act(D, P, "silu", dY=dY, d_bias=again)
    assert torch.equal(again, db)
