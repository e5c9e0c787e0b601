"""Every kernel behind logra_linear and its gradients, whole and split, against products in
64 bits, with ragged edges and the epilogue (linear_kernel_shapes.py; which shape reaches
which kernel is checked in test_launches_step.py).

Operands are small whole numbers: products, sums, bias and residual stay below 2^24, so
fp32 holds every partial sum and results have to be equal (bf16 ones: the exact value
rounded once).  Rows are padded with NaN, of operands and of results, where it has to
stay.  Gelu: a sum of K exact products errs by at most K u M, M = sum |x w|, u = 2^-24, the
slope is at most 1.13, gelu itself good to 2^-20 (|pre| + 1); the residual's sum and the
result's rounding are half a step each.
"""
import pytest
import torch

from linear_kernel_shapes import SHAPES, form_of, has

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U, H = 2.0 ** -24, 2.0 ** -8
NAN = float("nan")
IDS = ["{0.kernel}{1}{2}-{0.M}x{0.N}x{0.K}".format(s, "-once" * s.once, "-split" * s.split)
       for s in SHAPES]


@pytest.fixture(scope="module")
def lg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rank_gradient_sketching_amd as m
    return m


def say(*a):
    print(*a, flush=True)


def padded(t, pad=0):
    n, c = t.shape
    buf = torch.full((n, -(-c // 8) * 8 + 8 * pad), NAN, dtype=t.dtype, device="cuda")
    buf[:, :c] = t
    return buf[:, :c]


def blank(n, c, dtype):
    return padded(torch.full((n, c), NAN, dtype=dtype, device="cuda"), 1)


def behind_is_nan(t):
    n, c = t.shape
    return bool(t.as_strided((n, t.stride(0)), (t.stride(0), 1))[:, c:].isnan().all())


class Numbers:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def __call__(self, n, c, top=2, dtype=BF):
        x = torch.randint(-top, top + 1, (n, c), device="cuda", generator=self.g, dtype=torch.int16)
        return x.to(dtype)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_forward(lg, shape):
    say("forward", shape)
    T, d, k = form_of(shape, "forward")
    whole = Numbers(1)
    X, W, R = padded(whole(T, k), 1), padded(whole(d, k)), padded(whole(T, d, 40), 1)
    sums = X.to(F64) @ W.to(F64).t()
    out = blank(T, d, F32)
    lg.linear(X, W, out=out)
    assert torch.equal(out.to(F64), sums) and behind_is_nan(out)
    for bias, out_type in ((whole(1, d, 60)[0], BF), (whole(1, d, 3000, F32)[0], F32)):
        pre_want = sums + bias.to(F64)
        for act, res in (("relu", R), (None, R), ("relu", None)):
            want = pre_want.clamp(min=0) if act else pre_want
            want = (want if res is None else want + R.to(F64)).to(F32).to(out_type)
            out, pre = blank(T, d, out_type), blank(T, d, BF)
            lg.linear(X, W, bias=bias, act=act, residual=res, out=out, pre=pre)
            assert torch.equal(out, want) and behind_is_nan(out)
            assert torch.equal(pre, pre_want.to(F32).to(BF)) and behind_is_nan(pre)
    want = (pre_want.clamp(min=0) + R.to(F64)).to(F32).to(BF)
    lg.linear(X, W, bias=bias, act="relu", residual=R, out=R)      # in place
    assert torch.equal(R, want) and behind_is_nan(R)


@pytest.mark.parametrize("shape", [s for s in SHAPES if has(s, "input")],
                         ids=[i for i, s in zip(IDS, SHAPES) if has(s, "input")])
def test_input_gradient(lg, shape):
    say("input", shape)
    T, d, k = form_of(shape, "input")
    whole = Numbers(2)
    dY, W, R = padded(whole(T, d), 1), padded(whole(d, k)), padded(whole(T, k, 40), 1)
    sums = dY.to(F64) @ W.to(F64)
    for res in (None, R):
        out = blank(T, k, BF)
        lg.linear_backward_input(dY, W, residual=res, out=out)
        want = sums if res is None else sums + R.to(F64)
        assert torch.equal(out, want.to(F32).to(BF)) and behind_is_nan(out)
    lg.linear_backward_input(dY, W, residual=R, out=R)
    assert torch.equal(R, out) and behind_is_nan(R)


@pytest.mark.parametrize("shape", [s for s in SHAPES if has(s, "weight")],
                         ids=[i for i, s in zip(IDS, SHAPES) if has(s, "weight")])
def test_weight_gradient(lg, shape):
    say("weight", shape)
    T, d, k = form_of(shape, "weight")
    whole = Numbers(3)
    dY, X = padded(whole(T, d), 1), padded(whole(T, k))
    sums = dY.to(F64).t().contiguous() @ X.to(F64)
    dW = blank(d, k, F32)
    lg.linear_backward_weight(dY, X, dW=dW)
    assert torch.equal(dW.to(F64), sums) and behind_is_nan(dW)
    dW += 7
    lg.linear_backward_weight(dY, X, dW=dW, accumulate=True)
    assert torch.equal(dW.to(F64), 2 * sums + 7) and behind_is_nan(dW)
    dW = blank(d, k, BF)
    lg.linear_backward_weight(dY, X, dW=dW)
    assert torch.equal(dW, sums.to(F32).to(BF)) and behind_is_nan(dW)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gelu(lg, shape):
    say("gelu", shape)
    T, d, k = form_of(shape, "forward")
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    N = lambda *s, sig=1.0: (torch.randn(*s, device="cuda", generator=g) * sig).to(BF)
    X, W, R, b = padded(N(T, k)), padded(N(d, k, sig=3 * k ** -0.5)), padded(N(T, d)), N(d)
    out, pre = blank(T, d, BF), blank(T, d, BF)
    lg.linear(X, W, bias=b, act="gelu", residual=R, out=out, pre=pre)
    p = X.to(F64) @ W.to(F64).t() + b.to(F64)
    M = X.to(F64).abs() @ W.to(F64).abs().t() + b.to(F64).abs()
    want = p * 0.5 * torch.special.erfc(p * -0.5 ** 0.5) + R.to(F64)
    tol = 1.13 * (k + 2) * U * M + 2.0 ** -20 * (p.abs() + 1) + (2 * U + H) * want.abs()
    assert bool(((out.to(F64) - want).abs() <= tol).all()) and behind_is_nan(out)
    assert bool(((pre.to(F64) - p).abs() <= (k + 2) * U * M + H * p.abs()).all())
    assert behind_is_nan(pre)
