"""logra_linear and its gradients on the GPU against the fp64 oracle.

Exact cases: operands of small integers, whose products and sums are whole numbers
below 2^24, so fp32 holds every partial sum and the results have to be equal (bf16
ones: equal to the exact value rounded once).  A lost, doubled or misplaced term
shows in any of them.

Tolerances for the others (u = 2^-24, half a step of fp32; half a step of bf16 2^-8):
  products of bf16 are exact in fp32; a sum of K of them in any order errs by at most
  K u M, M = sum |x w|.  An activation passes an error on by at most its largest
  slope, 1.13, and adds 2^-20 (|pre| + 1) of its own (the exponential's argument is
  rounded to 2^-24 of at most 18 where the result is not 0 or pre; erfc's 2 units in
  the last place).  Adding the residual and rounding to the type are half a step each.
"""
import numpy as np
import pytest
import torch

from oracle import linear as olin

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32
ACTS = [None, "relu", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def lg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rank_gradient_sketching_amd as m
    return m


def say(*a):
    print(*a, flush=True)


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(t, pad=0, fill=float("nan")):
    """GPU copy with a row stride of whole 16-byte groups (and `pad` more), NaN behind."""
    n, c = t.shape
    buf = torch.full((n, -(-c // 8) * 8 + 8 * pad), fill, dtype=t.dtype, device="cuda")
    buf[:, :c] = t.cuda()
    return buf[:, :c]


def whole(n, c, seed, top=2, dtype=BF):
    rng = np.random.default_rng([seed, n, c])
    return torch.from_numpy(rng.integers(-top, top + 1, (n, c)).astype(np.float32)).to(dtype)


def normal(n, c, seed, scale=1.0, dtype=BF):
    rng = np.random.default_rng([seed, n, c])
    return torch.from_numpy(rng.standard_normal((n, c), dtype=np.float32) * np.float32(scale)).to(dtype)


def blank(n, c, dtype, pad=0):
    """An output whose rows are followed by NaN that has to stay."""
    return rows(torch.zeros(n, c, dtype=dtype), pad + 1)


def behind_is_nan(t):
    n, c = t.shape
    full = t.as_strided((n, t.stride(0)), (t.stride(0), 1))
    return bool(full[:, c:].isnan().all())


# T, k, d: one of everything, tile edges on every side, odd sizes, few rows, long K
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 4096, 520), (2, 7, 9), (3, 63, 130), (5, 65, 1),
          (8, 1000, 300), (15, 128, 257), (16, 512, 128), (17, 96, 264), (33, 200, 129),
          (64, 1536, 1000), (65, 72, 400), (100, 1003, 777), (127, 64, 128), (128, 128, 128),
          (129, 130, 131), (200, 1536, 512), (257, 320, 255), (300, 40, 2000), (513, 513, 513),
          (1000, 2050, 300), (2049, 257, 136), (260, 4097, 520), (70, 12000, 40),
          (1030, 1100, 2060)]


@pytest.mark.parametrize("T,k,d", SHAPES)
def test_products_exact(lg, T, k, d):
    say("linear exact", T, k, d)
    X, W, dY = whole(T, k, 1), whole(d, k, 2), whole(T, d, 3)
    x, w, y = f64(X), f64(W), f64(dY)
    gx, gw, gy = rows(X, 1), rows(W), rows(dY, 2)
    out = blank(T, d, F32)
    lg.linear(gx, gw, out=out)
    assert np.array_equal(f64(out), x @ w.T) and behind_is_nan(out)
    dX = blank(T, k, BF)
    lg.linear_backward_input(gy, gw, out=dX)
    assert torch.equal(dX.cpu(), torch.from_numpy(y @ w).to(BF)) and behind_is_nan(dX)
    dW = blank(d, k, F32)
    lg.linear_backward_weight(gy, gx, dW=dW)
    assert np.array_equal(f64(dW), y.T @ x) and behind_is_nan(dW)
    lg.linear_backward_weight(gy, gx, dW=dW, accumulate=True)
    assert np.array_equal(f64(dW), 2 * (y.T @ x)) and behind_is_nan(dW)
    dW = blank(d, k, BF)
    lg.linear_backward_weight(gy, gx, dW=dW)
    assert torch.equal(dW.cpu(), torch.from_numpy(y.T @ x).to(BF)) and behind_is_nan(dW)


@pytest.mark.parametrize("T,k,d", [(1, 512, 300), (7, 100, 65), (64, 512, 1000), (130, 70, 333),
                                   (520, 260, 264), (33, 9000, 129)])
@pytest.mark.parametrize("out_type", [BF, F32])
def test_epilogue_exact(lg, T, k, d, out_type):
    """Bias of both types, residual, relu, pre; sums that bf16 holds only rounded."""
    say("linear epilogue", T, k, d, out_type)
    X, W, R = whole(T, k, 4), whole(d, k, 5), whole(T, d, 6, 40)
    x, w = f64(X), f64(W)
    gx, gw, gr = rows(X), rows(W, 1), rows(R, 1)
    for bias in (None, whole(1, d, 7, 60)[0], whole(1, d, 8, 3000, F32)[0]):
        for act in (None, "relu"):
            for res in (None, R):
                want, pre = olin.forward(x, w, None if bias is None else f64(bias), act,
                                         None if res is None else f64(R))
                out, gp = blank(T, d, out_type), blank(T, d, BF)
                got = lg.linear(gx, gw, bias=None if bias is None else bias.cuda(), act=act,
                                residual=None if res is None else gr, out=out, pre=gp)
                assert got is out
                assert torch.equal(out.cpu(), torch.from_numpy(want).to(out_type))
                assert torch.equal(gp.cpu(), torch.from_numpy(pre).to(BF))
                assert behind_is_nan(out) and behind_is_nan(gp)
    # into the residual itself, and without given outputs
    want = torch.from_numpy(x @ w.T + f64(R)).to(BF)
    lg.linear(gx, gw, residual=gr, out=gr)
    assert torch.equal(gr.cpu(), want) and behind_is_nan(gr)
    got = lg.linear(gx, gw, out_dtype=out_type)
    assert got.dtype == out_type and np.array_equal(
        f64(got), f64(torch.from_numpy(x @ w.T).to(out_type)))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T,k,d", [(3, 300, 70), (150, 520, 260), (400, 128, 640)])
def test_activations(lg, act, T, k, d):
    say("linear act", act, T, k, d)
    X, W, R = normal(T, k, 9), normal(d, k, 10, 4 / np.sqrt(k)), normal(T, d, 11)
    b = normal(1, d, 12, 2.0, F32)[0]
    for out_type in (F32, BF):
        pre = blank(T, d, BF)
        out = lg.linear(rows(X), rows(W), bias=b.cuda(), act=act, residual=rows(R), pre=pre,
                        out_dtype=out_type)
        want, p = olin.forward(f64(X), f64(W), f64(b), act, f64(R))
        M = np.abs(f64(X)) @ np.abs(f64(W)).T + np.abs(f64(b))
        tol = 1.13 * (k + 2) * U * M + 2.0 ** -20 * (np.abs(p) + 1) + 2 * U * np.abs(want)
        if out_type == BF:
            tol = tol + H * np.abs(want)
        assert np.all(np.abs(f64(out) - want) <= tol)
        assert np.all(np.abs(f64(pre) - p) <= (k + 2) * U * M + H * np.abs(p))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("d_type", [BF, F32])
@pytest.mark.parametrize("T,d", [(1, 1), (1, 300), (7, 8), (9, 257), (64, 1000), (1000, 129),
                                 (4099, 36)])
def test_backward_act(lg, act, d_type, T, d):
    D, P = normal(T, d, 13, 1.0, d_type), normal(T, d, 14, 3.0)
    want, bias = olin.backward_act(f64(D), f64(P), act)
    gd, gp = rows(D, 1), None if act is None else rows(P)
    dY, d_bias = blank(T, d, BF), torch.full((d,), float("nan"), device="cuda")
    got = lg.linear_backward_act(gd, gp, act, dY=dY, d_bias=d_bias)
    assert got is dY and behind_is_nan(dY)
    # the slope's terms are below 20 and carry a few units of fp32 each
    err = 2.0 ** -18 * np.abs(f64(D)) * (act not in (None, "relu"))
    assert np.all(np.abs(f64(dY) - want) <= H * np.abs(want) + err + 2.0 ** -133)
    # T terms, added in fp32: T u of their magnitudes at most
    tol = T * U * np.abs(want).sum(0) + err.sum(0) + 1e-30
    assert np.all(np.abs(f64(d_bias) - bias) <= tol)
    other = torch.empty_like(d_bias)
    lg.linear_backward_act(gd, gp, act, dY=None if act is None and d_type == BF else dY,
                           d_bias=other)
    assert torch.equal(other, d_bias)
    # in place, over d_out or over pre
    if d_type == BF:
        again = rows(D, 1)
        assert torch.equal(lg.linear_backward_act(again, gp, act, dY=again), dY)
    if act is not None:
        assert torch.equal(lg.linear_backward_act(gd, gp, act, dY=gp), dY)


@pytest.mark.parametrize("act", ACTS[1:])
def test_slopes_far_out(lg, act):
    """Ends of the range: slopes of 0 and 1, NaN kept; relu'(0) = 0."""
    p = torch.tensor([[0.0, -0.0, 30.0, -30.0, 200.0, -200.0, 3e38, -3e38, float("inf"),
                       -float("inf"), float("nan"), 1e-40, 88.0, -88.0, 13.0, -13.0]], dtype=BF)
    d = torch.full_like(p, 2.0)
    got = f64(lg.linear_backward_act(rows(d), rows(p), act))[0]
    x = np.clip(f64(p)[0], -300, 300)
    want = 2 * olin.act(x, act)[1]
    assert np.isnan(got[10])
    ok = np.arange(16) != 10
    assert np.all(np.abs(got - want)[ok] <= H * np.abs(want)[ok] + 2.0 ** -17)


def test_gradients_against_differences(lg):
    """The chain of the three gradients is the difference quotient of the loss
    <G, out> along random directions (fp64 forward; 3 h^2 and the roundings of dY)."""
    T, k, d, h = 9, 40, 24, 1e-4
    X, W, b = normal(T, k, 15), normal(d, k, 16, 0.3), normal(1, d, 17)[0]
    G = normal(T, d, 18)
    rng = np.random.default_rng(19)
    for act in ACTS[1:]:
        pre = blank(T, d, BF)
        lg.linear(rows(X), rows(W), bias=b.cuda(), act=act, pre=pre)
        d_bias = torch.empty(d, device="cuda")
        dY = lg.linear_backward_act(rows(G), pre, act, d_bias=d_bias)
        dX = lg.linear_backward_input(dY, rows(W))
        dW = lg.linear_backward_weight(dY, rows(X))
        loss = lambda x, w, v: np.sum(f64(G) * olin.forward(x, w, v, act)[0])
        ex, ew, eb = (rng.standard_normal(s) for s in ((T, k), (d, k), (d,)))
        x, w, v = f64(X), f64(W), f64(b)
        for grad, e, lo, hi in (
                (dX, ex, (x - h * ex, w, v), (x + h * ex, w, v)),
                (dW, ew, (x, w - h * ew, v), (x, w + h * ew, v)),
                (d_bias, eb, (x, w, v - h * eb), (x, w, v + h * eb))):
            slope = (loss(*hi) - loss(*lo)) / (2 * h)
            # pre rounded (2^-8 of up to 6, slopes change by at most 1 per unit), dY rounded
            tol = 4 * H * np.linalg.norm(f64(grad)) * np.linalg.norm(e) / np.sqrt(e.size) + 1e-2
            if act == "relu":       # a kink within h of a value moves the quotient
                tol *= 2
            assert abs(np.sum(f64(grad) * e) - slope) <= tol, act


def test_non_finite_values_stay_in_their_rows(lg):
    T, k, d = 40, 200, 300
    X, W, dY = whole(T, k, 20), whole(d, k, 21), whole(T, d, 22)
    x, w, y = f64(X), f64(W), f64(dY)
    gx, gw, gy = rows(X), rows(W), rows(dY)
    gx[7, 3], gw[11, 5], gy[9, 1] = float("nan"), float("inf"), float("nan")
    ok_t, ok_d = np.arange(T) != 7, np.arange(d) != 11
    out = f64(lg.linear(gx, gw, out_dtype=F32))
    assert np.array_equal(out[np.ix_(ok_t, ok_d)], (x @ w.T)[np.ix_(ok_t, ok_d)])
    assert np.isnan(out[7]).all()
    dX = f64(lg.linear_backward_input(gy, rows(W)))
    ok = np.arange(T) != 9
    assert np.array_equal(dX[ok], f64(torch.from_numpy(y @ w).to(BF))[ok]) and np.isnan(dX[9]).all()
    dW = f64(lg.linear_backward_weight(gy, rows(X)))
    ok = np.arange(d) != 1
    assert np.array_equal(dW[ok], (y.T @ x)[ok]) and np.isnan(dW[1]).all()


def test_empty_batch(lg):
    X, W = torch.empty(0, 16, device="cuda", dtype=BF), whole(8, 16, 23).cuda()
    assert lg.linear(X, W).shape == (0, 8)
    dY = torch.empty(0, 8, device="cuda", dtype=BF)
    d_bias = torch.full((8,), 5.0, device="cuda")
    lg.linear_backward_act(dY, d_bias=d_bias)
    assert torch.equal(d_bias, torch.zeros_like(d_bias))
    assert lg.linear_backward_input(dY, W).shape == (0, 16)
    dW = torch.full((8, 16), 5.0, device="cuda")
    lg.linear_backward_weight(dY, X, dW=dW, accumulate=True)
    assert dW.eq(5).all()
    lg.linear_backward_weight(dY, X, dW=dW)
    assert dW.eq(0).all()


def test_long_strides(lg):
    """Row offsets past 2^31 elements in every operand."""
    T, k, d, ld = 3, 130, 140, (1 << 30) + 8
    bufs = [torch.empty(2 * ld + 1024, dtype=BF, device="cuda") for _ in range(3)]
    X, W, R = whole(T, k, 24), whole(3, k, 25), whole(T, 3, 26)
    far = [b.as_strided(t.shape, (ld, 1)) for b, t in zip(bufs, (X, W, R))]
    for v, t in zip(far, (X, W, R)):
        v.copy_(t)
    out = lg.linear(far[0], far[1], residual=far[2], out_dtype=F32)
    assert np.array_equal(f64(out), f64(X) @ f64(W).T + f64(R))
    dY = whole(T, 3, 27)
    dX = lg.linear_backward_input(rows(dY), far[1])
    assert np.array_equal(f64(dX), f64(torch.from_numpy(f64(dY) @ f64(W)).to(BF)))
    far[2].copy_(dY)
    dW = lg.linear_backward_weight(far[2], far[0])
    assert np.array_equal(f64(dW), f64(dY).T @ f64(X))
    lg.linear(rows(X), rows(W), out=far[2])
    assert torch.equal(far[2].cpu(), torch.from_numpy(f64(X) @ f64(W).T).to(BF))


def test_bits_graph_and_streams(lg):
    T, k, d = 90, 2000, 300
    X, W, R = normal(T, k, 28), normal(d, k, 29, 0.02), normal(T, d, 30)
    gx, gw, gr = rows(X), rows(W), rows(R)

    def run(out, pre, dX, dW, db, ws):
        lg.linear(gx, gw, act="gelu", residual=gr, out=out, pre=pre, ws=ws[0])
        dY = lg.linear_backward_act(gr, pre, "gelu", dY=pre, d_bias=db, ws=ws[1])
        lg.linear_backward_input(dY, gw, residual=gx, out=dX, ws=ws[0])
        lg.linear_backward_weight(dY, gx, dW=dW, ws=ws[0])
        return [x.clone() for x in (out, pre, dX, dW, db)]

    def buffers():
        byte = lambda n: torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        return (blank(T, d, BF), blank(T, d, BF), blank(T, k, BF), blank(d, k, F32),
                torch.empty(d, device="cuda"),
                (byte(lg.linear_ws_bytes(T, d, k)), byte(lg.linear_backward_act_ws_bytes(T, d))))

    a, b = buffers(), buffers()
    ref = run(*a)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(*a)
    for rep in range(4):
        for x in a[:5]:
            x.zero_()
        got = run(*b[:5], a[5])                   # eager work through the same scratch
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a[:5], ref)), rep
        assert all(torch.equal(x, y) for x, y in zip(got, ref)), rep
    streams = [torch.cuda.Stream() for _ in range(2)]
    for buf, q in zip((a, b), streams):
        q.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(q):
            run(*buf)
    torch.cuda.synchronize()
    for buf in (a, b):
        assert all(torch.equal(x, y) for x, y in zip(buf[:5], ref))


def test_large(lg):
    """A training microbatch's sizes, on sampled rows and columns."""
    T, k, d = 4100, 4096, 4104
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    X, W, dY = (torch.randint(-2, 3, s, device="cuda", generator=g).to(BF)
                for s in ((T, k), (d, k), (T, d)))
    t = [0, 1, 127, 128, 255, 256, 2047, 2048, 4095, 4096, 4099]
    n = [0, 7, 8, 128, 1000, 2048, 4095]
    out = lg.linear(X, W, out_dtype=F32)
    assert np.array_equal(f64(out[t]), f64(X[t]) @ f64(W).T)
    assert np.array_equal(f64(out[:, n]), f64(X) @ f64(W[n]).T)
    dX = lg.linear_backward_input(dY, W)
    want = torch.from_numpy(f64(dY[t]) @ f64(W)).to(BF)
    assert torch.equal(dX[t].cpu(), want)
    dW = lg.linear_backward_weight(dY, X)
    assert np.array_equal(f64(dW[n]), f64(dY[:, n]).T @ f64(X))
    assert np.array_equal(f64(dW[:, n]), f64(dY).T @ f64(X[:, n]))
