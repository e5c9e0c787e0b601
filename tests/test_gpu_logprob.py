"""logra_token_logprob and its gradient on the GPU against the fp64 oracle.

Tolerances (u = 2^-24, half a step of fp32):
  s, u: each weight 2^d carries the exponential's own error (2 u) and that of
  its exponent, 2 u |d| ln 2 weighted by the weight itself (the mean of |d| ln 2
  is at most ln V + 1 <= 13); a thread adds ceil(V / 256) of them one after the
  other, then ten to eighteen merges of five roundings each: relative error R =
  u (ceil(V / 256) + 160).
  lse: |lse| is rounded three times, ln s carries R:  R + 3 u |lse|.
  logp: (z - m) / tau three times, ln s, the sum:     R + 4 u (|logp| + ln V).
  H = ln s + ln 2 |u| / s, both terms up to ln V + 1:  R (2 + 2 (ln V + 1)).
  dz: log p = z / tau - lse has error u (|lse| + |log p|), the exponent's
  scaling 2 u |log p|, the exponential 2 u; the factor k0 + k1 log p of a few
  terms 8 u of their magnitudes; then the rounding to the type, half a step.
Rounding to bf16 is at most 2^-8 of the value.
"""
import numpy as np
import pytest
import torch

from oracle import logprob as olp

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def lg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rank_gradient_sketching_amd as m
    return m


def say(*a):
    print(*a, flush=True)


def padded(t, extra=0):
    """GPU copy whose rows have a stride of whole 16-byte groups; NaN behind them."""
    n, V = t.shape
    buf = torch.full((n, -(-V // 8) * 8 + 8 * extra), float("nan"), dtype=t.dtype, device="cuda")
    buf[:, :V] = t.cuda()
    return buf[:, :V]


def logits(n, V, dtype, seed, scale=3.0):
    rng = np.random.default_rng([seed, n, V])
    z = torch.from_numpy(rng.standard_normal((n, V), dtype=np.float32) * np.float32(scale))
    return z.to(DT[dtype])


def targets(n, V, seed, left_out=0.2):
    rng = np.random.default_rng([seed, 9, n])
    t = rng.integers(0, V, n)
    t[rng.random(n) < left_out] = -100
    return torch.from_numpy(t)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def close(got, ref, tol, what):
    got = f64(got)
    same = (got == ref) | (np.isnan(got) & np.isnan(ref))
    with np.errstate(invalid="ignore"):
        err = np.where(same, 0.0, np.abs(got - ref))
    assert np.all(err <= tol), (what, float(np.nanmax(err)), float(np.nanmax(err / tol)))


def check_forward(lg, z, target, tau, n_top, out):
    n, V = z.shape
    zz = f64(z)
    ref = olp.rows(zz, None if target is None else target.cpu().numpy(), tau, n_top)
    R = U * (-(-V // 256) + 160)
    lnV = np.log(V) + 1
    with np.errstate(invalid="ignore"):
        close(out.lse, ref["lse"], R + 3 * U * np.nan_to_num(np.abs(ref["lse"]), posinf=0), "lse")
        close(out.entropy, ref["entropy"], R * (2 + 2 * lnV), "entropy")
        if target is not None:
            tol = R + 4 * U * (np.nan_to_num(np.abs(ref["logp"]), posinf=0) + lnV)
            close(out.logp, ref["logp"], tol, "logp")
        else:
            assert out.logp is None
        if n_top:
            assert np.array_equal(out.top_idx.cpu().numpy(), ref["top_idx"])
            tol = R + 4 * U * (np.nan_to_num(np.abs(ref["top_logp"]), posinf=0, neginf=0) + lnV)
            close(out.top_logp, ref["top_logp"], tol, "top_logp")
    return ref


SHAPES = [
    # n, V, n_top, tau
    (1, 1, 1, 1.0), (3, 2, 4, 1.0), (5, 7, 7, 0.7), (2, 9, 64, 1.0), (4, 63, 5, 1.3),
    (7, 255, 1, 1.0), (3, 2047, 64, 1.0), (2, 2048, 3, 1.0), (2, 2049, 20, 0.5),
    (1, 50001, 8, 1.0), (3, 152064, 64, 1.0), (300, 4099, 5, 1.0), (1100, 5000, 2, 1.0),
    (1500, 640, 0, 0.9), (70, 32003, 0, 1.0),
]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,V,n_top,tau", SHAPES)
def test_forward(lg, n, V, n_top, tau, dtype):
    say("logprob", n, V, n_top, tau, dtype)
    z = padded(logits(n, V, dtype, 1), extra=n % 3)
    t = targets(n, V, 2).cuda()
    out = lg.token_logprob(z, t, tau=tau, n_top=n_top)
    check_forward(lg, z, t, tau, n_top, out)
    # without targets no row is left out
    out = lg.token_logprob(z, tau=tau, n_top=n_top)
    check_forward(lg, z, None, tau, n_top, out)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,V", [(6, 1003), (6, 40000), (1030, 3001)])
def test_masked_and_nonfinite_rows(lg, n, V, dtype):
    say("logprob masks", n, V, dtype)
    z = logits(n, V, dtype, 3)
    lowest = torch.finfo(z.dtype).min
    z[0, : V - 3] = -float("inf")               # three tokens left
    z[1] = -float("inf")                        # none
    z[2, 5:] = lowest                           # masked with the type's lowest value
    z[3, V // 2] = float("nan")
    z[4, V - 1] = float("inf")
    z[5] = lowest                               # uniform at the lowest value
    t = torch.arange(n) % V
    t[0], t[3] = 1, 0                           # a masked token is given
    z, t = padded(z), t.cuda()
    out = lg.token_logprob(z, t, n_top=8)
    ref = check_forward(lg, z, t, 1.0, 8, out)
    assert ref["logp"][0] == -np.inf and out.top_idx[0, 3:].eq(-1).all()
    assert torch.isnan(out.logp[1]) and torch.isnan(out.entropy[1]) and out.lse[1] == -float("inf")
    assert torch.isnan(out.lse[3]) and torch.isnan(out.lse[4])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,V", [(2, 30000), (600, 9001)])
def test_ties_and_orders(lg, n, V, dtype):
    """Equal logits in the order of their index; rising, falling and constant
    rows (every element of a rising row is a new best one)."""
    say("logprob ties", n, V, dtype)
    rng = np.random.default_rng(7)
    z = torch.from_numpy(rng.integers(-2, 3, (n, V)).astype(np.float32))
    z[0] = torch.arange(V, dtype=torch.float32) / 64
    z[1] = 1.0
    z[n - 1, ::3] = -0.0
    z[n - 1, 1::3] = 0.0
    z = padded(z.to(DT[dtype]))
    for n_top in (1, 5, 64):
        out = lg.token_logprob(z, n_top=n_top)
        check_forward(lg, z, None, 1.0, n_top, out)


def test_large_offsets_and_peaks(lg):
    """Rows far from zero (the maximum is subtracted first) and all but certain
    ones."""
    say("logprob offsets")
    z = logits(8, 5003, "fp32", 4)
    z[0] += 3e4
    z[1] -= 3e4
    z[2, 17] = 80.0
    z[3] *= 1e-6
    z = padded(z)
    t = torch.tensor([5, 6, 17, 0, 1, 2, 3, 4]).cuda()
    out = lg.token_logprob(z, t, n_top=3)
    check_forward(lg, z, t, 1.0, 3, out)


def test_out_arguments_streams_and_rows_behind(lg):
    say("logprob out, streams")
    n, V = 37, 5000
    big = padded(logits(n + 4, V, "bf16", 5))
    z, t = big[2:2 + n], targets(n, V, 6).cuda()
    ref = lg.token_logprob(z, t, n_top=4)
    torch.cuda.synchronize()
    guard = {}

    def framed(shape, dtype):
        flat = torch.full((int(np.prod(shape)) + 16,), 7, dtype=dtype, device="cuda")
        guard[len(guard)] = flat
        return flat[8:-8].view(shape)

    out = lg.TokenLogprob(*[framed((n,), torch.float32) for _ in range(3)],
                          framed((n, 4), torch.int32), framed((n, 4), torch.float32))
    ws = torch.full((lg.token_logprob_ws_bytes(n, V, 4),), 0xFF, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = lg.token_logprob(z, t, n_top=4, out=out, ws=ws)
    side.synchronize()
    assert got is out
    for a, b in zip(out, ref):
        assert torch.equal(a, b)                # deterministic
    for flat in guard.values():
        assert flat[:8].eq(7).all() and flat[-8:].eq(7).all()
    # only some of the outputs
    part = lg.token_logprob(z, t, out=lg.TokenLogprob(None, None, torch.empty(n, device="cuda"),
                                                      None, None))
    assert torch.equal(part.lse, ref.lse)
    # no rows
    none = lg.token_logprob(z[:0], t[:0], n_top=2)
    assert none.logp.shape == (0,) and none.top_idx.shape == (0, 2)


# ------------------------------------------------------------------ gradient
def check_grad(z, t, tau, lse, H, g, gh, gl, dz):
    zz = f64(z)
    n, V = zz.shape
    args = [None if x is None else f64(x) for x in (H, g, gh, gl)]
    ref = olp.gradient(zz, None if t is None else t.cpu().numpy(), tau, f64(lse), *args)
    zero = np.zeros(n)
    aH, ag, agh, agl = (zero if x is None else np.abs(x) for x in args)
    with np.errstate(invalid="ignore", over="ignore"):
        lp = zz / tau - f64(lse)[:, None]
        p = np.exp(lp)
        al = np.where(np.isfinite(lp), np.abs(lp), 0.0)
        mag = (ag + agl + agh * aH)[:, None] + agh[:, None] * al
        rel = U * (np.abs(f64(lse))[:, None] + 3 * al + 16)
        tol = np.nan_to_num(rel * p * mag) / tau + 4 * U * ag[:, None] / tau * (t is not None)
    tol = tol + (2.0 ** -8 if z.dtype == torch.bfloat16 else U) * np.abs(np.nan_to_num(ref)) + 1e-37
    close(dz, ref, tol, "dz")
    return ref


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,V,tau", [(1, 1, 1.0), (3, 7, 0.7), (5, 1003, 1.0), (2, 8192, 1.3),
                                     (4, 8193, 1.0), (260, 2050, 1.0), (3, 152064, 1.0)])
def test_gradient(lg, n, V, tau, dtype):
    say("logprob grad", n, V, tau, dtype)
    z = padded(logits(n, V, dtype, 11), extra=1)
    t = targets(n, V, 12).cuda()
    f = lg.token_logprob(z, t, tau=tau)
    rng = np.random.default_rng(13)
    g, gh, gl = (torch.from_numpy(rng.standard_normal(n).astype(np.float32)).cuda()
                 for _ in range(3))
    for sel in ((g, None, None), (None, gh, None), (None, None, gl), (g, gh, gl)):
        H = f.entropy if sel[1] is not None else None
        dz = lg.token_logprob_backward(z, t, f.lse, H, *sel, tau=tau)
        check_grad(z, t, tau, f.lse, H, *sel, dz)
    # no targets: no row is left out
    f = lg.token_logprob(z, tau=tau)
    dz = lg.token_logprob_backward(z, None, f.lse, f.entropy, d_entropy=gh, d_lse=gl, tau=tau)
    check_grad(z, None, tau, f.lse, f.entropy, None, gh, gl, dz)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_masks_in_place_and_padding(lg, dtype):
    say("logprob grad masks", dtype)
    n, V = 5, 3001
    z = logits(n, V, dtype, 14)
    z[0, 10:] = -float("inf")
    z[1] = -float("inf")
    z[2, 7] = float("nan")
    z[3, 9:] = torch.finfo(z.dtype).min
    z = padded(z, extra=2)
    t = torch.tensor([20, 0, 1, 3, -1]).cuda()       # a masked one is given; one left out
    f = lg.token_logprob(z, t)
    g, gh = torch.full((n,), 0.5, device="cuda"), torch.full((n,), -0.25, device="cuda")
    dz = lg.token_logprob_backward(z, t, f.lse, f.entropy, g, gh)
    # (row 0's entropy gradient uses H; the masked target's own term is d_logp)
    check_grad(z, t, 1.0, f.lse, f.entropy, g, gh, None, dz)
    assert dz[0, 20] == 0.5 and dz[0, 21:].eq(0).all() and dz[4].eq(0).all()
    assert torch.isnan(dz[1]).all()
    # in place: same bits, and the columns behind the rows stay as they were
    base = z._base
    before = base[:, V:].clone().view(torch.int16)
    same = lg.token_logprob_backward(z, t, f.lse, f.entropy, g, gh, dz=z)
    assert same is z
    bits = torch.int16 if dtype == "bf16" else torch.int32
    a, b = z.contiguous().view(bits), dz.contiguous().view(bits)
    ok = torch.isfinite(dz)
    assert torch.equal(a[ok], b[ok]) and torch.isnan(z[~ok]).all()
    assert torch.equal(base[:, V:].clone().view(torch.int16), before)


def test_gradient_against_differences(lg):
    """The gradient is that of the forward kernel's own loss: central
    differences of its fp32 outputs.  The step h = 2^-5 leaves a cubic error of
    h^2 / 6 |f'''| <= 2^-12.6 x 6 and fp32 noise R / h in each output."""
    say("logprob grad differences")
    n, V, tau, h = 4, 40, 1.25, 2.0 ** -5
    z = padded(logits(n, V, "fp32", 15, scale=1.0))
    t = torch.tensor([0, 39, 17, 5]).cuda()
    g, gh, gl = (torch.tensor(x, device="cuda") for x in
                 ([1.0, -0.5, 0.25, 2.0], [0.5, 1.0, -1.0, 0.0], [0.0, 0.3, 0.0, -1.0]))
    f = lg.token_logprob(z, t, tau=tau)
    dz = lg.token_logprob_backward(z, t, f.lse, f.entropy, g, gh, gl, tau=tau)

    def loss(x):
        r = lg.token_logprob(x, t, tau=tau)
        return (g.double() * r.logp + gh.double() * r.entropy + gl.double() * r.lse)

    for j in range(V):
        up, down = z.clone(), z.clone()
        up[:, j] += h
        down[:, j] -= h
        d = (loss(padded(up)) - loss(padded(down))) / (2 * h)
        # (third derivatives of logp and lse are below 0.2, of H below 1, / tau^3)
        assert (d - dz[:, j].double()).abs().max() < 4 * (h * h / 6 + 200 * U * 12 / h)


def test_refusals(lg):
    say("logprob refusals")
    z = padded(logits(4, 100, "bf16", 16))
    t = torch.zeros(4, dtype=torch.int64, device="cuda")
    f = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="z must be"):
        lg.token_logprob(z.half())
    with pytest.raises(ValueError, match="target"):
        lg.token_logprob(z, t.int())
    with pytest.raises(ValueError, match="target"):
        lg.token_logprob(z, t[:3])
    with pytest.raises(ValueError, match="n_top"):
        lg.token_logprob(z, t, n_top=65)
    with pytest.raises(ValueError, match="2-D"):
        lg.token_logprob(z.t())
    with pytest.raises(lg._lib.LograError):
        lg.token_logprob(z, t, tau=0.0)
    odd = torch.zeros(4, 101, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(lg._lib.LograError):
        lg.token_logprob(odd, t)                       # rows off their 16-byte boundaries
    with pytest.raises(lg._lib.LograError):
        lg.token_logprob_backward(z, t, f)             # no gradient given
    with pytest.raises(lg._lib.LograError):
        lg.token_logprob_backward(z, t, f, d_entropy=f)
    with pytest.raises(ValueError, match="dz"):
        lg.token_logprob_backward(z, t, f, d_logp=f, dz=torch.zeros(4, 100, device="cuda"))
    with pytest.raises(lg._lib.LograError):
        lg.token_logprob(padded(logits(4, 9000, "bf16", 1)), t, n_top=8,
                         ws=torch.zeros(256, device="cuda", dtype=torch.uint8))


# ------------------------------------------------------------------ far logits
def in_fp32(x):
    """A reference value as fp32 holds it (past the range: infinite)."""
    with np.errstate(over="ignore", invalid="ignore"):
        return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def check_far(lg, z, t, tau, n_top):
    """check_forward for logits of any finite size: log p of a far token is
    ((z - m) l2t) ln 2 - ln s, six roundings of its magnitude (the difference, l2t,
    two products, ln 2, the sum), and the reference is rounded to fp32, half a step
    more; results past fp32's range are infinities."""
    tau = float(np.float32(tau))
    out = lg.token_logprob(z, t, tau=tau, n_top=n_top)
    V = z.shape[1]
    ref = olp.rows(f64(z), t.cpu().numpy(), tau, n_top)
    R = U * (-(-V // 256) + 160)
    lnV = np.log(V) + 1
    size = lambda x: np.where(np.isfinite(x), np.abs(x), 0.0)
    want = {k: in_fp32(ref[k]) for k in ("lse", "entropy", "logp", "top_logp")}
    close(out.lse, want["lse"], R + 4 * U * size(want["lse"]), "lse")
    close(out.entropy, want["entropy"], R * (2 + 2 * lnV), "entropy")
    close(out.logp, want["logp"], R + 8 * U * (size(want["logp"]) + lnV), "logp")
    if n_top:
        assert np.array_equal(out.top_idx.cpu().numpy(), ref["top_idx"])
        close(out.top_logp, want["top_logp"], R + 8 * U * (size(want["top_logp"]) + lnV), "top_logp")


@pytest.mark.parametrize("tau", [0.7, 1.0, 1.5, 2.0])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,V", [(24, 9001), (24, 40000), (600, 2600)])
def test_far_values(lg, n, V, dtype, tau):
    """Finite values so large that one step of fp32 at z log2(e) / tau is more than
    the exponent's whole range: as masks over the head, the tail, or all but a few
    tokens of a row, in all of it, and as peaks above it.  (24 rows are cut into
    pieces whose states are joined, 600 are not.)"""
    say("logprob far", n, V, dtype, tau)
    z = logits(n, V, dtype, 21)
    t = torch.arange(n) * 37 % V
    row = 0
    for size in (1e8, 1e10, 1e20, 1e30, torch.finfo(z.dtype).max):
        z[row] = -size                          # uniform: log p = -log V
        z[row + 1, V // 3:] = -size             # the tail of the vocabulary
        z[row + 2, :V - 700] = -size            # its head (the first groups of every thread)
        z[row + 3, 1000:] = size                # a uniform distribution above a finite rest
        t[row:row + 4] = torch.tensor([3, V - 1, V - 5, 17])
        row += 4
    z[row, ::2] = -torch.finfo(z.dtype).max     # every group holds some
    z[row + 1] = torch.finfo(z.dtype).max
    z[row + 2] = torch.linspace(-1e9, 1e9, V)   # one token far above the next
    z[row + 3] = torch.linspace(1e9, -1e9, V)
    check_far(lg, padded(z), t.cuda(), tau, 4)


@pytest.mark.parametrize("tau", [0.7, 1.0, 1.5])
@pytest.mark.parametrize("n,V", [(6, 9001), (600, 2600)])
def test_where_the_fused_exponent_ends(lg, n, V, tau):
    """fp32 rows whose values lie on both sides of |z| log2(e) / tau = 2^24, whole
    numbers apart, so that threads whose references lie on either side are joined."""
    say("logprob fused border", n, V, tau)
    z = logits(n, V, "fp32", 22)
    at = float(np.float32(2.0 ** 24 / np.log2(np.e) * tau))
    rng = np.random.default_rng(23)
    for row, sign in ((0, 1), (1, -1), (2, 1), (3, -1)):
        step = torch.from_numpy(rng.integers(-3, 4, V).astype(np.float32))
        z[row] = sign * round(at) + step
        if row >= 2:                            # rising: every group raises its reference
            z[row] = sign * round(at) + torch.arange(V, dtype=torch.float32) // (V // 16) - 8
    z[4, :V // 2] = round(at) - 12
    z[4, V // 2:] = round(at) + 12
    z[5] = -round(at)
    z[5, V - 1] = 1e7
    t = torch.arange(n) * 37 % V
    check_far(lg, padded(z), t.cuda(), tau, 0 if n > 100 else 4)


def test_gradient_rows_without_a_finite_lse(lg):
    """Where z / tau leaves fp32's range the forward's lse is infinite: such a row's
    gradient is NaN, whatever the signs, and its neighbours' are their own."""
    say("logprob grad infinite lse")
    n, V = 6, 3001
    for dtype in ("bf16", "fp32"):
        z = logits(n, V, dtype, 24)
        z[1, 9] = 1e38
        z[3] = -float("inf")
        z[4] = -3e38
        z = padded(z)
        t = torch.tensor([5, 9, 6, 7, 8, -1]).cuda()
        f = lg.token_logprob(z, t, tau=0.1)
        assert f.lse[1] == float("inf") and f.lse[3] == f.lse[4] == -float("inf")
        g, gh = torch.full((n,), 0.5, device="cuda"), torch.full((n,), -0.25, device="cuda")
        H = torch.nan_to_num(f.entropy)         # (NaN itself would do)
        for a, b, c in ((g, None, None), (None, gh, None), (None, None, g), (g, gh, g)):
            dz = lg.token_logprob_backward(z, t, f.lse, None if b is None else H, a, b, c, tau=0.1)
            assert torch.isnan(dz[[1, 3, 4]]).all(), dtype
            assert torch.isfinite(dz[[0, 2, 5]]).all() and dz[5].eq(0).all()
        lse = f.lse.clone()                     # (a left-out row stays zero)
        lse[5] = float("inf")
        assert lg.token_logprob_backward(z, t, lse, d_lse=g, tau=0.1)[5].eq(0).all()


@pytest.mark.parametrize("tau", [4e-8, 3e-8, 1.7e-8, 1e-8, 7e-12, 1.3e-20])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_masks_at_small_temperatures(lg, dtype, tau):
    """Masked tokens, by -inf and by the type's lowest value, are zero at any
    temperature; the others follow the formula."""
    say("logprob grad small tau", dtype, tau)
    n, V, tau = 4, 2050, float(np.float32(tau))
    z = (logits(n, V, "fp32", 25).double() * tau).to(DT[dtype])
    z[0, 100:] = -float("inf")
    z[1, ::3] = torch.finfo(z.dtype).min
    z[2, :600] = -1e30
    z = padded(z)
    t = torch.tensor([200, 1, 700, 5]).cuda()   # (row 0: a masked one is given)
    f = lg.token_logprob(z, t, tau=tau)
    g, gh = torch.full((n,), 0.5, device="cuda"), torch.full((n,), -0.25, device="cuda")
    dz = lg.token_logprob_backward(z, t, f.lse, f.entropy, g, gh, tau=tau)
    assert dz[0, 100:200].eq(0).all() and dz[0, 201:].eq(0).all()
    assert abs(dz[0, 200].item() * tau - 0.5) <= 0.5 * 2.0 ** -7
    assert dz[1, ::3].eq(0).all() and dz[2, :600].eq(0).all()
    zz, ok = f64(z), np.arange(1, n)
    ref = olp.gradient(zz, t.cpu().numpy(), tau, f64(f.lse), f64(f.entropy), f64(g), f64(gh))[ok]
    # (log p's error u (|lse| + |log p|) + 2 u |log p|, beside a factor of up to
    # 0.5 + 0.25 (H + |log p|) <= 8; H <= ln V = 8, |log p| <= 25)
    with np.errstate(over="ignore"):
        p = np.exp(zz / tau - f64(f.lse)[:, None])[ok]
    step = 2.0 ** -8 if dtype == "bf16" else U
    tol = U * (100 * p * 8 + 2) / tau + step * np.abs(ref)
    assert np.all(np.abs(f64(dz)[ok] - ref) <= tol), np.max(np.abs(f64(dz)[ok] - ref) / tol)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_masks_at_the_smallest_temperatures(lg, dtype):
    """1 / tau near fp32's largest value: a masked token's clamped log p must not
    carry the entropy's factor past it."""
    test_gradient_masks_at_small_temperatures(lg, dtype, 2e-37)


@pytest.mark.parametrize("tau", [0.7, 1.0, 1.5])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_of_far_rows(lg, dtype, tau):
    """Rows that are masked whole by a large finite value, or peak at one: fp32's lse
    cannot tell their tokens apart, but no p is above 1, so the gradient stays finite,
    and zero where the loss's own gradients are.  Rows with a part masked follow the
    formula."""
    say("logprob grad far rows", dtype, tau)
    n, V, tau = 18, 3001, float(np.float32(tau))
    z = logits(n, V, dtype, 26)
    sizes = (1e6, 3e7, 1e10, 7e15, 1e20, 1e30)
    for i, size in enumerate(sizes):
        z[3 * i] = -size
        z[3 * i + 1, V // 2:] = size
        z[3 * i + 2, V // 2:] = -size
    z = padded(z)
    t = (torch.arange(n) * 37 % (V // 2)).cuda()
    f = lg.token_logprob(z, t, tau=tau)
    g, gh = torch.full((n,), 0.5, device="cuda"), torch.full((n,), -0.25, device="cuda")
    dz = lg.token_logprob_backward(z, t, f.lse, f.entropy, g, gh, tau=tau)
    # (0.5 + 0.25 (H + 0) with p = 1, or e^-1 / 4 more; and the target's 0.5)
    assert torch.isfinite(dz).all() and dz.float().abs().max().item() <= (1 + 0.25 * 9) / tau
    part = torch.arange(2, n, 3).cuda()
    sel = lambda x: x[part].contiguous()
    check_grad(z[part], t[part], tau, sel(f.lse), sel(f.entropy), sel(g), sel(gh), None, dz[part])
    zero = torch.zeros(n, device="cuda")
    assert lg.token_logprob_backward(z, t, f.lse, f.entropy, zero, zero, tau=tau).eq(0).all()
    # a NaN logit beside a finite lse is still seen
    z[2, 5] = float("nan")
    assert torch.isnan(lg.token_logprob_backward(z, t, f.lse, d_logp=g, tau=tau)[2, 5])
