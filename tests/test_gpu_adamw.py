"""logra_adamw_step and the 8-bit states on the GPU against the fp64 oracle.

Tolerances (u = 2^-24): m' = b1 m + c1 g has three roundings and c1's own, 4 u
of its terms; v' the same, 5 u; the step m / bc1 / (r / sqrt(bc2) + eps) another
six roundings and half of v's error: 12 u of the step beside m's error; the
weight 3 u.  A bf16 weight is rounded once, 2^-8 of the value.  The 8-bit codes
must lie between those that the oracle gives for the value less and more its
tolerance (encoding is monotone for entries above the block's least code).
"""
import numpy as np
import pytest
import torch

from oracle import adamw as oad

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B1, B2, EPS, LR = 0.9, 0.999, 1e-8, 1e-3
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def lg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rank_gradient_sketching_amd as m
    return m


def say(*a):
    print(*a, flush=True)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def place(x, dtype, off):
    """GPU copy of x that starts `off` entries past a 16-byte boundary, with
    guard entries on both sides."""
    buf = torch.full((x.size + off + 24,), 3, dtype=dtype, device="cuda")
    view = buf[8 + off:8 + off + x.size]
    view.copy_(torch.from_numpy(np.ascontiguousarray(x)).to(dtype))
    return view


def guards_ok(t):
    b, lo = t._base, t.storage_offset()
    return bool(b[:lo].eq(3).all()) and bool(b[lo + t.numel():].eq(3).all())


def tensors(sizes, param, grad, master, bits, off, seed):
    rng = np.random.default_rng([seed, bits, off])
    out = []
    for n in sizes:
        sc = 1e-3 * np.exp(rng.standard_normal())
        w = rng.standard_normal(n) * 0.05
        q = dict(n=n, p=place(w, DT[param], off), g=place(rng.standard_normal(n) * sc, DT[grad], off),
                 master=place(w, torch.float32, off) if master else None, m_exp=None, v_exp=None)
        m = (rng.standard_normal(n) * sc * 0.3).astype(np.float32)
        r = ((0.2 + rng.random(n)) * sc).astype(np.float32)
        if bits == 8:
            (cm, em), (cv, ev) = oad.encode(m, 5, "m"), oad.encode(r, 5, "v")
            q.update(m=place(cm, torch.uint8, off), v=place(cv, torch.uint8, off),
                     m_exp=place(em, torch.uint8, off), v_exp=place(ev, torch.uint8, off))
        else:
            q.update(m=place(m, torch.float32, off), v=place(r.astype(np.float64) ** 2, torch.float32, off))
        out.append(q)
    return out


def bind(lg, qs, wd):
    col = lambda k: [q[k] for q in qs]
    return lg.adamw_bind(col("p"), col("g"), col("m"), col("v"), master=col("master"),
                         m_exp=col("m_exp"), v_exp=col("v_exp"), weight_decay=wd)


def state(q):
    if q["m_exp"] is None:
        return f64(q["m"]), f64(q["v"])
    c, e = (x.cpu().numpy() for x in (q["m"], q["m_exp"]))
    d, k = (x.cpu().numpy() for x in (q["v"], q["v_exp"]))
    return oad.decode(c, e, "m"), oad.decode(d, k, "v") ** 2


def check_codes(q, which, x, tol, t, first):
    code, e = q[which].cpu().numpy(), q[which + "_exp"].cpu().numpy()
    got = oad.decode(code, e, which)
    s = np.where(np.signbit(x), -1.0, 1.0)
    a, tol = np.abs(x), np.minimum(tol, np.abs(x))
    # (the block's exponent is that of its largest entry: the same for both ends
    # or between them)
    lo = oad.decode(*oad.encode((s * (a - tol)), t, which, first), which)
    hi = oad.decode(*oad.encode((s * (a + tol)), t, which, first), which)
    l, h = np.minimum(lo, hi), np.maximum(lo, hi)
    assert np.all((got >= l) & (got <= h)), (which, np.max(np.maximum(l - got, got - h)))
    assert np.mean(lo != hi) < 0.01             # the bracket is narrow


def run_and_check(lg, sizes, param, grad, master, bits, off, wd, steps=(6, 7), gscale=None, seed=0):
    qs = tensors(sizes, param, grad, master, bits, off, seed)
    bound = bind(lg, qs, wd)
    wds = wd if isinstance(wd, list) else [wd] * len(qs)
    scale = None if gscale is None else torch.tensor([gscale], device="cuda")
    gs = 1.0 if gscale is None else float(np.float32(gscale))
    for t in steps:
        before = []
        for q in qs:
            w = f64(q["p"] if q["master"] is None else q["master"])
            before.append((w, f64(q["g"]) * gs, *state(q)))
        lg.adamw_step(bound, LR, t, B1, B2, EPS, grad_scale=scale)
        torch.cuda.synchronize()
        first = 0
        for q, (w, g, m, v), decay in zip(qs, before, wds):
            decay = float(np.float32(decay))
            w1, m1, v1 = oad.step(w, g, m, v, LR, B1, B2, EPS, decay, t)
            tm = 4 * U * (np.abs(B1 * m) + 2 * np.abs((1 - B1) * g))
            tv = 5 * U * (B2 * v + 2 * (1 - B2) * g * g)
            bc1, bc2 = 1 - B1 ** t, 1 - B2 ** t
            den = np.sqrt(v1 / bc2) + EPS
            upd = np.abs(m1 / bc1 / den)
            tw = LR * (12 * U * upd + 4 * tm / bc1 / den) + 3 * U * (np.abs(w) + LR * upd + LR * decay * np.abs(w))
            got = f64(q["p"])
            if q["master"] is not None:
                mw = f64(q["master"])
                assert np.all(np.abs(mw - w1) <= tw)
                assert torch.equal(q["p"], q["master"].to(torch.bfloat16))
            else:
                extra = 2.0 ** -8 * np.abs(w1) if param == "bf16" else 0.0
                assert np.all(np.abs(got - w1) <= tw + extra), np.max(np.abs(got - w1) / (tw + extra))
            if bits == 32:
                assert np.all(np.abs(f64(q["m"]) - m1) <= tm + 1e-45)
                assert np.all(np.abs(f64(q["v"]) - v1) <= tv + 1e-45)
            else:
                check_codes(q, "m", m1, tm, t, first)
                check_codes(q, "v", np.sqrt(v1), 0.5 * tv / np.sqrt(v1) + 2 * U * np.sqrt(v1), t, first)
            first += -(-q["n"] // 32) * 32
    for q in qs:
        for k in ("p", "g", "m", "v", "master", "m_exp", "v_exp"):
            assert q[k] is None or guards_ok(q[k]), k


FORMS = [("fp32", "fp32", False), ("fp32", "bf16", False), ("bf16", "bf16", False),
         ("bf16", "fp32", False), ("bf16", "bf16", True), ("bf16", "fp32", True)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,master", FORMS)
@pytest.mark.parametrize("off", [0, 1])
def test_step(lg, param, grad, master, bits, off):
    say("adamw", param, grad, master, bits, off)
    run_and_check(lg, [1, 31, 32, 33, 100, 4095, 4096, 4097, 12345], param, grad, master, bits, off,
                  [0.0, 0.1, 0.0, 0.01, 0.1, 0.0, 0.1, 0.1, 0.05])


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(lg, bits):
    """More tensors than one launch takes, and than one block of the list."""
    say("adamw many", bits)
    rng = np.random.default_rng(3)
    run_and_check(lg, [int(x) for x in rng.integers(1, 700, 300)], "bf16", "bf16", True, bits, 0,
                  0.1, steps=(1,))


@pytest.mark.parametrize("bits", [32, 8])
def test_grad_scale_and_large(lg, bits):
    say("adamw large", bits)
    run_and_check(lg, [1500007], "bf16", "bf16", False, bits, 0, 0.1, steps=(1, 1000), gscale=0.37)


def test_mixed_forms_in_one_list(lg):
    say("adamw mixed")
    qs = []
    for i, (param, grad, master) in enumerate(FORMS):
        qs += tensors([77 + i], param, grad, master, 32 if i % 2 else 8, i % 3, i)
    ref = [{k: (v.clone() if torch.is_tensor(v) else v) for k, v in q.items()} for q in qs]
    lg.adamw_step(bind(lg, qs, 0.1), LR, 3)
    # each tensor by itself; the dither counts blocks of the tensors before it
    for i, q in enumerate(ref):
        if q["m_exp"] is None:
            lg.adamw_step(bind(lg, [q], 0.1), LR, 3)
            for k in ("p", "m", "v"):
                assert torch.equal(q[k], qs[i][k]), (i, k)
        else:
            w, m, v = f64(q["p"] if q["master"] is None else q["master"]), *state(q)
            w1, _, _ = oad.step(w, f64(q["g"]), m, v, LR, B1, B2, EPS, 0.1, 3)
            got = f64(qs[i]["p"] if q["master"] is None else qs[i]["master"])
            assert np.all(np.abs(got - w1) <= 2.0 ** -8 * np.abs(w1) + 1e-7)


def test_8bit_codes_are_the_formula_s(lg):
    """Inputs whose new states are exact in fp32 (g = 0, betas of 1/2 and 1/4):
    every code and exponent, over the whole range of the form."""
    say("adamw codes")
    rng = np.random.default_rng(8)
    n = 32 * 40 + 5
    m = np.exp(rng.uniform(-14, 14, n)) * np.where(rng.random(n) < 0.5, -1, 1)
    r = np.exp(rng.uniform(-14, 14, n))
    m[::7], r[::11] = 0, 0
    m[:32] *= 1e-38
    r[32:64] *= 1e-38
    m[64:96] = 0
    r[96:128] = 0
    (cm, em), (cv, ev) = oad.encode(m.astype(np.float32), 1, "m"), oad.encode(r.astype(np.float32), 1, "v")
    q = dict(p=place(np.zeros(n), torch.float32, 0), g=place(np.zeros(n), torch.float32, 0),
             m=place(cm, torch.uint8, 0), v=place(cv, torch.uint8, 0),
             m_exp=place(em, torch.uint8, 0), v_exp=place(ev, torch.uint8, 0), master=None)
    x, y = oad.decode(cm, em, "m"), oad.decode(cv, ev, "v")
    # (roots whose square leaves fp32's normal range are left to the next test)
    keep = (y == 0) | ((y > 1e-18) & (y < 1e18))
    for k in range(0, n, 32):
        if not keep[k:k + 32].all():
            y[k:k + 32] = 0
            cv[k:k + 32] = 0
    q["v"].copy_(torch.from_numpy(cv))
    pad = place(np.zeros(64), torch.float32, 0)
    small = dict(p=pad, g=place(np.zeros(64), torch.float32, 0), m=place(np.zeros(64), torch.float32, 0),
                 v=place(np.zeros(64), torch.float32, 0), m_exp=None, v_exp=None, master=None)
    lg.adamw_step(bind(lg, [small, q], 0.0), 0.0, 9, beta1=0.5, beta2=0.25)
    for which, val in (("m", x / 2 + 0.0), ("v", y / 2)):   # (-0 + 0 g is +0)
        code, e = oad.encode(val, 9, which, first=64)
        assert np.array_equal(q[which].cpu().numpy(), code), which
        assert np.array_equal(q[which + "_exp"].cpu().numpy(), e), which
        out = lg.adamw_state_values(q[which], q[which + "_exp"], which)
        assert np.array_equal(f64(out), oad.decode(code, e, which))


@pytest.mark.parametrize("bits", [32, 8])
def test_nonfinite_gradients(lg, bits):
    """A NaN or infinite gradient stays in its entry (8 bits: in its block)."""
    say("adamw nonfinite", bits)
    n = 200
    qs = tensors([n], "fp32", "fp32", False, bits, 0, 4)
    qs[0]["g"][40] = float("nan")
    qs[0]["g"][130] = float("inf")
    lg.adamw_step(bind(lg, qs, 0.0), LR, 3)
    q = qs[0]
    p = q["p"].cpu()
    assert torch.isnan(p[40])
    clean = torch.ones(n, dtype=bool)
    clean[40] = clean[130] = False
    assert torch.isfinite(p[clean]).all()
    if bits == 8:
        m = f64(lg.adamw_state_values(q["m"], q["m_exp"], "m"))
        assert np.isnan(m[32:64]).all() and np.isnan(m[128:160]).all()
        rest = np.r_[0:32, 64:128, 160:n]
        assert np.isfinite(m[rest]).all()


def test_zero_states_first_step_and_huge_values(lg):
    say("adamw zero states")
    n = 100
    z8 = lambda k: torch.zeros(k, dtype=torch.uint8, device="cuda")
    g = torch.zeros(n, device="cuda")
    g[::2] = 2.0
    p = torch.zeros(n, device="cuda")
    b = lg.adamw_bind([p], [g], [z8(n)], [z8(n)], m_exp=[z8(4)], v_exp=[z8(4)])
    lg.adamw_step(b, 0.5, 1)
    # the first step is lr times the gradient's sign; no gradient, no step
    assert (p[::2] + 0.5).abs().max() < 1e-6 and p[1::2].eq(0).all()
    # values near the ends of fp32's range
    for size in (1e30, 1e-30):
        q = tensors([64], "fp32", "fp32", False, 8, 0, 6)[0]
        q["g"].copy_(torch.linspace(-2, 2, 64) * size)
        q["m"].zero_()
        q["v"].zero_()
        lg.adamw_step(bind(lg, [q], 0.0), LR, 1)
        m = f64(lg.adamw_state_values(q["m"], q["m_exp"], "m"))
        ref = 0.1 * f64(q["g"])
        assert np.all(np.abs(m - ref) <= 2.0 ** -3 * np.abs(ref) + 2.0 ** -15 * np.abs(ref).max())


def test_follows_adamw_over_steps(lg):
    """8-bit states over 400 steps of a noisy quadratic: the second moments keep
    to the 32-bit run's (dithered rounding does not drift; the spread of sqrt(v)
    simulated on the CPU is 8 % after 1000 steps at beta2 = 0.999)."""
    say("adamw 400 steps")
    n = 4096
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    z8 = lambda k: torch.zeros(k, dtype=torch.uint8, device="cuda")
    f = lambda: torch.zeros(n, device="cuda")
    p8, p32, g = f(), f(), f()
    m8, v8, em, ev = z8(n), z8(n), z8(n // 32), z8(n // 32)
    m32, v32 = f(), f()
    b8 = lg.adamw_bind([p8], [g], [m8], [v8], m_exp=[em], v_exp=[ev])
    b32 = lg.adamw_bind([p32], [g], [m32], [v32])
    scale = torch.exp(torch.randn(n // 32, 1, device="cuda", generator=gen)).expand(-1, 32).reshape(-1)
    for t in range(1, 401):
        g.copy_(torch.randn(n, device="cuda", generator=gen) * scale)
        lg.adamw_step(b8, 1e-3, t)
        lg.adamw_step(b32, 1e-3, t)
    ratio = lg.adamw_state_values(v8, ev, "v").float() / v32.sqrt()
    assert abs(ratio.mean().item() - 1) < 0.02 and ratio.std().item() < 0.12


def test_refusals_and_overlaps(lg):
    say("adamw refusals")
    t = lambda dt=torch.float32, n=64: torch.zeros(n, dtype=dt, device="cuda")
    p, g, m, v = t(), t(), t(), t()
    with pytest.raises(ValueError, match="overlaps"):
        lg.adamw_bind([p], [p], [m], [v])
    with pytest.raises(ValueError, match="overlaps"):
        lg.adamw_bind([p, p], [g, g], [m, t()], [v, t()])
    lg.adamw_bind([p, t()], [g, g], [m, t()], [v, t()])        # a shared gradient is fine
    with pytest.raises(ValueError, match="entries"):
        lg.adamw_bind([p], [t(n=63)], [m], [v])
    with pytest.raises(ValueError, match="entries"):
        lg.adamw_bind([p], [g], [m], [v, v])
    with pytest.raises(ValueError, match="contiguous"):
        lg.adamw_bind([t(n=128)[::2]], [g], [m], [v])
    with pytest.raises(ValueError, match="master"):
        lg.adamw_bind([p], [g], [m], [v], master=[t()])
    with pytest.raises(ValueError, match="v_exp"):
        lg.adamw_bind([p], [g], [t(torch.uint8)], [t(torch.uint8)], m_exp=[t(torch.uint8, 2)])
    with pytest.raises(ValueError, match="m_exp"):
        lg.adamw_bind([p], [g], [t(torch.uint8)], [t(torch.uint8)], m_exp=[t(torch.uint8, 3)],
                      v_exp=[t(torch.uint8, 2)])
    with pytest.raises(ValueError, match="uint8"):
        lg.adamw_bind([p], [g], [m], [v], m_exp=[t(torch.uint8, 2)], v_exp=[t(torch.uint8, 2)])
    with pytest.raises(ValueError, match="must be"):
        lg.adamw_bind([p.half()], [g], [m], [v])
    b = lg.adamw_bind([p], [g], [m], [v])
    for kw in (dict(lr=-1.0, step=1), dict(lr=1.0, step=0), dict(lr=1.0, step=1, beta2=1.0)):
        with pytest.raises(lg._lib.LograError):
            lg.adamw_step(b, **kw)
    with pytest.raises(ValueError, match="one entry"):
        lg.adamw_step(b, 1.0, 1, grad_scale=t(n=2))
    with pytest.raises(ValueError, match="exps"):
        lg.adamw_state_values(t(torch.uint8), t(torch.uint8, 3), "m")
    # empty tensors are left out
    lg.adamw_step(lg.adamw_bind([t(n=0), p], [t(n=0), g], [t(n=0), m], [t(n=0), v]), 1e-3, 1)
    assert p.eq(0).all()


@pytest.mark.parametrize("which", ["m", "v"])
@pytest.mark.parametrize("off", [0, 1])
def test_state_values_of_every_code(lg, which, off):
    """All codes under all exponents, in whole vectors and (one entry off) not;
    the last block is short."""
    say(f"adamw values {which} off {off}")
    exps = np.repeat(np.arange(16, 256, dtype=np.uint8), 8)
    codes = np.tile(np.arange(256, dtype=np.uint8), 240)
    codes[codes == 128] = 0 if which == "m" else 128     # (the form has no -0)
    n = codes.size - 5
    q = torch.zeros(codes.size + off, dtype=torch.uint8, device="cuda")[off:off + n]
    q.copy_(torch.from_numpy(codes[:n]))
    out = lg.adamw_state_values(q, torch.from_numpy(exps).cuda(), which)
    want = oad.decode(codes[:n], exps, which)
    assert np.array_equal(f64(out), want, equal_nan=True)
    assert np.isnan(want[-251:]).all() and np.isfinite(want[:-251]).all()


@pytest.mark.parametrize("grad", ["bf16", "fp32"])
def test_nan_gradients_of_every_payload(lg, grad):
    """8-bit states: a NaN marks both states' blocks whatever its sign and its
    payload (all bits set, e.g. of memory filled with 0xFF), under any dither;
    every other block is what it is without."""
    say("adamw nan payloads", grad)
    bits = ([0x7FFF, 0xFFFF, 0xFFFE, 0x7F81, 0xFF81, 0xFFC0] if grad == "bf16" else
            [0x7FFFFFFF, 0xFFFFFFFF, 0xFFFFFFFE, 0xFFF80000, 0xFFF7FFFF, 0x7F800001, 0xFF800001,
             0xFFC00000])
    whole = torch.int16 if grad == "bf16" else torch.int32
    wrap = 1 << (16 if grad == "bf16" else 32)
    n = 64 * len(bits)
    for step in (3, 4, 5, 6):
        clean, q = (tensors([n], "bf16", grad, True, 8, 0, 9)[0] for _ in range(2))
        for i, b in enumerate(bits):
            at = 64 * i + (7 * i + step) % 32           # every other block of 32
            q["g"].view(whole)[at] = b - wrap if b >= wrap // 2 else b
        for x in (clean, q):
            lg.adamw_step(bind(lg, [x], 0.1), LR, step)
        for which in ("m", "v"):
            e = q[which + "_exp"].cpu()
            assert e[::2].eq(255).all(), (which, step, e[::2])
            assert torch.equal(e[1::2], clean[which + "_exp"].cpu()[1::2])
            got = lg.adamw_state_values(q[which], q[which + "_exp"], which).view(-1, 2, 32)
            ref = lg.adamw_state_values(clean[which], clean[which + "_exp"], which).view(-1, 2, 32)
            assert torch.isnan(got[:, 0]).all() and torch.equal(got[:, 1], ref[:, 1])


def test_bind_names_what_is_no_tensor(lg):
    say("adamw bind types")
    t = lambda: torch.zeros(64, device="cuda")
    four = [[t(), t()] for _ in range(4)]
    for i, name in enumerate("pgmv"):
        args = [list(x) for x in four]
        args[i][1] = 3.0
        with pytest.raises(TypeError, match=rf"{name}\[1\] must be a torch.Tensor"):
            lg.adamw_bind(*args)
    with pytest.raises(TypeError, match=r"p\[1\] must be a torch.Tensor"):
        lg.adamw_bind([t(), None], *four[1:])


def layout(bound, form):
    """(tensors, work-groups, steps of a work-group) of a form in a bound table:
    five 32-bit numbers a form behind two 64-bit ones."""
    return tuple(np.frombuffer(bound.table, np.int32)[4 + 5 * form:7 + 5 * form].tolist())


# from this many entries in a form on, a work-group takes four steps of 1024 (about
# 2^22 entries: 1024 work-groups)
LONG = [1, 4300007, 33, 4095, 4097, 12345, 1023, 1025, 7]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("form", range(6))
def test_long_tensors(lg, form, bits):
    """Work-groups of four steps: whole ones, ones that end inside each of their
    steps, single entries; on vector boundaries and (every other form) off them."""
    param, grad, master = FORMS[form]
    off = (form + bits // 8) % 2
    say("adamw long", param, grad, master, bits, off)
    qs = tensors(LONG, param, grad, master, bits, off, 11)
    weights = 0 if param == "fp32" else 2 if master else 1
    table = layout(bind(lg, qs, 0.1), weights * 4 + (2 if grad == "fp32" else 0) + (bits == 8))
    assert table == (len(LONG), sum(-(-n // 4096) for n in LONG), 4)
    del qs
    run_and_check(lg, LONG, param, grad, master, bits, off, [0.1, 0.0, 0.05] * 3, steps=(9,),
                  gscale=0.7 if form == 2 else None, seed=11)


@pytest.mark.parametrize("bits", [32, 8])
def test_long_and_short_work_groups_agree(lg, bits):
    """A tensor steps to the same bits in a table of long work-groups and alone in
    one of short ones (the dither counts the entries of the tensors before it)."""
    say("adamw long and short", bits)
    n = [50001, 4300800]
    a = tensors(n, "bf16", "bf16", True, bits, 0, 12)
    b = tensors(n, "bf16", "bf16", True, bits, 0, 12)[0]
    both, one = bind(lg, a, 0.1), bind(lg, [b], 0.1)
    assert layout(both, 8 + (bits == 8))[2] == 4 and layout(one, 8 + (bits == 8))[2] == 1
    for step in (1, 2):
        lg.adamw_step(both, LR, step)
        lg.adamw_step(one, LR, step)
    for k in ("p", "master", "m", "v", "m_exp", "v_exp"):
        assert b[k] is None or torch.equal(a[0][k], b[k]), k


def test_a_handle_steps_the_storage_it_was_bound_to(lg):
    """What the binding promises: tensors given other storage later are not seen, the
    old ones are kept and stepped; a new handle steps the new ones."""
    say("adamw handle and storage")
    t = lambda x: torch.full((70,), x, device="cuda")
    p, g, m, v = t(1.0), t(2.0), t(0.0), t(0.0)
    bound = lg.adamw_bind([p], [g], [m], [v])
    old_p, old_g = p.detach(), g.detach()
    p.data, g.data = t(5.0), t(-2.0)
    lg.adamw_step(bound, 0.5, 1)
    assert p.eq(5.0).all() and (old_p - 0.5).abs().max() < 1e-6
    del old_g                                     # (the handle keeps it)
    lg.adamw_step(bound, 0.5, 2)
    assert p.eq(5.0).all() and old_p.abs().max() < 1e-6
    m.zero_()
    v.zero_()
    lg.adamw_step(lg.adamw_bind([p], [g], [m], [v]), 0.5, 1)
    assert (p - 5.5).abs().max() < 1e-6 and old_p.abs().max() < 1e-6
