"""logra_adapter_apply on the GPU against the fp64 oracle.

Tolerance of an output: its rounding to bf16, 2^-8 of the value; beside it, in
units of M = |scale| |X| |A|^T |U|^T (sums of magnitudes): P = X A^T is a sum of
k products in fp32, k 2^-24 at most; P, and an fp32 U, enter as pairs of 16
significant bits, 2^-16 each; lo x lo, 2^-16, is left out; the second sum has r
terms of up to three products, and c, scale and the pieces of k a few roundings
more: (k + 3 r + 64) 2^-24 + 3 2^-16.
"""
import numpy as np
import pytest
import torch

from oracle import adapter as oad
from oracle import projection as oproj

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rank_gradient_sketching_amd as m
    return m


def say(*a):
    print(*a, flush=True)


def padded(t, extra=0):
    n, c = t.shape
    buf = torch.full((n, -(-c // 8) * 8 + 8 * extra), float("nan"), dtype=t.dtype, device="cuda")
    buf[:, :c] = t.cuda()
    return buf[:, :c]


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def normal(shape, seed, sigma=1.0, dtype=torch.bfloat16):
    rng = np.random.default_rng([seed, *shape])
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * np.float32(sigma)).to(dtype)


def case(T, k, d, r, n, signs, u_dtype, rows, seed=0):
    rng = np.random.default_rng([seed, T, k, d, r, n])
    c = dict(X=padded(normal((T, k), 1), T % 2), Y=padded(normal((T, d), 2), 1),
             U=normal((n, d, r), 3, 15.0, u_dtype).cuda(),
             scale=torch.from_numpy((-2e-4 * (0.5 + rng.random(n))).astype(np.float32)).cuda())
    if rows == "mixed":
        ids = rng.integers(-1, n, T)
    elif rows == "one":
        ids = np.full(T, n - 1)
    else:
        ids = np.sort(rng.integers(0, n, T))
    c["adapter"] = torch.from_numpy(ids.astype(np.int32)).cuda()
    if signs:
        seeds = rng.integers(0, 1 << 62, (n, 2))
        c["seeds"] = torch.from_numpy(seeds).cuda()
        c["ref_A"] = [oproj.projection(int(s), int(t), 0, r, k) for s, t in seeds]
    else:
        A = normal((n * r, k), 4, 1 / np.sqrt(r))
        c["A"] = padded(A, 1).unflatten(0, (n, r))
        c["ref_A"] = list(f64(A).reshape(n, r, k))
    return c


def apply(lg, c, **kw):
    return lg.adapter_apply(c["X"], c["Y"], c["adapter"], c["U"], c["scale"], seeds=c.get("seeds"),
                            A=c.get("A"), **kw)


def check(c, out, rows=None):
    T, k = c["X"].shape
    r = c["U"].shape[2]
    X, Y, U = f64(c["X"]), f64(c["Y"]), f64(c["U"])
    ref, M = oad.apply(X, Y, c["adapter"].cpu().numpy(), U, c["ref_A"], f64(c["scale"]))
    tol = 2.0 ** -8 * np.abs(ref) + M * ((k + 3 * r + 64) * 2.0 ** -24 + 3 * 2.0 ** -16) + 1e-37
    err = np.abs(f64(out) - ref)
    if rows is not None:
        err, tol = err[rows], tol[rows]
    assert np.all(err <= tol), float(np.max(err / tol))


SHAPES = [
    # T, k, d, r, n, rows
    (1, 1, 1, 1, 1, "one"), (1, 4096, 4096, 64, 3, "one"), (2, 37, 65, 3, 2, "mixed"),
    (15, 256, 64, 4, 4, "mixed"), (16, 255, 63, 16, 16, "mixed"), (17, 257, 72, 17, 2, "mixed"),
    (33, 1000, 130, 32, 5, "mixed"), (64, 520, 264, 33, 8, "runs"), (100, 776, 300, 100, 33, "mixed"),
    (200, 1536, 1000, 16, 16, "mixed"), (129, 300, 515, 128, 3, "runs"), (70, 264, 136, 250, 2, "mixed"),
    (70, 264, 136, 256, 70, "mixed"), (1030, 512, 1028, 64, 4, "runs"), (2000, 264, 2056, 8, 3, "mixed"),
    (1500, 1000, 1031, 24, 6, "runs"),
    # many rows and columns
    (4100, 264, 1100, 64, 5, "runs"), (4099, 2500, 1096, 256, 3, "runs"),
    (3000, 136, 1501, 100, 4, "mixed"), (3001, 300, 1500, 128, 9, "runs"),
    (9000, 520, 260, 32, 40, "runs"), (2100, 5000, 1024, 16, 2, "one"),
    # few rows of many policies: rows in whole fp32 lines, but not in bf16
    (40, 264, 640, 12, 40, "mixed"), (20, 520, 300, 36, 20, "mixed"), (5, 136, 70, 132, 3, "mixed"),
    (1, 600, 1030, 252, 1, "one"), (130, 264, 2050, 20, 12, "mixed"),
    (200, 5000, 520, 200, 7, "mixed"), (128, 300, 64, 64, 128, "mixed"),
]


@pytest.mark.parametrize("u_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("signs", [True, False])
@pytest.mark.parametrize("T,k,d,r,n,rows", SHAPES)
def test_apply(lg, T, k, d, r, n, rows, signs, u_dtype):
    say("adapter", T, k, d, r, n, rows, signs, u_dtype)
    c = case(T, k, d, r, n, signs, u_dtype, rows)
    out = padded(torch.zeros(T, d, dtype=torch.bfloat16), 2)
    pad = out._base[:, d:].clone().view(torch.int16)
    got = apply(lg, c, out=out)
    assert got is out
    check(c, out)
    assert torch.equal(out._base[:, d:].clone().view(torch.int16), pad)
    # rows without a policy keep their bits
    none = (c["adapter"] < 0)
    assert torch.equal(out[none].view(torch.int16), c["Y"][none].view(torch.int16))
    # in place, same bits
    Y = padded(c["Y"].cpu(), 1)
    same = lg.adapter_apply(c["X"], Y, c["adapter"], c["U"], c["scale"], seeds=c.get("seeds"),
                            A=c.get("A"))
    assert same is Y and torch.equal(Y.view(torch.int16) if Y.is_contiguous() else
                                     Y.contiguous().view(torch.int16), out.contiguous().view(torch.int16))


def test_rows_do_not_touch_each_other(lg):
    """NaN and infinite rows, policies and ids out of range: every other row is
    what it is without them; nor does their order matter where k has two pieces (a
    sum of two)."""
    say("adapter isolation")
    c = case(50, 300, 200, 16, 5, True, torch.float32, "mixed", seed=1)
    ref = apply(lg, c, out=torch.empty_like(c["Y"])).clone()
    bad = dict(c, X=c["X"].clone(), Y=c["Y"].clone(), U=c["U"].clone(), adapter=c["adapter"].clone())
    bad["X"] = padded(c["X"].cpu())
    bad["X"][7] = float("nan")
    bad["X"][20, 3] = float("inf")
    bad["U"][2] = float("nan")
    bad["adapter"][30] = 5
    bad["adapter"][31] = -2 ** 31
    bad["adapter"][32] = 2 ** 31 - 1
    got = apply(lg, bad, out=torch.empty_like(c["Y"]))
    ok = torch.ones(50, dtype=torch.bool, device="cuda")
    ok[[7, 20, 30, 31, 32]] = False
    ok &= c["adapter"] != 2
    assert torch.equal(got[ok].view(torch.int16), ref[ok].view(torch.int16))
    assert torch.equal(got[30:33].view(torch.int16), c["Y"][30:33].view(torch.int16))
    assert torch.isnan(got[7]).all() or bad["adapter"][7] < 0
    perm = torch.from_numpy(np.random.default_rng(0).permutation(50)).cuda()
    p = dict(c, X=padded(c["X"][perm].cpu()), Y=padded(c["Y"][perm].cpu()), adapter=c["adapter"][perm].contiguous())
    assert torch.equal(apply(lg, p).contiguous().view(torch.int16), ref[perm].contiguous().view(torch.int16))


@pytest.mark.parametrize("T,k,d,r,n", [(1, 1, 8, 1, 1), (5, 37, 65, 3, 2), (40, 255, 72, 17, 5),
                                       (70, 1041, 264, 100, 9), (33, 777, 128, 250, 3),
                                       (612, 2601, 72, 40, 33)])
@pytest.mark.parametrize("off", [0, 1, 2])
def test_bases_on_any_boundary(lg, T, k, d, r, n, off):
    """Given bases packed without padding (odd k: rows on 2-byte boundaries)
    and starting inside an allocation: the bits of the padded ones."""
    say(f"adapter bases at {off}: {T} {k} {d} {r} {n}")
    c = case(T, k, d, r, n, False, torch.float32, "mixed", seed=off)
    to = padded(torch.zeros(T, d, dtype=torch.bfloat16))
    ref = apply(lg, c, out=to).contiguous().view(torch.int16).clone()
    flat = torch.full((n * r * k + off,), float("nan"), dtype=torch.bfloat16, device="cuda")
    A = flat[off:].view(n, r, k)
    A.copy_(c["A"])
    to.zero_()
    got = apply(lg, dict(c, A=A), out=to).contiguous().view(torch.int16)
    assert torch.equal(got, ref)


@pytest.mark.parametrize("signs", [True, False])
def test_same_bits_again_and_inside_a_tile(lg, signs):
    """The same call twice, and rows that trade places inside their tiles of 32."""
    say(f"adapter order inside tiles signs {signs}")
    for T, k, d, r, n in ((90, 5000, 200, 64, 7), (1100, 2600, 1100, 32, 5)):
        c = case(T, k, d, r, n, signs, torch.float32, "mixed", seed=T)
        to = padded(torch.zeros(T, d, dtype=torch.bfloat16))
        out = lambda q: apply(lg, q, out=to).contiguous().view(torch.int16)
        ref = out(c).clone()
        to.zero_()
        assert torch.equal(out(c), ref)
        rng = np.random.default_rng(T)
        perm = np.concatenate([t + rng.permutation(min(32, T - t)) for t in range(0, T, 32)])
        perm = torch.from_numpy(perm).cuda()
        p = dict(c, X=padded(c["X"][perm].cpu()), Y=padded(c["Y"][perm].cpu()),
                 adapter=c["adapter"][perm].contiguous())
        assert torch.equal(out(p), ref[perm])


def test_signed_zeros_and_nan_bits_of_base_rows(lg):
    say("adapter base rows")
    T, d = 40, 72
    Y = torch.zeros(T, d, dtype=torch.bfloat16)
    Y[::2] = -0.0
    Y[5] = float("nan")
    Y = padded(Y)
    ids = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    out = torch.empty_like(Y)
    lg.adapter_apply(padded(normal((T, 64), 1)), Y, ids, torch.zeros(1, d, 8, device="cuda"),
                     torch.ones(1, device="cuda"), seeds=torch.zeros(1, 2, dtype=torch.int64, device="cuda"),
                     out=out)
    assert torch.equal(out.contiguous().view(torch.int16), Y.contiguous().view(torch.int16))


@pytest.mark.parametrize("kind", [0, 1])
def test_equals_the_merge(lg, kind):
    """Y = X W^T with an unmerged update against X W'^T with W' of logra_merge:
    W' is rounded to bf16 (2^-8 of each weight), which dominates."""
    say("adapter against merge", kind)
    T, d, k, r, seed = 64, 200, 512, 32, 77
    X, W = padded(normal((T, k), 1)), padded(normal((d, k), 2, 0.02))
    S = normal((d, r), 3, 15.0, torch.float32).cuda()
    eta = 2e-4
    W2 = padded(W.cpu())
    lg.merge(W2, S, seed, 1, kind, 1.0, eta)
    Y = padded((f64t(X) @ f64t(W).t()).to(torch.bfloat16))
    args = (dict(seeds=torch.tensor([[seed, 1]], device="cuda")) if kind == 0 else
            dict(A=lg.regen_A(seed, 1, 1, r, k).to(torch.bfloat16)[None]))
    out = lg.adapter_apply(X, Y, torch.zeros(T, dtype=torch.int32, device="cuda"), S[None],
                           torch.tensor([-eta], device="cuda"), out=torch.empty_like(Y), **args)
    want = f64t(X) @ f64t(W2).t()
    tol = 2.0 ** -8 * (f64t(X).abs() @ f64t(W2).abs().t()) + 2.0 ** -7 * (want.abs() + Y.cpu().double().abs())
    assert ((out.cpu().double() - want).abs() <= tol).all()


def f64t(t):
    return t.detach().cpu().double()


def test_workspace_streams_and_empty(lg):
    say("adapter workspace, stream")
    c = case(90, 520, 300, 24, 4, True, torch.float32, "mixed", seed=2)
    ref = apply(lg, c, out=padded(torch.zeros(90, 300, dtype=torch.bfloat16)))
    torch.cuda.synchronize()
    ws = torch.full((lg.adapter_ws_bytes(90, 300, 520, 24),), 0xFF, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = apply(lg, c, out=padded(torch.zeros(90, 300, dtype=torch.bfloat16)), ws=ws)
    side.synchronize()
    assert torch.equal(got.contiguous().view(torch.int16), ref.contiguous().view(torch.int16))
    e = lambda cols: torch.empty(0, cols, dtype=torch.bfloat16, device="cuda")
    out = lg.adapter_apply(e(520), e(300), c["adapter"][:0], c["U"], c["scale"], seeds=c["seeds"])
    assert out.shape == (0, 300)


def test_refusals(lg):
    say("adapter refusals")
    c = case(8, 64, 64, 8, 2, True, torch.float32, "mixed")
    def call(**kw):
        a = dict(X=c["X"], Y=c["Y"], adapter=c["adapter"], U=c["U"], scale=c["scale"], seeds=c["seeds"])
        a.update(kw)
        return lg.adapter_apply(**a)
    A = torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    for kw, match in [(dict(seeds=None), "seeds"), (dict(A=A), "seeds"),
                      (dict(adapter=c["adapter"].long()), "adapter"), (dict(adapter=c["adapter"][:4]), "adapter"),
                      (dict(scale=c["scale"][:1]), "scale"), (dict(U=c["U"][:, :63].contiguous()), "columns"),
                      (dict(U=c["U"].transpose(1, 2)), "contiguous"), (dict(Y=c["Y"][:4]), "rows"),
                      (dict(X=c["X"].float()), "X must be"), (dict(seeds=c["seeds"].int()), "seeds"),
                      (dict(seeds=None, A=A[:, :4]), "A must"), (dict(seeds=None, A=A.float()), "A must"),
                      (dict(out=c["Y"].float()), "out must"),
                      (dict(seeds=None, A=torch.zeros(2, 9, 64, dtype=torch.bfloat16, device="cuda")[:, :8]),
                       "rows apart")]:
        with pytest.raises(ValueError, match=match):
            call(**kw)
    with pytest.raises(lg._lib.LograError):
        call(ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(lg._lib.LograError):
        call(out=c["X"])                              # out over X


@pytest.mark.parametrize("basis", ["signs", "rows", "any rows"])
@pytest.mark.parametrize("k", [2 ** 31 - 1, 2 ** 31 - 255])
def test_the_longest_rows(lg, k, basis):
    """k up to the last one accepted, where the chunk count and a column past the
    last chunk pass 31 bits.  X is zero but for some columns, so the oracle needs
    only those of A; X and A end in NaN padding where their rows have any."""
    say("adapter longest rows", k, basis)
    from oracle.philox import philox4x64_10_np
    T, d, r, seed = 2, 24, 2, 91
    cols = np.array([0, 1, 255, 256, 2 ** 30 + 3, k - 600, k - 257, k - 256, k - 200, k - 9, k - 2, k - 1])
    at = torch.from_numpy(cols).cuda()
    X = torch.zeros(T, 2 ** 31, dtype=torch.bfloat16, device="cuda")
    X[:, k:] = float("nan")
    X[:, at] = normal((T, len(cols)), 1).cuda()
    U, Y = normal((1, d, r), 3, 15.0, torch.float32).cuda(), padded(normal((T, d), 2))
    args = {}
    if basis == "signs":
        j = cols.astype(np.uint64)
        words = np.stack(philox4x64_10_np((j >> np.uint64(8))[None], np.arange(r, dtype=np.uint64)[:, None],
                                          np.uint64(0), np.uint64(0), seed, 0), axis=-1)
        word = np.take_along_axis(words, ((cols >> 6) & 3)[None, :, None], axis=2)[:, :, 0]
        A = (1.0 - 2.0 * ((word >> (j & np.uint64(63))[None]) & np.uint64(1)).astype(np.float64)) / np.sqrt(r)
        args["seeds"] = torch.tensor([[seed, 0]], device="cuda")
    else:
        # (rows k apart start on any boundary)
        full = torch.zeros(r * (k if basis == "any rows" else 2 ** 31), dtype=torch.bfloat16,
                           device="cuda").view(1, r, -1)
        full[:, :, k:] = float("nan")
        full[0, :, at] = normal((r, len(cols)), 4).cuda()
        A, args["A"] = f64(full[0, :, at]), full[:, :, :k]
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    out = lg.adapter_apply(X[:, :k], Y, ids, U, torch.ones(1, device="cuda"),
                           out=padded(torch.zeros(T, d, dtype=torch.bfloat16)), **args)
    ref, M = oad.apply(f64(X[:, at]), f64(Y), np.zeros(T, int), f64(U), [A], np.ones(1))
    tol = 2.0 ** -8 * np.abs(ref) + M * ((len(cols) + 3 * r + 64) * 2.0 ** -24 + 3 * 2.0 ** -16)
    assert np.all(np.abs(f64(out) - ref) <= tol)
    assert np.abs(ref - f64(Y)).max() > 1                 # (an update that is seen)


# The kernels of many rows: from 8192 blocks of 16 rows x 64 columns on, those of
# rank up to 64 whose rows of U lie on 16-byte boundaries by adapter_rows_kernel,
# others by adapter_strip_kernel.  k of 2600 and more is cut into pieces.
MANY = [
    # kernel, T, k, d, r, n, rows, U's type, entries U lies off a boundary
    ("rows", 8201, 136, 1100, 8, 5, "runs", "bf16", 0),
    ("rows", 8201, 264, 1100, 64, 5, "mixed", "fp32", 0),
    ("rows", 2500, 2600, 3400, 32, 3, "mixed", "bf16", 0),
    ("rows", 2500, 2600, 3400, 40, 8, "runs", "fp32", 0),
    ("rows", 600, 5000, 17000, 64, 6, "runs", "bf16", 0),
    ("rows", 9000, 300, 1031, 16, 1, "one", "fp32", 0),
    ("rows", 33000, 136, 260, 4, 40, "mixed", "fp32", 0),
    ("rows", 16500, 136, 515, 64, 300, "runs", "fp32", 0),
    ("strip", 8201, 136, 1100, 24, 5, "mixed", "bf16", 3),
    ("strip", 8201, 264, 1100, 64, 5, "runs", "fp32", 1),
    ("strip", 2500, 2600, 3400, 100, 8, "runs", "bf16", 0),
    ("strip", 2500, 2600, 3400, 100, 3, "mixed", "fp32", 0),
    ("strip", 600, 5000, 17000, 256, 6, "runs", "fp32", 0),
    ("strip", 9000, 300, 1031, 128, 1, "one", "bf16", 0),
    ("strip", 8201, 136, 1100, 128, 33, "mixed", "fp32", 0),
    ("strip", 33000, 136, 260, 250, 12, "runs", "fp32", 0),
    ("strip", 16500, 136, 515, 7, 40, "mixed", "fp32", 0),
]


@pytest.mark.parametrize("signs", [True, False])
@pytest.mark.parametrize("kernel,T,k,d,r,n,rows,u_type,off", MANY)
def test_many_rows(lg, kernel, T, k, d, r, n, rows, u_type, off, signs):
    say("adapter many rows", kernel, T, k, d, r, n, rows, u_type, off, signs)
    u_dtype = torch.float32 if u_type == "fp32" else torch.bfloat16
    vec = r % (4 if u_type == "fp32" else 8) == 0 and off == 0
    assert -(-T // 16) * -(-d // 64) >= 8192
    assert kernel == ("rows" if vec and r <= 64 else "strip")
    c = case(T, k, d, r, n, signs, u_dtype, rows)
    if off:
        U = torch.empty(c["U"].numel() + off, dtype=u_dtype, device="cuda")[off:].view_as(c["U"])
        c["U"] = U.copy_(c["U"])
    out = padded(torch.zeros(T, d, dtype=torch.bfloat16), 2)
    pad = out._base[:, d:].clone().view(torch.int16)
    apply(lg, c, out=out)
    check(c, out)
    bits = out.contiguous().view(torch.int16)
    assert torch.equal(out._base[:, d:].clone().view(torch.int16), pad)
    none = c["adapter"] < 0
    assert torch.equal(bits[none], c["Y"].contiguous().view(torch.int16)[none])
    # in place, the same bits
    Y = padded(c["Y"].cpu(), 1)
    same = lg.adapter_apply(c["X"], Y, c["adapter"], c["U"], c["scale"], seeds=c.get("seeds"),
                            A=c.get("A"))
    assert same is Y and torch.equal(Y.contiguous().view(torch.int16), bits)
    assert Y._base[:, d:].isnan().all()


@pytest.mark.parametrize("r", [32, 128])
def test_many_rows_do_not_touch_each_other(lg, r):
    """NaN and infinite rows, a NaN policy and indices out of range among many rows:
    every other row is what it is without them."""
    say("adapter many rows, isolation", r)
    T, d = 8300, 1100
    c = case(T, 264, d, r, 5, True, torch.float32, "mixed", seed=3)
    to = padded(torch.zeros(T, d, dtype=torch.bfloat16))
    ref = apply(lg, c, out=to).contiguous().view(torch.int16).clone()
    bad = dict(c, X=padded(c["X"].cpu()), U=c["U"].clone(), adapter=c["adapter"].clone())
    bad["X"][7::100] = float("nan")
    bad["X"][20::100, 3] = float("inf")
    bad["U"][2] = float("nan")
    out_of = torch.arange(31, T, 100, device="cuda")
    bad["adapter"][out_of] = torch.tensor([5, -2 ** 31, 2 ** 31 - 1, 77], dtype=torch.int32,
                                          device="cuda").repeat(len(out_of))[:len(out_of)]
    got = apply(lg, bad, out=to)
    ok = (c["adapter"] != 2)
    for first in (7, 20, 31):
        ok[first::100] = False
    bits = got.contiguous().view(torch.int16)
    assert torch.equal(bits[ok], ref[ok])
    assert torch.equal(bits[out_of], c["Y"].contiguous().view(torch.int16)[out_of])
    assert torch.isnan(got[(c["adapter"] == 2) & (bad["adapter"] == 2)]).all()
