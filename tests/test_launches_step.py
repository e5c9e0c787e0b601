"""Launches of the operators that close a policy step, followed on the CPU
(launches.py): grids of the largest sizes."""
import pytest

from launches import follow
from linear_kernel_shapes import BIAS_SHAPES, FORMS, SHAPES, form_of, has

A, B, C, D, E, F, G, W = (0x10000000000000 * i for i in range(1, 9))   # 2^52 bytes apart
TOP = (1 << 31) - 1
MANY = 1 << 50           # bytes of scratch


@pytest.fixture(scope="module")
def folder(tmp_path_factory):
    return tmp_path_factory.mktemp("launches")


def up(x, m):
    return -(-x // m) * m


def act(T, d, act=0, dY=C, d_bias=D, d_type=0, d_out=A):
    ld = up(d, 8)
    return ("logra_linear_backward_act",
            [d_out, d_type, ld, B if act else None, ld, act, T, d, dY, ld, d_bias, W, MANY, None])


@pytest.mark.parametrize("d", [TOP, TOP - 1, (1 << 31) - 255, (1 << 31) - 256, (1 << 31) - 257, 10241])
def test_activation_gradient_of_wide_rows(folder, d):
    """The columns' work-groups, also where d and their rounding up pass 2^31 together."""
    for call in (act(1, d), act(1, d, act=3), act(1, d, dY=None), act(1, d, d_bias=None),
                 act(1, d, d_type=1, act=1)):
        (st, (first, *rest)), = follow([call], folder)
        assert st == 0 and "act_grad_kernel" in first.name and not rest
        assert first.grid == (up(d, 256) // 256, 1, 1) and first.block == (256, 1, 1)


def test_bias_join_of_wide_rows(folder):
    for d in (TOP, (1 << 31) - 64, (1 << 31) - 63):
        # (strips of 256 columns enough for the chip, so rows are cut only where they pass 2^30)
        (st, (first, join)), = follow([act((1 << 30) + 8, d, dY=None, d_out=1 << 61)],
                                        folder)
        assert st == 0 and "bias_join_kernel" in join.name
        assert first.grid == (up(d, 256) // 256, 2, 1)
        assert join.grid == (up(d, 64) // 64, 1, 1)


SIZES = [1, 16, 17, 255, 257, 5000, 152064, (1 << 20) + 1, 1 << 24, TOP - 300, TOP]


def test_grids_of_all_sizes(folder):
    """Every accepted size gives grids that a launch can have (2^32 threads, 65535 along y
    and z); those refused are refused before anything is launched."""
    calls = []
    for a in SIZES:
        for b in SIZES:
            ld = up(b, 8)
            calls.append(act(a, b, act=2))
            calls.append(("logra_sample_tokens", [A, 0, a, b, ld, B, 1.0, 0, 1.0, 0.0, None, None,
                                                  None, None, C, D, E, F, W, MANY, None]))
            for c in SIZES:
                lc = up(c, 8)
                calls.append(("logra_linear", [A, lc, B, lc, a, b, c, C, 1, 2, D, ld, E, 1, ld, F,
                                               ld, W, MANY, None]))
                calls.append(("logra_linear_backward_input", [A, ld, B, lc, a, b, c, None, 0, C, lc,
                                                              W, MANY, None]))
                calls.append(("logra_linear_backward_weight", [A, ld, B, lc, a, b, c, 1, C, 1, lc,
                                                               W, MANY, None]))
    taken = 0
    for (name, args), (st, launches) in zip(calls, follow(calls, folder)):
        assert (st == 0) == (len(launches) > 0), (name, args, st)
        taken += st == 0
        for x in launches:
            threads = x.grid[0] * x.block[0]
            assert 0 < threads < 1 << 32 and max(x.grid[1:]) <= 65535, (name, args, x)
            assert x.block[0] <= 1024 and x.block[1:] == (1, 1)
    assert taken > len(calls) // 2


def test_many_rows_of_draws(folder):
    """Rows past 2^22 are cut into several launches."""
    calls = [("logra_sample_tokens", [A, 0, n, 8, 8, B, 1.0, 0, 1.0, 0.0, None, None, None, None, C,
                                      None, None, None, None, 0, None])
             for n in ((1 << 22) - 1, 1 << 22, (1 << 22) + 1, TOP)]
    for (_, args), (st, launches) in zip(calls, follow(calls, folder)):
        assert st == 0 and sum(x.grid[0] for x in launches) == args[2]
        assert all(x.grid[0] <= 1 << 22 for x in launches)


BF16, F32 = 0, 1
MIB = 1 << 20


@pytest.mark.parametrize("grads,past", [
    ([[100, F32]] * 4096, False),                       # 1.6 MB: a work-group each, but few bytes
    ([[1536, F32]] * 5000, False),
    ([[1, BF16]] * 20000, False),
    ([[16 * MIB, BF16], [24 * MIB - 1, F32]], False),   # one entry short of 128 MiB
    ([[16 * MIB, BF16], [24 * MIB, F32]], True),
    ([[64 * MIB - 1, BF16]], False),
    ([[64 * MIB, BF16]], True),
    ([[4 * MIB, F32]] * 8 + [[0, F32]] * 9, True),
    ([[152064 * 1536, BF16]], True),
], ids=lambda x: str(x) if isinstance(x, bool) else f"{len(x)}x{x[0]}")
def test_clip_passes_the_caches_from_128_mib(folder, grads, past):
    (st, (clip,)), = follow([("logra_grad_clip", [{"grads": grads}, W, C, None])], folder)
    assert st == 0 and f"clip_kernelILb{int(past)}E" in clip.name


def test_products_reach_the_kernels_that_are_tested(folder):
    """Each shape of linear_kernel_shapes.py, in each form, goes to the kernel that it is there
    for; all of the library's product kernels are among them, split and whole."""
    cases = [(s, f) for s in SHAPES for f in FORMS if has(s, f)]
    calls = []
    for s, form in cases:
        T, d, k = form_of(s, form)
        ld, lk = up(d, 8), up(k, 8)
        calls.append({
            "forward": ("logra_linear", [A, lk, B, lk, T, d, k, None, 0, 0, None, 0, C, 1, ld, None,
                                         0, W, MANY, None]),
            "input": ("logra_linear_backward_input", [A, ld, B, lk, T, d, k, None, 0, C, lk, W, MANY,
                                                      None]),
            "weight": ("logra_linear_backward_weight", [A, ld, B, lk, T, d, k, 0, C, 1, lk, W, MANY,
                                                        None])}[form])
    for (s, form), (st, (first, *join)) in zip(cases, follow(calls, folder)):
        bits = {"forward": "Lb0ELb0E", "input": "Lb0ELb1E", "weight": "Lb1ELb1E"}[form]
        if s.kernel == "few":
            want = "few_rows_kernelE"
        elif s.kernel.startswith("64"):
            want = "tile_kernelILi%sELi%sE" % tuple(s.kernel.split("x"))
            assert first.name.split("EE")[0].endswith(bits + f"Lb{int(s.once)}"), (s, form, first)
        else:
            want = "big_kernelILi%sE%sE" % (s.kernel.split("x")[1], bits)
        assert st == 0 and want in first.name, (s, form, first)
        assert [("join_kernel" in x.name) for x in join] == [True] * s.split, (s, form, join)
    kinds = {(s.kernel, s.once, s.split) for s in SHAPES}
    assert kinds == {("few", False, False)} | {
        (t, o, p) for t in ("64x64", "64x128", "256x128", "256x256") for p in (False, True)
        for o in ((False, True) if t.startswith("64") else (False,))}


def test_bias_gradients_reach_the_kernels_that_are_tested(folder):
    for T, d, strips, chunks in BIAS_SHAPES:
        for kind in (BF16, F32):
            (st, (first, *join)), = follow([act(T, d, act=2, d_type=kind)], folder)
            cols, threads = (256, 256) if strips else (16, 512)
            assert st == 0 and (f"act_grad_kernelILi2ELb{kind}ELi{cols // 8}ELi{threads}E"
                                in first.name), (T, d)
            assert first.grid == (up(d, cols) // cols, chunks, 1), (T, d, first)
            assert ["bias_join_kernel" in x.name for x in join] == [True] * (chunks > 1)
