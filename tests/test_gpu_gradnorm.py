"""logra_grad_norm and logra_grad_clip on the GPU against the fp64 oracle.

Sums are fp64 on both sides (relative difference below 1e-12 at these sizes), so a
norm or a scale is off by its one rounding to fp32: half a step, u = 2^-24.
"""
import numpy as np
import pytest
import torch

from oracle import gradnorm as onorm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import rank_gradient_sketching_amd as m
    return m


def tensors(sizes, dtypes, seed=0, scale=1.0):
    rng = np.random.default_rng(seed)
    return [torch.from_numpy(rng.standard_normal(n, dtype=np.float32) * np.float32(scale)).to(t).cuda()
            for n, t in zip(sizes, dtypes)]


def f64(t):
    return t.detach().double().cpu().numpy()


def near(got, ref):
    got = got.item() if isinstance(got, torch.Tensor) else got
    return got == ref or abs(got - ref) <= 1.001 * U * abs(ref) or (np.isnan(got) and np.isnan(ref))


SETS = {
    "one entry": ([1], [F32]),
    "odd": ([1, 3, 7, 8, 9, 31, 33, 1023, 1025], [F32, BF] * 5),
    "empty among": ([0, 5, 0, 0, 4097, 0], [F32, BF] * 3),
    "a chunk and around": ([4095, 4096, 4097, 8191, 8192, 8193, 16385], [F32, BF] * 4),
    "many": ([17 + 5 * i for i in range(300)], [F32, BF] * 150),
    "long": ([5_000_001, 3_000_003], [BF, F32]),
}


@pytest.mark.parametrize("name", SETS)
@pytest.mark.parametrize("kind", [2, "inf"])
def test_norm_matches_the_oracle(lg, name, kind):
    gs = tensors(*SETS[name], seed=1)
    b = lg.grad_norm_bind(gs)
    assert len(b) == len(gs)
    for max_norm, s in ((None, None), (0.5, None), (1e9, 0.25), (0.25, -0.125), (0.0, 3.0)):
        st = None if s is None else torch.tensor([s], device="cuda")
        got = lg.grad_norm(b, max_norm=max_norm, grad_scale=st, norm_type=kind, per_tensor=True)
        ref = onorm.norm([f64(g) for g in gs], np.inf if max_norm is None else max_norm,
                         1.0 if s is None else s, kind)
        assert near(got.norm, ref[0]) and near(got.scale, ref[1])
        assert all(near(x, y) for x, y in zip(got.norms.tolist(), ref[2]))


def test_unaligned_tensors(lg):
    flat = tensors([9001, 9001], [F32, BF], seed=2)
    gs = [flat[0][1:4001], flat[0][4002:], flat[1][3:5000], flat[1][5001:]]
    got = lg.grad_norm(lg.grad_norm_bind(gs))
    assert near(got.norm, onorm.norm([f64(g) for g in gs])[0])


@pytest.mark.parametrize("scale", [3e38, 1e-38, 1e-42, 1e19, 1e-23])
def test_ends_of_the_range(lg, scale):
    """Squares far past fp32's range, both ways."""
    g = torch.tensor([scale, -scale, scale, 0.0], device="cuda")
    got = lg.grad_norm(lg.grad_norm_bind([g, g[:1].to(BF)]), max_norm=scale / 2)
    ref = onorm.norm([f64(g), f64(g[:1].to(BF))], scale / 2)
    if ref[0] > 3.4028235e38:
        assert got.norm.item() == np.inf
    elif ref[0] > 2e-38:
        assert near(got.norm, ref[0])
    else:
        assert abs(got.norm.item() - ref[0]) <= 2.0 ** -149
    assert near(got.scale, ref[1])


def test_nan_and_infinity(lg):
    for kind in (2, "inf"):
        for bad, dtype in ((float("nan"), F32), (float("nan"), BF), (-float("nan"), F32)):
            gs = tensors([100, 5000], [F32, dtype], seed=3)
            gs[1][4321] = bad
            gs[0][5] = float("inf")
            got = lg.grad_norm(lg.grad_norm_bind(gs), 1.0, norm_type=kind, per_tensor=True)
            assert got.norm.isnan() and got.scale.isnan()
            assert got.norms[0] == float("inf") and got.norms[1].isnan()
        gs = tensors([100, 5000], [F32, BF], seed=3)
        gs[1][7] = -float("inf")
        got = lg.grad_norm(lg.grad_norm_bind(gs), 1.0, norm_type=kind)
        assert got.norm == float("inf") and got.scale == 0
        got = lg.grad_norm(lg.grad_norm_bind(gs), None, norm_type=kind)
        assert got.norm == float("inf") and got.scale == 1


@pytest.mark.parametrize("gt", [BF, F32])
@pytest.mark.parametrize("ot", [None, BF, F32])
@pytest.mark.parametrize("offset", [0, 1])
def test_clip(lg, gt, ot, offset):
    sizes = [1, 6, 4096, 40001, 0, 255]
    gs = [t[offset:] for t in tensors([n + offset for n in sizes], [gt] * 6, seed=4)]
    outs = None if ot is None else [torch.full((n + offset,), 9.0, device="cuda", dtype=ot)[offset:]
                                    for n in sizes]
    before = [g.clone() for g in gs]
    b = lg.grad_norm_bind(gs, out=outs)
    scale = lg.grad_norm(b, max_norm=3.0).scale
    lg.grad_clip(b, scale)
    for g, old, o in zip(gs, before, gs if outs is None else outs):
        assert torch.equal(o, (old.float() * scale).to(o.dtype))    # one rounding of fp32's product
        if outs is not None:
            assert torch.equal(g, old)
    if outs is None:           # now within the norm, up to the types' rounding
        assert lg.grad_norm(b).norm.item() <= 3.0 * (1 + 2.0 ** -8)


def test_scale_of_one_leaves_bits(lg):
    g = torch.tensor([float("nan"), 1.0, -0.0, 1e-42], device="cuda")
    bits = g.view(torch.int32).clone()
    b = lg.grad_norm_bind([g])
    lg.grad_clip(b, torch.ones(1, device="cuda"))
    assert torch.equal(g.view(torch.int32), bits)
    lg.grad_clip(b, torch.full((1,), 0.5, device="cuda"))
    assert g[1] == 0.5 and g[0].isnan()


def test_neighbours_are_left_alone(lg):
    flat = torch.ones(10000, device="cuda", dtype=BF)
    b = lg.grad_norm_bind([flat[8:4001], flat[4003:9990]])
    lg.grad_clip(b, torch.full((1,), 2.0, device="cuda"))
    want = torch.full_like(flat, 2.0)
    want[:8] = want[4001:4003] = want[9990:] = 1.0
    assert torch.equal(flat, want)


def test_bits_graph_and_streams(lg):
    gs = tensors([100_000, 33, 7000], [BF, F32, F32], seed=5)
    outs = [torch.empty_like(g) for g in gs]
    b = lg.grad_norm_bind(gs, out=outs)
    one = torch.tensor([0.5], device="cuda")
    ref = lg.grad_norm(b, 1.0, one, per_tensor=True)
    lg.grad_clip(b, ref.scale)
    want = [o.clone() for o in outs]
    res = lg.GradNorm(*(torch.empty_like(x) for x in ref))
    ws = torch.empty(b.ws_bytes, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lg.grad_norm(b, 1.0, one, per_tensor=True, out=res, ws=ws)
        lg.grad_clip(b, res.scale)
    other = lg.grad_norm_bind(tensors([50_000], [F32], seed=6))
    for rep in range(4):
        for o in (*outs, *res):
            o.zero_()
        lg.grad_norm(other, ws=ws if other.ws_bytes <= b.ws_bytes else None)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(res, ref))
        assert all(torch.equal(x, y) for x, y in zip(outs, want))
    with torch.cuda.stream(torch.cuda.Stream()):
        again = lg.grad_norm(b, 1.0, one, per_tensor=True)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(again, ref))


def test_sketch_norm_estimates_the_gradients(lg):
    """E ||S||^2 = ||G||^2: the norm of a sketch over many bases is near the gradient's."""
    T, d, k, r = 64, 96, 256, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    X, dY = (torch.randn(T, c, device="cuda", generator=g).to(BF) for c in (k, d))
    G = np.linalg.norm(f64(dY).T @ f64(X))
    squares = []
    for seed in range(24):
        S = torch.empty(d, r, device="cuda")
        lg.sketch_accumulate(X, dY, S, seed, overwrite=True)
        squares.append(lg.grad_norm(lg.grad_norm_bind([S])).norm.item() ** 2)
    # one sketch's square spreads by at most sqrt(2 / r) of it: four deviations of 24
    assert abs(np.mean(squares) / G ** 2 - 1) < 4 * np.sqrt(2 / r / 24)


@pytest.mark.parametrize("gt,ot", [(BF, None), (BF, F32), (F32, BF), (F32, None)])
def test_clip_past_the_caches(lg, gt, ot):
    """Enough gradients (128 MiB) for the loads and stores that pass the caches, beside a
    small tensor; products of fp32 rounded once, as torch's own."""
    n = (72_000_005 if gt == BF else 36_000_003)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    gs = [torch.randn(m, device="cuda", generator=g).to(gt) for m in (n, 13)]
    want = [(x.float() * 0.375).to(ot or gt) for x in gs]
    outs = None if ot is None else [torch.full_like(x, float("nan"), dtype=ot) for x in gs]
    b = lg.grad_norm_bind(gs, out=outs)
    norm = lg.grad_norm(b).norm.item()
    ref = np.sqrt(sum(float(x.double().square().sum()) for x in gs))
    assert abs(norm - ref) <= 1.001 * U * ref
    lg.grad_clip(b, torch.tensor([0.375], device="cuda"))
    assert all(torch.equal(x, w) for x, w in zip(gs if ot is None else outs, want))


def test_handle_keeps_the_storage(lg):
    """Gradients that the caller drops (or gives other storage) are still the handle's."""
    gs = tensors([100_003, 77], [F32, BF], seed=12)
    ref = onorm.norm([f64(g) for g in gs])[0]
    b = lg.grad_norm_bind(gs)
    gs[0].data = torch.zeros(5, device="cuda")
    del gs
    other = [torch.full((100_003,), 9.0, device="cuda") for _ in range(4)]
    assert near(lg.grad_norm(b).norm, ref)
    del other
