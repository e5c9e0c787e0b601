"""A whole policy step through the library: the rollout's forward pass (linear
with its epilogues, adapter_apply), the drawn tokens (sample_tokens), their
loss's gradient (token_logprob, token_logprob_backward), the backward pass
(linear_backward_act, _input, _weight) into the sketches (sketch_accumulate),
the global norm over sketches and full gradients (grad_norm), AdamW with its
factor (adamw_step) and the clipped sketches (grad_clip).  Each stage is held to
the oracle on the GPU's own input of that stage.  Then the same step captured in
a HIP graph and replayed, and calls on two streams at once.

Tolerances (u = 2^-24, half a step of bf16 H = 2^-8): a sum of K exact products
in fp32 errs by at most K u M, M = sum |x w|, and passes an activation with a
slope of at most 1.13, which adds 2^-20 (|pre| + 1); a bf16 result rounds by H.
"""
import numpy as np
import pytest
import torch

from oracle import adamw as oadw
from oracle import adapter as oadp
from oracle import gradnorm as onorm
from oracle import linear as olin
from oracle import logprob as olp
from oracle import projection as oproj
from oracle import sample as osample
from oracle import sketch as osketch

pytestmark = pytest.mark.gpu

U, H = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16


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


def rel_fro(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


class Step:
    """h = silu(X W1^T + b1), y = h W2^T + X (and a policy's unmerged update of W2),
    z = y head^T; W1 and W2 are sketched, b1 and head stepped by AdamW."""

    def __init__(self, lg, T=200, k=264, d=520, V=1003, r=32, n=3, seed=5, z_type=BF):
        self.lg, self.r, self.z_type, self.V = lg, r, z_type, V
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        N = lambda *s, sig=1.0: torch.randn(*s, device="cuda", generator=g) * sig
        E = lambda *s, t=BF: torch.empty(*s, dtype=t, device="cuda")
        Z = lambda c: torch.zeros(c, device="cuda")
        Vp = -(-V // 8) * 8
        self.X = N(T, k).to(BF)
        self.W1, self.W2 = N(d, k, sig=k ** -0.5).to(BF), N(k, d, sig=d ** -0.5).to(BF)
        self.b1, self.head = N(d, sig=0.1), N(V, k, sig=0.1).to(BF)
        self.kept0 = [self.b1.clone(), self.head.clone()]
        self.policy = torch.randint(-1, n, (T,), device="cuda", generator=g, dtype=torch.int32)
        self.Uu = N(n, k, r, sig=15)
        self.scale = -2e-4 * (1 + torch.rand(n, device="cuda", generator=g))
        self.keys = torch.tensor([[100 + i, i] for i in range(n)], device="cuda")
        self.u = torch.rand(T, device="cuda", generator=g)
        self.u[::17] = -1                       # sequences that have ended
        self.adv = N(T) / T
        self.pre, self.h, self.y0, self.y = E(T, d), E(T, d), E(T, k), E(T, k)
        self.z, self.dz = E(T, Vp, t=z_type)[:, :V], E(T, Vp)[:, :V]
        self.dz_z = E(T, Vp, t=z_type)[:, :V]
        F = lambda t=torch.float32: E(T, t=t)
        self.drawn = lg.SampledTokens(F(torch.int64), F(), F(), F(torch.int32))
        self.lp = lg.TokenLogprob(F(), F(), F(), None, None)
        self.dy, self.dh, self.dpre, self.dX = E(T, k), E(T, d), E(T, d), E(T, k)
        self.S1, self.S2 = E(d, r, t=torch.float32), E(k, r, t=torch.float32)
        self.g_head, self.g_b1 = E(V, k, t=torch.float32), E(d, t=torch.float32)
        self.state = [Z(d), Z(d), torch.zeros(V, k, device="cuda"), torch.zeros(V, k, device="cuda")]
        m1, v1, m2, v2 = self.state
        self.adam = lg.adamw_bind([self.b1, self.head], [self.g_b1, self.g_head], [m1, m2],
                                  [v1, v2], weight_decay=[0.0, 0.1])
        self.all = lg.grad_norm_bind([self.S1, self.g_b1, self.S2, self.g_head])
        self.sketches = lg.grad_norm_bind([self.S1, self.S2])
        self.norm = lg.GradNorm(E(1, t=torch.float32), E(1, t=torch.float32),
                                E(4, t=torch.float32))
        # one scratch for all calls of the step: they run one after the other
        need = [lg.linear_ws_bytes(T, a, b) for a, b in ((d, k), (k, d), (V, k))]
        need += [lg.sample_tokens_ws_bytes(T, V), lg.token_logprob_ws_bytes(T, V, 0),
                 lg.linear_backward_act_ws_bytes(T, d), lg.adapter_ws_bytes(T, k, d, r),
                 self.all.ws_bytes, 256]
        self.ws = E(max(need), t=torch.uint8)
        self.ws_s = [lg.sketch_workspace(T, d, k, r), lg.sketch_workspace(T, k, d, r)]

    def outputs(self):
        lp = self.lp
        return [self.pre, self.h, self.y0, self.y, self.z, *self.drawn, lp.logp, lp.entropy, lp.lse,
                self.dz_z, self.dz, self.dy, self.dh, self.dpre, self.dX, self.S1, self.S2,
                self.g_head, self.g_b1, *self.norm]

    def reset(self):
        for p, p0 in zip((self.b1, self.head), self.kept0):
            p.copy_(p0)
        for x in self.state:
            x.zero_()
        for x in self.outputs():
            x.fill_(-7 if x.dtype in (torch.int32, torch.int64) else float("nan"))

    def run(self, after_gradients=lambda: None):
        lg, ws = self.lg, self.ws
        lg.linear(self.X, self.W1, bias=self.b1, act="silu", pre=self.pre, out=self.h, ws=ws)
        lg.linear(self.h, self.W2, residual=self.X, out=self.y0, ws=ws)
        lg.adapter_apply(self.h, self.y0, self.policy, self.Uu, self.scale, seeds=self.keys,
                         out=self.y, ws=ws)
        lg.linear(self.y, self.head, out=self.z, ws=ws)
        lg.sample_tokens(self.z, self.u, tau=0.8, top_k=100, top_p=0.95, out=self.drawn, ws=ws)
        token = self.drawn.token
        lg.token_logprob(self.z, token, tau=0.8, out=self.lp, ws=ws)
        lg.token_logprob_backward(self.z, token, self.lp.lse, self.lp.entropy, self.adv, tau=0.8,
                                  dz=self.dz_z)
        lg.linear_backward_act(self.dz_z, dY=self.dz)
        lg.linear_backward_weight(self.dz, self.y, dW=self.g_head, ws=ws)
        lg.linear_backward_input(self.dz, self.head, out=self.dy, ws=ws)
        lg.sketch_accumulate(self.h, self.dy, self.S2, 8, ws=self.ws_s[1], overwrite=True)
        lg.linear_backward_input(self.dy, self.W2, out=self.dh, ws=ws)
        lg.linear_backward_act(self.dh, self.pre, "silu", dY=self.dpre, d_bias=self.g_b1, ws=ws)
        lg.sketch_accumulate(self.X, self.dpre, self.S1, 7, ws=self.ws_s[0], overwrite=True)
        lg.linear_backward_input(self.dpre, self.W1, residual=self.dy, out=self.dX, ws=ws)
        after_gradients()
        lg.grad_norm(self.all, max_norm=1e-2, per_tensor=True, out=self.norm, ws=ws)
        lg.adamw_step(self.adam, 1e-2, 1, grad_scale=self.norm.scale)
        lg.grad_clip(self.sketches, self.norm.scale)

    def results(self):
        return [x.clone() for x in (*self.outputs(), self.b1, self.head, *self.state)]


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def product_ok(got, want, M, K, extra=0.0):
    return np.all(np.abs(f64(got) - want) <= (K + 2) * U * M + H * np.abs(want) + extra)


@pytest.mark.parametrize("T,z_type", [(200, BF), (5, BF), (70, torch.float32)])
def test_step_matches_the_oracle(lg, T, z_type):
    say("step", T, z_type)
    s = Step(lg, T=T, z_type=z_type)
    s.reset()
    raw = {}
    s.run(lambda: raw.update(S1=s.S1.clone(), S2=s.S2.clone()))
    torch.cuda.synchronize()
    X, W1, W2, head = f64(s.X), f64(s.W1), f64(s.W2), f64(s.kept0[1])
    k, d = X.shape[1], W1.shape[0]
    # forward
    h, pre = olin.forward(X, W1, f64(s.kept0[0]), "silu")
    M = np.abs(X) @ np.abs(W1).T + np.abs(f64(s.kept0[0]))
    assert product_ok(s.pre, pre, M, k)
    assert product_ok(s.h, h, 1.13 * M, k, 2.0 ** -20 * (np.abs(pre) + 1))
    h = f64(s.h)
    y, _ = olin.forward(h, W2, residual=X)
    assert product_ok(s.y0, y, np.abs(h) @ np.abs(W2).T + np.abs(X), d)
    A = [oproj.projection(100 + i, i, 0, s.r, d) for i in range(3)]
    y, M = oadp.apply(h, f64(s.y0), s.policy.cpu().numpy(), f64(s.Uu), A, f64(s.scale))
    assert np.all(np.abs(f64(s.y) - y) <= H * np.abs(y) + 1e-4 * M)
    y = f64(s.y)
    M = np.abs(y) @ np.abs(head).T
    err = np.abs(f64(s.z) - y @ head.T)
    assert np.all(err <= (k + 2) * U * M + (H * np.abs(y @ head.T) if z_type == BF else 0))
    # the tokens and their loss
    tau = float(np.float32(0.8))
    token, logp, logq, kept = osample.rows(f64(s.z), f64(s.u), tau, 100, float(np.float32(0.95)))
    assert np.array_equal(s.drawn.token.cpu().numpy(), token)
    assert np.array_equal(s.drawn.kept.cpu().numpy(), kept)
    assert np.all(token[::17] == -1) and np.all(token[1:17] >= 0)
    assert np.all(np.abs(f64(s.drawn.logq) - logq) <= U * np.abs(logq) + 1e-7)
    assert np.all(np.abs(f64(s.drawn.logp) - logp) <= U * np.abs(logp) + 1e-7)
    live = token >= 0
    # (token_logprob's own tolerance: fp32 sums over the vocabulary)
    assert np.max(np.abs(f64(s.lp.logp) - logp)[live]) < 1e-4 and np.all(f64(s.lp.logp)[~live] == 0)
    dz = olp.gradient(f64(s.z), token, tau, f64(s.lp.lse), f64(s.lp.entropy), f64(s.adv))
    assert rel_fro(f64(s.dz_z), dz) < H and np.all(f64(s.dz)[~live] == 0)
    assert torch.equal(s.dz, s.dz_z.to(BF))
    # backward
    dz = f64(s.dz)
    assert np.all(np.abs(f64(s.g_head) - dz.T @ y) <= (T + 2) * U * (np.abs(dz).T @ np.abs(y)))
    assert product_ok(s.dy, dz @ head, np.abs(dz) @ np.abs(head), s.V)
    dy = f64(s.dy)
    assert rel_fro(f64(raw["S2"]), osketch.sketch_input_first(h, dy, oproj.projection(8, 0, 0, s.r, d))) < 2e-3
    assert product_ok(s.dh, dy @ W2, np.abs(dy) @ np.abs(W2), k)
    dpre, d_b1 = olin.backward_act(f64(s.dh), f64(s.pre), "silu")
    err = 2.0 ** -18 * np.abs(f64(s.dh))
    assert np.all(np.abs(f64(s.dpre) - dpre) <= H * np.abs(dpre) + err)
    assert np.all(np.abs(f64(s.g_b1) - d_b1) <= T * U * np.abs(dpre).sum(0) + err.sum(0))
    dpre = f64(s.dpre)
    assert rel_fro(f64(raw["S1"]), osketch.sketch_input_first(X, dpre, oproj.projection(7, 0, 0, s.r, k))) < 2e-3
    assert product_ok(s.dX, dpre @ W1 + dy, np.abs(dpre) @ np.abs(W1) + np.abs(dy), d)
    # clipping and the steps
    total, scale, each = onorm.norm([f64(raw["S1"]), f64(s.g_b1), f64(raw["S2"]), f64(s.g_head)], 1e-2)
    assert scale < 1                                     # it does clip
    assert abs(s.norm.norm.item() - total) <= 1.001 * U * total
    assert abs(s.norm.scale.item() - scale) <= 1.001 * U * scale
    assert np.all(np.abs(f64(s.norm.norms) - each) <= 1.001 * U * each)
    c = s.norm.scale
    assert torch.equal(s.S1, raw["S1"] * c) and torch.equal(s.S2, raw["S2"] * c)
    for p, p0, g, m, v, wd in ((s.b1, s.kept0[0], s.g_b1, *s.state[:2], 0.0),
                               (s.head, s.kept0[1], s.g_head, *s.state[2:], float(np.float32(0.1)))):
        zero = np.zeros(p.numel())
        w, mm, vv = oadw.step(f64(p0).ravel(), f64(g).ravel() * c.item(), zero, zero, 1e-2, 0.9,
                              0.999, 1e-8, wd, 1)
        half = H if p.dtype == BF else U
        # a first step moves an entry by lr g / (|g| + eps), of relative precision 1e-5
        assert np.all(np.abs(f64(p).ravel() - w) <= half * np.abs(w) + 1e-6)
        assert rel_fro(f64(m).ravel(), mm) < 1e-6


def test_step_graph_replays_equal_eager(lg):
    say("step graph")
    s = Step(lg, T=6, V=20011)                # (few rows: the draw's and products' split forms)
    s.reset()
    s.run()
    torch.cuda.synchronize()
    ref = s.results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    s.reset()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    torch.cuda.synchronize()
    other = Step(lg, T=6, V=20011, seed=9)
    for rep in range(4):
        s.reset()
        other.ws, other.ws_s = s.ws, s.ws_s
        other.run()                             # eager work through the same scratch
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(s.results(), ref)):
            assert same_bits(a, b), (rep, i)
    del g


def test_two_graphs_share_a_scratch(lg):
    """Two captured steps with one scratch, replayed in turn on one stream."""
    say("two step graphs")
    steps = [Step(lg, T=6, V=20011, seed=31), Step(lg, T=9, V=15000, seed=32)]
    big = max(steps, key=lambda s: s.ws.numel())
    refs, graphs = [], []
    for s in steps:
        s.ws = big.ws
        s.reset()
        s.run()
        torch.cuda.synchronize()
        refs.append(s.results())
    for s in steps:
        s.reset()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        torch.cuda.synchronize()
        graphs.append(g)
    for rep in range(3):
        for s in steps:
            s.reset()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s, ref in zip(steps, refs):
            for i, (a, b) in enumerate(zip(s.results(), ref)):
                assert same_bits(a, b), (rep, i)
    del graphs, g


def test_two_streams_at_once(lg):
    say("step, two streams")
    steps = [Step(lg, seed=21), Step(lg, T=7, k=512, d=200, V=30000, r=64, seed=22)]
    refs = []
    for s in steps:
        s.reset()
        s.run()
        torch.cuda.synchronize()
        refs.append(s.results())
    streams = [torch.cuda.Stream() for _ in steps]
    for rep in range(3):
        for s in steps:
            s.reset()
        torch.cuda.synchronize()
        for s, q in zip(steps, streams):
            with torch.cuda.stream(q):
                s.run()
        torch.cuda.synchronize()
        for s, ref in zip(steps, refs):
            for i, (a, b) in enumerate(zip(s.results(), ref)):
                assert same_bits(a, b), (rep, i)


def test_binding_refuses(lg):
    X, W = torch.zeros(64, 128, dtype=BF, device="cuda"), torch.zeros(96, 128, dtype=BF, device="cuda")
    u, f = torch.zeros(64, device="cuda"), torch.zeros(96, device="cuda")
    err = lg._lib.LograError
    for kind, call in (
            (err, lambda: lg.linear(X, W[:, :128].contiguous(), out=X[:, :96])),    # over its input
            (err, lambda: lg.linear(X[:1].expand(64, 128), W)),
            (ValueError, lambda: lg.linear(X.t(), W)),
            (ValueError, lambda: lg.linear(X, W[:, :64])),
            (ValueError, lambda: lg.linear(X, W, bias=f[:64])),
            (ValueError, lambda: lg.linear(X, W, act="tanh")),
            (ValueError, lambda: lg.linear(X, W, out_dtype=torch.float16)),
            (ValueError, lambda: lg.linear(X.float(), W)),
            (ValueError, lambda: lg.linear(X, W, residual=X)),
            (ValueError, lambda: lg.linear_backward_act(X, act="relu")),
            (ValueError, lambda: lg.linear_backward_act(X, pre=X)),
            (ValueError, lambda: lg.linear_backward_input(X, W)),
            (ValueError, lambda: lg.linear_backward_weight(X, W)),
            (ValueError, lambda: lg.linear_backward_weight(X, X, accumulate=True)),
            (ValueError, lambda: lg.linear_backward_weight(X, X, dW=torch.zeros_like(X), accumulate=True)),
            (ValueError, lambda: lg.sample_tokens(X, u[:63])),
            (ValueError, lambda: lg.sample_tokens(X.half(), u)),
            (ValueError, lambda: lg.sample_tokens(X, u, top_k=-1)),
            (ValueError, lambda: lg.sample_tokens(X, u, top_k=u)),
            (ValueError, lambda: lg.sample_tokens(X, u, tau=u[:3])),
            (err, lambda: lg.sample_tokens(X, u, tau=0)),
            (err, lambda: lg.sample_tokens(X, u, top_p=1.5)),
            (ValueError, lambda: lg.grad_norm_bind([X, X])),
            (ValueError, lambda: lg.grad_norm_bind([X.t()])),
            (ValueError, lambda: lg.grad_norm_bind([X], out=[f])),
            (ValueError, lambda: lg.grad_norm(lg.grad_norm_bind([X]), norm_type=1)),
            (ValueError, lambda: lg.grad_norm(lg.grad_norm_bind([X]), grad_scale=u)),
            (ValueError, lambda: lg.grad_clip(lg.grad_norm_bind([X]), u))):
        with pytest.raises(kind):
            call()
    assert not X.any() and not W.any()


def test_the_same_tensor_twice(lg):
    """One tensor as two inputs, and a batch without rows."""
    X = torch.randint(-2, 3, (64, 128), device="cuda").to(BF)
    W = torch.randint(-2, 3, (128, 128), device="cuda").to(BF)
    x, w = f64(X), f64(W)
    bf16 = lambda a: torch.from_numpy(a).to(BF)
    assert torch.equal(lg.linear(X, W, residual=X).cpu(), bf16(x @ w.T + x))
    assert torch.equal(lg.linear(W, W).cpu(), bf16(w @ w.T))
    assert torch.equal(lg.linear_backward_input(X, W, residual=X).cpu(), bf16(x @ w + x))
    assert np.array_equal(f64(lg.linear_backward_weight(X, X)), x.T @ x)
    none = torch.empty(0, 128, dtype=BF, device="cuda")
    assert lg.linear(none, W).shape == (0, 128) and lg.linear_backward_act(none).shape == (0, 128)
    assert lg.sample_tokens(none, torch.empty(0, device="cuda")).token.shape == (0,)
    assert not lg.linear_backward_weight(none, none).any()
