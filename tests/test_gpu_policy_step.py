"""The policy-step operators as they are used together with the sketch: a
batch of several policies through a shared layer (adapter_apply), its logits'
log probabilities and entropy (token_logprob), the loss gradient
(token_logprob_backward) into the head's sketch (sketch_accumulate), AdamW on
what is not sketched (adamw_step), and a proposal's predicted KL from logits
formed with the weights left alone.  Each stage is held to the oracle on the
GPU's own input of that stage.  Then the same step captured in a HIP graph and
replayed, and calls on two streams at once.
"""
import numpy as np
import pytest
import torch

from oracle import adamw as oadw
from oracle import adapter as oadp
from oracle import kl as okl
from oracle import logprob as olp
from oracle import projection as oproj
from oracle import sketch as osketch

pytestmark = pytest.mark.gpu


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


def rel_fro(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


class Step:
    """Buffers of one step: T tokens, k -> d hidden layer, vocabulary V."""

    def __init__(self, lg, T=200, k=256, d=384, V=1000, r=32, n=3, seed=5):
        self.lg, self.r, self.seed = lg, r, seed
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        N = lambda *s, sig=1.0: torch.randn(*s, device="cuda", generator=g) * sig
        bf = torch.bfloat16
        self.X, self.Y = N(T, k).to(bf), N(T, d).to(bf)
        self.head = N(V, d, sig=0.05).to(bf)
        self.adapter = torch.randint(-1, n, (T,), device="cuda", generator=g, dtype=torch.int32)
        self.U, self.scale = N(n, d, r, sig=15), -2e-4 * (1 + torch.rand(n, device="cuda", generator=g))
        self.keys = torch.tensor([[100 + i, i] for i in range(n)], device="cuda")
        self.target = torch.randint(0, V, (T,), device="cuda", generator=g)
        self.target[::17] = -100
        self.adv = N(T) / T
        self.bonus = torch.full((T,), -1e-2 / T, device="cuda")
        self.h = torch.empty(T, d, dtype=bf, device="cuda")
        self.z = torch.empty(T, V, dtype=bf, device="cuda")
        self.dz = torch.empty(T, V, dtype=bf, device="cuda")
        self.lp = lg.TokenLogprob(*(torch.empty(T, device="cuda") for _ in range(3)),
                                  torch.empty(T, 4, dtype=torch.int32, device="cuda"),
                                  torch.empty(T, 4, device="cuda"))
        self.S = torch.empty(V, r, device="cuda")
        self.ws_a = torch.empty(lg.adapter_ws_bytes(T, d, k, r), dtype=torch.uint8, device="cuda")
        self.ws_l = torch.empty(max(256, lg.token_logprob_ws_bytes(T, V, 4)), dtype=torch.uint8,
                                device="cuda")
        self.ws_s = lg.sketch_workspace(T, V, d, r)
        z8 = lambda c: torch.zeros(c, dtype=torch.uint8, device="cuda")
        self.norm, self.bias = N(d, sig=0.1) + 1, N(V, sig=0.1).to(bf)
        self.norm0, self.bias0 = self.norm.clone(), self.bias.clone()
        self.gn, self.gb = N(d, sig=1e-2), N(V, sig=1e-2).to(bf)
        self.state = [torch.zeros(d, device="cuda"), torch.zeros(d, device="cuda"), z8(V), z8(V),
                      z8(-(-V // 32)), z8(-(-V // 32))]
        m32, v32, m8, v8, em, ev = self.state
        self.bound = lg.adamw_bind([self.norm, self.bias], [self.gn, self.gb], [m32, m8],
                                   [v32, v8], m_exp=[None, em], v_exp=[None, ev],
                                   weight_decay=[0.0, 0.1])

    def reset(self):
        self.norm.copy_(self.norm0)
        self.bias.copy_(self.bias0)
        for x in self.state:
            x.zero_()
        for x in (self.h, self.z, self.dz, self.S, *self.lp[:3], self.lp.top_logp):
            x.fill_(float("nan"))
        self.lp.top_idx.fill_(-7)

    def run(self):
        lg = self.lg
        lg.adapter_apply(self.X, self.Y, self.adapter, self.U, self.scale, seeds=self.keys,
                         out=self.h, ws=self.ws_a)
        torch.matmul(self.h, self.head.t(), out=self.z)
        lg.token_logprob(self.z, self.target, n_top=4, out=self.lp, ws=self.ws_l)
        lg.token_logprob_backward(self.z, self.target, self.lp.lse, self.lp.entropy, self.adv,
                                  self.bonus, dz=self.dz)
        lg.sketch_accumulate(self.h, self.dz, self.S, 7, ws=self.ws_s, overwrite=True)
        lg.adamw_step(self.bound, 1e-2, 1)

    def results(self):
        return [x.clone() for x in (self.h, self.z, self.dz, self.S, *self.lp, self.norm, self.bias,
                                    *self.state)]


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def test_step_matches_the_oracle(lg):
    say("policy step")
    s = Step(lg)
    s.reset()
    s.run()
    torch.cuda.synchronize()
    A = [oproj.projection(100 + i, i, 0, s.r, s.X.shape[1]) for i in range(3)]
    ref, M = oadp.apply(f64(s.X), f64(s.Y), s.adapter.cpu().numpy(), f64(s.U), A, f64(s.scale))
    assert np.all(np.abs(f64(s.h) - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-4 * M)
    t = s.target.cpu().numpy()
    ref = olp.rows(f64(s.z), t, 1.0, 4)
    for got, want in ((s.lp.logp, ref["logp"]), (s.lp.entropy, ref["entropy"]), (s.lp.lse, ref["lse"])):
        assert np.max(np.abs(f64(got) - want)) < 1e-4       # (164 u (2 + 2 (ln V + 1)), u = 2^-24)
    assert np.array_equal(s.lp.top_idx.cpu().numpy(), ref["top_idx"])
    dz = olp.gradient(f64(s.z), t, 1.0, f64(s.lp.lse), f64(s.lp.entropy), f64(s.adv), f64(s.bonus))
    assert rel_fro(f64(s.dz), dz) < 2.0 ** -8
    S = osketch.sketch_input_first(f64(s.h), f64(s.dz), oproj.projection(7, 0, 0, s.r, s.h.shape[1]))
    assert rel_fro(f64(s.S), S) < 2e-3
    # the head's gradient sketch equals the sketch of the formula's dz, to dz's rounding
    S = osketch.sketch_input_first(f64(s.h), dz, oproj.projection(7, 0, 0, s.r, s.h.shape[1]))
    assert rel_fro(f64(s.S), S) < 1e-2
    zero = np.zeros(s.norm.numel())
    w, m, v = oadw.step(f64(s.norm0), f64(s.gn), zero, zero, 1e-2, 0.9, 0.999, 1e-8, 0.0, 1)
    assert np.max(np.abs(f64(s.norm) - w)) < 1e-6 and rel_fro(f64(s.state[0]), m) < 1e-6
    zero = np.zeros(s.bias.numel())
    w, m, v = oadw.step(f64(s.bias0), f64(s.gb), zero, zero, 1e-2, 0.9, 0.999, 1e-8,
                        float(np.float32(0.1)), 1)
    assert np.all(np.abs(f64(s.bias) - w) <= 2.0 ** -8 * np.abs(w) + 1e-6)
    got = f64(lg.adamw_state_values(s.state[2], s.state[4], "m"))
    assert np.all(np.abs(got - m) <= 2.0 ** -3 * np.abs(m) + 2.0 ** -15 * np.abs(m).max())


def test_proposal_logits_without_merging(lg):
    """The predicted KL of an update from logits formed by adapter_apply equals
    that of the oracle on the same logits, and is near the merged weights' one
    (whose bf16 rounding of W moves the logits by up to 2^-8 of them)."""
    say("proposal logits")
    T, d, V, r, seed, eta = 64, 256, 1500, 16, 31, 4e-4
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    N = lambda *s: torch.randn(*s, device="cuda", generator=g)
    X, W, S = N(T, d).to(torch.bfloat16), (N(V, d) * 0.1).to(torch.bfloat16), N(V, r) * 8
    z = torch.empty(T, 1504, dtype=torch.bfloat16, device="cuda")[:, :V]
    z.copy_((X.float() @ W.float().t()).to(torch.bfloat16))
    zp = torch.empty(T, 1504, dtype=torch.bfloat16, device="cuda")[:, :V]
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    lg.adapter_apply(X, z, ids, S[None], torch.tensor([-eta], device="cuda"),
                     seeds=torch.tensor([[seed, 0]], device="cuda"), out=zp)
    q = lg.predicted_kl(z, zp, 1.0, 2e-4, 4.0)[0].item()
    assert abs(q / okl.predicted_kl(f64(z), f64(zp), 1.0) - 1) < 1e-3
    W2 = W.clone()
    lg.merge(W2, S, seed, 0, 0, 1.0, eta)
    merged = okl.predicted_kl(f64(X) @ f64(W).T, f64(X) @ f64(W2).T, 1.0)
    assert 0.5 < q / merged < 2


def test_step_graph_replays_equal_eager(lg):
    say("policy step graph")
    s = Step(lg)
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
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    torch.cuda.synchronize()
    other = Step(lg, seed=9)
    for rep in range(4):
        s.reset()
        other.ws_a, other.ws_l, other.ws_s = s.ws_a, s.ws_l, s.ws_s
        other.run()                             # eager work through the same scratch
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(s.results(), ref)):
            assert same_bits(a, b), (rep, i)
    del g


def test_two_streams_at_once(lg):
    say("policy step, two streams")
    steps = [Step(lg, seed=21), Step(lg, T=333, k=512, d=200, V=5000, r=64, seed=22)]
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
