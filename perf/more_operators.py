"""Measured cases of the operators that close a policy step: drawing tokens from
logits, the layer product with its epilogue and its gradients, and the global
gradient norm with clipping.

With `own` false, run() computes each operator from elementary torch products,
sums, exponentials, comparisons and sorts (32 bits; 64 for the cumulative masses
of a draw and for the sums of a norm); with `own` true it makes the calls that a
program makes of the library.  Inputs come from the seed alone.

Definitions:
  sample     row t, a = z / tau, p = softmax(a), tokens in descending order of
             their logits (equal ones: ascending index).  Kept are the first K:
             K1 = top_k (0: all tokens above -inf), M1 their mass; Kp the fewest
             with mass >= top_p M1 (top_p = 1: no limit); Km those with p_j >=
             min_p max p; K = max(1, min(K1, Kp, Km)), M their mass.  The token
             is the first whose cumulative mass exceeds u M; logp = log p, logq =
             log (p / M).  A row with u outside [0, 1) is left out (-1, zeros);
             one with a NaN or +inf logit or none above -inf has no token (-1,
             NaN, none kept).  tau, top_p and min_p are the fp32 values.
  norm       |s| sqrt(sum over all tensors of g^2) with s = grad_scale, also per
             tensor; scale = s min(1, max_norm / norm).
  clip       out = g scale, rounded to out's type.
  linear     pre = X W^T + bias, out = act(pre) + residual.
  backward   dY = d_out act'(pre), d_bias = sum_t of the unrounded dY, dX = dY W +
             residual, dW = dY^T X, both from dY as rounded.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one step of a small rollout batch, the usual truncation for all rows
        dict(name="sample 8 x 152064, top 50, p 0.95", op="sample", n=8, V=152064, dtype="bf16",
             rows=False, tau=1.0, top_k=50, top_p=0.95, min_p=0.0, pad=0.0, mask=0.0),
        # fp32 logits of an odd vocabulary, on-policy: nothing truncated; ended
        # sequences and a masked part of the vocabulary
        dict(name="sample 65 x 32003 fp32, whole vocabulary", op="sample", n=65, V=32003,
             dtype="fp32", rows=False, tau=0.7, top_k=0, top_p=1.0, min_p=0.0, pad=0.1, mask=0.03),
        # a large rollout batch whose requests each have settings of their own
        dict(name="sample 512 x 152064, each row its own", op="sample", n=512, V=152064,
             dtype="bf16", rows=True, tau=1.0, top_k=0, top_p=1.0, min_p=0.0, pad=0.05, mask=0.0),
        # the norms and biases of 28 decoder layers (hidden 1536) with their rank-16
        # sketches: many small fp32 tensors
        dict(name="norm 168 small tensors", op="norm", shape="layers", count=28, size=1536,
             dtype="fp32", clip=False),
        # the gradient of a 152064 x 1536 token embedding
        dict(name="norm embedding bf16", op="norm", shape="one", count=1, size=152064 * 1536,
             dtype="bf16", clip=False),
        # ragged tensors of bf16 and fp32, norm and clipped copies
        dict(name="norm and clip, ragged", op="norm", shape="ragged", count=23, size=4014079,
             dtype="both", clip=True),
        # one request's next token through a layer
        dict(name="linear 1 x 4096 to 4096", op="linear", T=1, k=4096, d=4096, act="none",
             bias=True, residual=False, pre=False, out="bf16"),
        # a decoding batch up a feed-forward block
        dict(name="linear 200 x 1536 to 8960, silu", op="linear", T=200, k=1536, d=8960,
             act="silu", bias=True, residual=False, pre=False, out="bf16"),
        # the head of a decoding batch: fp32 logits
        dict(name="linear 64 x 1536 to 152064, fp32", op="linear", T=64, k=1536, d=152064,
             act="none", bias=False, residual=False, pre=False, out="fp32"),
        # a training microbatch: activation, residual, and pre kept for the backward pass
        dict(name="linear 8192 x 4096 to 4096, gelu", op="linear", T=8192, k=4096, d=4096,
             act="gelu", bias=True, residual=True, pre=True, out="bf16"),
        # a ragged microbatch of odd sizes, backward
        dict(name="backward 501 x 1543 to 1001, relu", op="backward", T=501, k=1543, d=1001,
             act="relu", residual=True, dW="fp32"),
        # the training microbatch, backward
        dict(name="backward 8192 x 4096 to 4096, silu", op="backward", T=8192, k=4096, d=4096,
             act="silu", residual=False, dW="bf16"),
    ]


ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "norm", "linear", "linear", "backward"])
    if op == "sample":
        return dict(op=op, n=_log_int(rng, 1, 512), V=_log_int(rng, 1000, 152064),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]), rows=rng.random() < 0.4,
                    tau=rng.choice([1.0, 0.7, 1.3]), top_k=rng.choice([0, 0, 1, 20, 50, 700]),
                    top_p=rng.choice([1.0, 0.95, 0.8]), min_p=rng.choice([0.0, 0.0, 0.05]),
                    pad=rng.choice([0.0, 0.1]), mask=rng.choice([0.0, 0.03]))
    if op == "norm":
        shape = rng.choice(["layers", "one", "ragged"])
        size = (_log_int(rng, 1000, 10 ** 8) if shape == "one" else
                rng.randrange(64, 4096) if shape == "layers" else _log_int(rng, 1000, 4 * 10 ** 6))
        return dict(op=op, shape=shape, count=1 if shape == "one" else rng.randrange(2, 30),
                    size=size, dtype=rng.choice(["bf16", "fp32", "both"]),
                    clip=rng.random() < 0.5)
    T, k, d = _log_int(rng, 1, 8192), _log_int(rng, 64, 8960), _log_int(rng, 64, 8960)
    while T * k * d > 8192 * 4096 * 4096:
        T = max(1, T // 2)
    c = dict(op=op, T=T, k=k, d=d, act=rng.choice(ACTS), residual=rng.random() < 0.4)
    if op == "linear":
        c.update(bias=rng.random() < 0.6, pre=rng.random() < 0.3,
                 out=rng.choice(["bf16", "bf16", "fp32"]))
    else:
        # (dY is rounded to bf16 before the products: where its formula is a smooth one,
        # two sound fp32 evaluations round one value in 10^4 apart, which 32 bits would show)
        c["dW"] = "fp32" if c["act"] in ("none", "relu") else "bf16"
    return c


def _sizes(case):
    """Numbers of entries of the case's tensors."""
    s = case["size"]
    if case["shape"] == "one":
        return [s]
    if case["shape"] == "layers":      # two norms, three biases and a sketch of a layer
        return [s, s, s, max(1, s // 6), max(1, s // 6), 16 * s] * case["count"]
    return [max(1, s // (i + 1) ** 2 + (i * 7) % 5) for i in range(case["count"])]


def _is_bf16(case, i):
    """Whether tensor i of the case is bf16: with both types, every other one."""
    return case["dtype"] == "bf16" or (case["dtype"] == "both" and i % 2 == 0)


def work(case):
    op = case["op"]
    if op == "sample":
        n, V = case["n"], case["V"]
        return dict(bytes=n * V * (2 if case["dtype"] == "bf16" else 4) + 24 * n, flops=8 * n * V)
    if op == "norm":
        b = sum(s * (2 if _is_bf16(case, i) else 4) for i, s in enumerate(_sizes(case)))
        n = sum(_sizes(case))
        # (the norm comes before the first clipped value: two reads and a write)
        return dict(bytes=3 * b if case["clip"] else b, flops=(3 if case["clip"] else 2) * n)
    T, k, d = case["T"], case["k"], case["d"]
    if op == "linear":
        b = 2 * (T * k + d * k) + T * d * (2 if case["out"] == "bf16" else 4)
        b += 2 * d * case["bias"] + 2 * T * d * (case["residual"] + case["pre"])
        return dict(bytes=b, flops=2 * T * k * d)
    b = 2 * T * d * (2 if case["act"] == "none" else 4) + 4 * d
    b += 2 * (d * k + 2 * T * k) + 2 * T * k * case["residual"]
    b += d * k * (2 if case["dW"] == "bf16" else 4)
    return dict(bytes=b, flops=4 * T * k * d)


# ------------------------------------------------------------------ the inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _rows(n, cols, dtype):
    """An n x cols tensor whose rows start on 16-byte boundaries."""
    return torch.empty(n, -(-cols // 8) * 8, dtype=dtype, device="cuda")[:, :cols]


def _normal(g, n, cols, sigma):
    x = _rows(n, cols, torch.bfloat16)
    for a in range(0, n, 16384):
        part = x[a:a + 16384]
        part.copy_(torch.randn(part.shape, device="cuda", generator=g) * sigma)
    return x


def _prepare_sample(case, seed):
    n, V = case["n"], case["V"]
    g = _gen(seed, 1)
    z = _rows(n, V, torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    for a in range(0, n, 256):
        m = min(256, n - a)
        x = torch.randn(m, V, device="cuda", generator=g) * 2.5
        # a few likely tokens stand out, as a model's do
        at = torch.randint(V, (m, 40), device="cuda", generator=g)
        lift = torch.rand(m, 40, device="cuda", generator=g) * torch.linspace(12, 2, 40,
                                                                               device="cuda")
        z[a:a + 256].copy_(x.scatter_add_(1, at, lift))
    if case["mask"]:
        z[:, torch.rand(V, device="cuda", generator=g) < case["mask"]] = -math.inf
    u = torch.rand(n, device="cuda", generator=g)
    u[torch.rand(n, device="cuda", generator=g) < case["pad"]] = -1.0
    st = dict(op="sample", z=z, u=u)
    if case["rows"]:
        pick = lambda v, t: torch.tensor(v, device="cuda", dtype=t)[
            torch.randint(len(v), (n,), device="cuda", generator=g)]
        st["tau"] = torch.rand(n, device="cuda", generator=g) * 0.7 + 0.6
        st["top_k"] = pick([0, 0, 1, 20, 50, 700], torch.int32)
        st["top_p"] = pick([1.0, 0.95, 0.9, 0.5], torch.float32)
        st["min_p"] = pick([0.0, 0.0, 0.02, 0.1], torch.float32)
    else:
        for name in ("tau", "top_p", "min_p"):
            st[name] = float(np.float32(case[name]))
        st["top_k"] = case["top_k"]
    return st


def _prepare_norm(case, seed):
    sizes = _sizes(case)
    g = _gen(seed, 2)
    st = dict(op="norm", sizes=sizes, clip=case["clip"], kinds=[], starts=[], n=len(sizes))
    total = dict(bf16=0, fp32=0)
    owner = dict(bf16=[], fp32=[])
    for i, s in enumerate(sizes):       # each tensor starts on a block of 32 entries
        kind = "bf16" if _is_bf16(case, i) else "fp32"
        st["kinds"].append(kind)
        st["starts"].append(total[kind])
        blocks = -(-s // 32)
        total[kind] += blocks * 32
        owner[kind].append((i, blocks))
    st["flat"], st["out"], st["of"] = {}, {}, {}
    for kind, n in total.items():
        if n == 0:
            continue
        dt = torch.bfloat16 if kind == "bf16" else torch.float32
        x = torch.randn(n, device="cuda", generator=g)
        live = torch.zeros(n, dtype=torch.bool, device="cuda")
        for a, s, of in zip(st["starts"], sizes, st["kinds"]):
            if of == kind:
                live[a:a + s] = True
        # gradients of different tensors differ in size
        ids = torch.cat([torch.full((b,), i, device="cuda") for i, b in owner[kind]])
        spread = torch.exp(torch.randn(len(sizes), device="cuda", generator=g))
        x = (x.view(-1, 32) * spread[ids][:, None]).view(-1) * 1e-3
        st["flat"][kind] = (x * live).to(dt)
        st["of"][kind] = (torch.tensor([i for i, _ in owner[kind]], device="cuda"),
                          torch.tensor([b for _, b in owner[kind]], device="cuda").cumsum(0) - 1)
        if case["clip"]:
            st["out"][kind] = torch.zeros(n, dtype=dt, device="cuda")
    # unscaled from a loss scale of 2^10, and clipped to about half of what it is
    st["grad_scale"] = torch.full((1,), 2.0 ** -10, device="cuda")
    st["max_norm"] = 0.5 * 2.0 ** -10 * 1e-3 * math.sqrt(sum(sizes))
    return st


def _prepare_linear(case, seed):
    T, k, d = case["T"], case["k"], case["d"]
    g = _gen(seed, 3)
    st = dict(op=case["op"], act=case["act"])
    st["X"] = _normal(g, T, k, 1.0)
    st["W"] = _normal(g, d, k, 1.0 / math.sqrt(k))
    if case["op"] == "linear":
        st["bias"] = _normal(g, 1, d, 0.5)[0] if case["bias"] else None
        st["residual"] = _normal(g, T, d, 1.0) if case["residual"] else None
        st["out"] = _rows(T, d, torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        st["pre"] = _rows(T, d, torch.bfloat16) if case["pre"] else None
        return st
    st["d_out"] = _normal(g, T, d, 1e-2)
    st["pre"] = _normal(g, T, d, 1.5)
    st["residual"] = _normal(g, T, k, 1e-2) if case["residual"] else None
    st["dY"] = _rows(T, d, torch.bfloat16)
    st["dX"] = _rows(T, k, torch.bfloat16)
    st["dW"] = _rows(d, k, torch.bfloat16 if case["dW"] == "bf16" else torch.float32)
    st["d_bias"] = torch.empty(d, device="cuda")
    return st


def prepare(case, seed):
    if case["op"] == "sample":
        return _prepare_sample(case, seed)
    if case["op"] == "norm":
        return _prepare_norm(case, seed)
    return _prepare_linear(case, seed)


# ------------------------------------------------------------------ one pass
def _plain_sample(st):
    z, u = st["z"], st["u"]
    n, V = z.shape
    f64 = lambda x: (x if isinstance(x, torch.Tensor) else torch.tensor([x], device="cuda",
                     dtype=torch.float64)).double()[:, None]
    tau, top_p, min_p, top_k = f64(st["tau"]), f64(st["top_p"]), f64(st["min_p"]), st["top_k"]
    # the order of the values, then of the indices: one whole number for both
    b = (z.float() + 0.0).view(torch.int32)
    key = (b ^ ((b >> 31) & 0x7FFFFFFF)).long() * (1 << 32)
    key += (1 << 32) - 1 - torch.arange(V, device=z.device)
    idx = (1 << 32) - 1 - (key.sort(dim=1, descending=True).values & 0xFFFFFFFF)
    a = z.double().gather(1, idx)
    x = (a - a[:, :1]) / tau
    mass = x.exp().cumsum(1)
    alive = (a > -math.inf).sum(1)
    k1 = top_k.long() if isinstance(top_k, torch.Tensor) else torch.full_like(alive, top_k)
    k1 = torch.minimum(torch.where(k1 > 0, k1, V), alive)
    at = lambda k: mass.gather(1, (k - 1).clamp(0, V - 1)[:, None])
    kp = (mass < top_p * at(k1)).sum(1) + 1
    kp = torch.where((top_p >= 1).expand(n, 1)[:, 0], V, kp)
    log_p = min_p.log()
    km = ((x >= log_p) & (a > -math.inf)).sum(1)
    kept = torch.minimum(torch.minimum(k1, kp), km).clamp(min=1)
    m = at(kept)
    j = (mass <= u.double()[:, None] * m).sum(1).minimum(kept - 1)
    pick = lambda t: t.gather(1, j[:, None])[:, 0]
    xj = pick(x)
    logp, logq = xj - mass[:, -1].log(), xj - m[:, 0].log()
    dead = (alive == 0) | (z == math.inf).any(1) | z.isnan().any(1)
    out = ~((u >= 0) & (u < 1))
    token = torch.where(dead | out, -1, pick(idx))
    logp, logq = (torch.where(out, 0.0, torch.where(dead, math.nan, x)) for x in (logp, logq))
    kept = torch.where(dead | out, 0, kept)
    return [token, logp.float(), logq.float(), kept.int()]


def _plain_norm(st):
    total = torch.zeros(st["n"], dtype=torch.float64, device="cuda")
    for kind, x in st["flat"].items():
        # (a tensor's sum is the difference of two running sums)
        ids, ends = st["of"][kind]
        run = x.view(-1, 32).double().square().sum(1).cumsum(0)[ends]
        total[ids] = run.diff(prepend=run.new_zeros(1))
    s = st["grad_scale"].double()
    norm = s.abs() * total.sum().sqrt()
    scale = (s * (st["max_norm"] / norm).clamp(max=1.0)).float()
    res = [norm.float(), scale, (s.abs() * total.sqrt()).float()]
    if st["clip"]:
        for kind, x in st["flat"].items():
            st["out"][kind].copy_(x.float() * scale)
        res += [st["out"][kind] for kind in st["flat"]]
    return res


SQRT_2PI = math.sqrt(2 / math.pi)


def _act(x, act):
    if act == "relu":
        return x.clamp(min=0)
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return x * 0.5 * torch.erfc(x * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return x * torch.sigmoid(2 * SQRT_2PI * (x + 0.044715 * x ** 3))
    return x


def _act_slope(x, act):
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "silu":
        s = torch.sigmoid(x)
        return s * (1 + x * torch.sigmoid(-x))
    if act == "gelu":
        return (0.5 * torch.erfc(x * -math.sqrt(0.5))
                + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi))
    s = torch.sigmoid(2 * SQRT_2PI * (x + 0.044715 * x ** 3))
    return s + x * s * (1 - s) * 2 * SQRT_2PI * (1 + 3 * 0.044715 * x * x)


def _plain_linear(st):
    pre = st["X"].float() @ st["W"].float().t()
    if st["bias"] is not None:
        pre = pre + st["bias"].float()
    y = _act(pre, st["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    out = [y.to(st["out"].dtype)]
    return out + ([pre.to(torch.bfloat16)] if st["pre"] is not None else [])


def _plain_backward(st):
    d = st["d_out"].float()
    if st["act"] != "none":
        d = d * _act_slope(st["pre"].float(), st["act"])
    dY = d.to(torch.bfloat16)
    r = dY.float()
    dX = r @ st["W"].float()
    if st["residual"] is not None:
        dX = dX + st["residual"].float()
    return [dY, d.sum(0), dX.to(torch.bfloat16), (r.t() @ st["X"].float()).to(st["dW"].dtype)]


def _own(st):
    import rank_gradient_sketching_amd as lg
    if st["op"] == "sample":
        return list(lg.sample_tokens(st["z"], st["u"], tau=st["tau"], top_k=st["top_k"],
                                     top_p=st["top_p"], min_p=st["min_p"]))
    if st["op"] == "norm":
        if "bound" not in st:           # the handle a program keeps for its tensors
            cut = lambda flat: [flat[kind][a:a + s] for kind, a, s in
                                zip(st["kinds"], st["starts"], st["sizes"])]
            st["bound"] = lg.grad_norm_bind(cut(st["flat"]),
                                            out=cut(st["out"]) if st["clip"] else None)
        res = lg.grad_norm(st["bound"], max_norm=st["max_norm"], grad_scale=st["grad_scale"],
                           per_tensor=True)
        if st["clip"]:
            lg.grad_clip(st["bound"], res.scale)
            return [res.norm, res.scale, res.norms] + [st["out"][kind] for kind in st["flat"]]
        return [res.norm, res.scale, res.norms]
    act = None if st["act"] == "none" else st["act"]
    if st["op"] == "linear":
        lg.linear(st["X"], st["W"], bias=st["bias"], act=act, residual=st["residual"],
                  out=st["out"], pre=st["pre"])
        return [st["out"]] + ([st["pre"]] if st["pre"] is not None else [])
    dY = st["d_out"]
    if act is None:
        lg.linear_backward_act(dY, d_bias=st["d_bias"])
    else:
        dY = lg.linear_backward_act(dY, st["pre"], act, dY=st["dY"], d_bias=st["d_bias"])
    lg.linear_backward_input(dY, st["W"], residual=st["residual"], out=st["dX"])
    lg.linear_backward_weight(dY, st["X"], dW=st["dW"])
    return [dY, st["d_bias"], st["dX"], st["dW"]]


def run(state):
    if own:
        return _own(state)
    return {"sample": _plain_sample, "norm": _plain_norm, "linear": _plain_linear,
            "backward": _plain_backward}[state["op"]](state)


# ------------------------------------------------------------------ in 64 bits
def _exact_sample_row(z, u, tau, top_k, top_p, min_p):
    """One row by its definition: (token, logp, logq, kept)."""
    if not 0 <= u < 1:
        return -1, 0.0, 0.0, 0
    live = int(torch.count_nonzero(z != -math.inf))
    if live == 0 or not bool((z < math.inf).all()):
        return -1, math.nan, math.nan, 0
    logits, order = torch.sort(z, descending=True, stable=True)
    p = torch.softmax(logits.double() / tau, 0)
    C = torch.cumsum(p, 0)
    K1 = live if top_k <= 0 else min(top_k, live)
    M1 = float(C[K1 - 1])
    K = K1
    if top_p < 1:
        K = min(K, int(torch.searchsorted(C, top_p * M1)) + 1)
    if min_p > 0:
        gap = (logits.double() - float(logits[0])) / tau
        K = min(K, int(torch.count_nonzero(gap >= math.log(min_p))))
    K = max(K, 1)
    M = float(C[K - 1])
    j = min(int(torch.searchsorted(C, u * M, right=True)), K - 1)
    log_all = float(torch.logsumexp(logits.double() / tau, 0))
    logp = float(logits[j]) / tau - log_all
    return int(order[j]), logp, logp - math.log(M), K


def _exact_sample(st):
    n = st["z"].shape[0]
    each = lambda x: x.tolist() if isinstance(x, torch.Tensor) else [x] * n
    rows = [_exact_sample_row(st["z"][t], *x) for t, x in enumerate(
        zip(each(st["u"]), each(st["tau"]), each(st["top_k"]), each(st["top_p"]),
            each(st["min_p"])))]
    token, logp, logq, kept = zip(*rows)
    return [torch.tensor(token), torch.tensor(logp, dtype=torch.float64),
            torch.tensor(logq, dtype=torch.float64), torch.tensor(kept, dtype=torch.int32)]


def _exact_norm(st):
    parts = [torch.linalg.vector_norm(st["flat"][k][a:a + s], dtype=torch.float64)
             for k, a, s in zip(st["kinds"], st["starts"], st["sizes"])]
    norms = torch.stack(parts) * abs(float(st["grad_scale"]))
    norm = torch.linalg.vector_norm(norms)
    scale = float(st["grad_scale"]) * min(1.0, st["max_norm"] / float(norm))
    out = [norm, torch.tensor([scale], dtype=torch.float64), norms]
    if st["clip"]:
        out += [x.double() * scale for x in st["flat"].values()]
    return out


def _exact_act(x, act):
    """(value, slope) in 64 bits, by the functions' textbook forms."""
    if act == "none":
        return x, torch.ones_like(x)
    if act == "relu":
        return torch.where(x > 0, x, 0.0), (x > 0).double()
    if act == "silu":
        s = 1 / (1 + torch.exp(-x))
        return x * s, s + x * s * (1 - s)
    if act == "gelu":
        c = (1 + torch.special.erf(x / math.sqrt(2))) / 2
        return x * c, c + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    t = torch.tanh(SQRT_2PI * (x + 0.044715 * x * x * x))
    slope = (1 + t) / 2 + x / 2 * (1 - t * t) * SQRT_2PI * (1 + 3 * 0.044715 * x * x)
    return x * (1 + t) / 2, slope


def _exact_linear(st):
    pre = torch.mm(st["X"].double(), st["W"].double().t())
    if st["bias"] is not None:
        pre += st["bias"].double()
    y, _ = _exact_act(pre, st["act"])
    if st["residual"] is not None:
        y = y + st["residual"].double()
    return [y] + ([pre] if st["pre"] is not None else [])


def _exact_backward(st):
    d = st["d_out"].double()
    if st["act"] != "none":
        d = d * _exact_act(st["pre"].double(), st["act"])[1]
    # (from dY as the library's type holds it; a formula in 64 bits rounds it elsewhere
    # now and then, so what follows from it is compared to the rounding of dY only)
    r = d.to(torch.bfloat16).double()
    dX = torch.mm(r, st["W"].double())
    if st["residual"] is not None:
        dX += st["residual"].double()
    return [d, d.sum(0), dX, torch.mm(r.t().contiguous(), st["X"].double())]


def exact(case, seed):
    st = prepare(case, seed)
    return {"sample": _exact_sample, "norm": _exact_norm, "linear": _exact_linear,
            "backward": _exact_backward}[case["op"]](st)
