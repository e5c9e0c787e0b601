"""Measured cases of the policy-step operators: token log probabilities with
their gradient, AdamW over many tensors, and unmerged low-rank updates beside a
shared projection.

With `own` false, run() computes each operator from elementary torch products,
sums, exponentials and comparisons in fp32; with `own` true it makes the calls
that a program makes of the library.  Inputs come from the seed alone.

Definitions (row t, vocabulary V, a = z / tau, p = softmax(a)):
  logprob    lse = log sum_j e^a_j, logp = a[target] - lse, H = -sum p log p,
             the n_top most probable tokens (ties to the lowest index) with
             their log probabilities.  A target outside [0, V) marks a row that
             is left out (zeros; index -1 and -inf among the alternatives).
  gradient   dz_j = (d_logp ([j = target] - p_j) - d_H p_j (log p_j + H)) / tau.
  adamw      m <- b1 m + (1 - b1) g, v <- b2 v + (1 - b2) g^2,
             w <- w - lr ((m / bc1) / (sqrt(v / bc2) + eps) + wd w).
  8-bit      blocks of 32 entries share an exponent byte E; m is a sign and
             seven bits (3 of mantissa), sqrt(v) eight bits (4 of mantissa):
             value = float bits ((E - 15) << 23) + (code << (23 - mantissa)),
             code 0 is zero.  Rounding adds a counter-based dither to the bits
             that are dropped.
  adapter    Y[t] + scale[a] (X[t] A_a^T) U_a^T with a = adapter[t]; rows with
             an index outside [0, n) keep Y[t].  A_a: +-1/sqrt(r) signs drawn
             from (seed, stream), or given.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one sampling step of a small rollout batch: log probability of the
        # sampled token, entropy and the eight best alternatives
        dict(name="logprob decode 8 x 152064, top 8", op="logprob", n=8, V=152064, dtype="bf16",
             tau=1.0, n_top=8, pad=0.0, mask=0.0),
        # fp32 logits of an odd vocabulary at a sampling temperature, with
        # padded positions and a masked part of the vocabulary
        dict(name="logprob 501 x 32003 fp32, top 5", op="logprob", n=501, V=32003, dtype="fp32",
             tau=0.7, n_top=5, pad=0.1, mask=0.03),
        # scoring four responses of 1024 tokens for the policy ratio
        dict(name="logprob 4096 x 152064", op="logprob", n=4096, V=152064, dtype="bf16", tau=1.0,
             n_top=0, pad=0.02, mask=0.0),
        # the policy loss and entropy bonus down to the logits, ragged batch
        dict(name="logprob grad 501 x 32003 fp32", op="logprob_grad", n=501, V=32003,
             dtype="fp32", tau=0.7, pad=0.1, mask=0.03),
        # the same over four responses of 1024 tokens
        dict(name="logprob grad 4096 x 152064", op="logprob_grad", n=4096, V=152064,
             dtype="bf16", tau=1.0, pad=0.02, mask=0.0),
        # norms and biases of 28 decoder layers (hidden 1536, kv 256): many small
        # tensors, kept in fp32
        dict(name="adamw 140 small tensors fp32", op="adamw", bits=32, param="fp32", grad="fp32",
             master=False, shape="layers", count=28, size=1536),
        # a 152064 x 1536 token embedding: bf16 weights with fp32 masters
        dict(name="adamw embedding, 32-bit states", op="adamw", bits=32, param="bf16",
             grad="bf16", master=True, shape="one", count=1, size=152064 * 1536),
        # ragged tensors of one unsketched layer in bf16, 8-bit states
        dict(name="adamw ragged layer, 8-bit states", op="adamw", bits=8, param="bf16",
             grad="bf16", master=False, shape="ragged", count=23, size=401407),
        # the embedding again with 8-bit states
        dict(name="adamw embedding, 8-bit states", op="adamw", bits=8, param="bf16", grad="bf16",
             master=True, shape="one", count=1, size=152064 * 1536),
        # one request's next token under its own policy version
        dict(name="adapter 1 token, 4096 x 4096 r 64", op="adapter", T=1, k=4096, d=4096, r=64,
             n=4, A="signs", U="fp32", rows="mixed"),
        # a decoding batch of 200 requests over 16 policies, given bases
        dict(name="adapter 200 tokens, 1536 to 8960 r 16", op="adapter", T=200, k=1536, d=8960,
             r=16, n=16, A="given", U="bf16", rows="mixed"),
        # prompts of eight policies, packed
        dict(name="adapter 8192 tokens, 4096 x 4096 r 64", op="adapter", T=8192, k=4096, d=4096,
             r=64, n=8, A="signs", U="fp32", rows="runs"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprob", "logprob_grad", "adamw", "adamw", "adapter", "adapter"])
    if op in ("logprob", "logprob_grad"):
        V = _log_int(rng, 1000, 160000)
        n = min(_log_int(rng, 1, 4096), 4096 * 152064 // V)
        dtype = rng.choice(["bf16", "fp32"])
        c = dict(op=op, n=max(1, n // 2 if dtype == "fp32" else n), V=V, dtype=dtype,
                 tau=rng.choice([1.0, 0.7, 1.3]), pad=rng.choice([0.0, 0.05, 0.2]),
                 mask=rng.choice([0.0, 0.02]))
        if op == "logprob":
            c["n_top"] = rng.choice([0, 1, 5, 8, 20]) if n <= 1024 else 0
        return c
    if op == "adamw":
        bits = rng.choice([32, 8])
        param = rng.choice(["bf16", "fp32"])
        shape = rng.choice(["layers", "one", "ragged"])
        size = (_log_int(rng, 1000, 10 ** 8) if shape == "one" else
                rng.randrange(64, 4096) if shape == "layers" else _log_int(rng, 1000, 10 ** 6))
        return dict(op=op, bits=bits, param=param, grad=rng.choice(["bf16", param]),
                    master=param == "bf16" and rng.random() < 0.5, shape=shape,
                    count=1 if shape == "one" else rng.randrange(2, 40), size=size)
    T, k, d = _log_int(rng, 1, 8192), _log_int(rng, 64, 8960), _log_int(rng, 64, 8960)
    r, n = rng.choice([1, 4, 8, 16, 24, 32, 64, 100, 128, 256]), rng.choice([1, 2, 5, 8, 16, 33])
    while T * n * r * (k + d) > 8192 * 512 * 8192:
        T = max(1, T // 2)
    return dict(op="adapter", T=T, k=k, d=d, r=r, n=n, A=rng.choice(["signs", "given"]),
                U=rng.choice(["fp32", "bf16"]), rows=rng.choice(["mixed", "runs"]))


def _sizes(case):
    """Numbers of entries of the case's tensors."""
    if case["shape"] == "one":
        return [case["size"]]
    if case["shape"] == "layers":      # two norms and the q/k/v biases of a layer
        s = case["size"]
        return [s, s, s, max(1, s // 6), max(1, s // 6)] * case["count"]
    s = case["size"]                   # ragged: from the size down to single entries
    return [max(1, s // (i + 1) ** 2 + (i * 7) % 5) for i in range(case["count"])]


def work(case):
    op = case["op"]
    if op in ("logprob", "logprob_grad"):
        e = 2 if case["dtype"] == "bf16" else 4
        nv = case["n"] * case["V"]
        if op == "logprob":
            return dict(bytes=nv * e + case["n"] * (20 + 12 * case["n_top"]), flops=6 * nv)
        return dict(bytes=2 * nv * e + case["n"] * 24, flops=8 * nv)
    if op == "adamw":
        n = sum(_sizes(case))
        p, g = (2 if case[x] == "bf16" else 4 for x in ("param", "grad"))
        state = 16 if case["bits"] == 32 else 4 + 4 / 32 + 4   # both ways; 8 bits: and as values
        weights = 8 + p if case["master"] else 2 * p           # read and written
        return dict(bytes=n * (weights + g + state), flops=20 * n)
    T, k, d, r, n = (case[x] for x in ("T", "k", "d", "r", "n"))
    used = min(n, T)
    b = T * (2 * k + 4 * d + 4) + used * (d * r * (4 if case["U"] == "fp32" else 2) + 4)
    b += used * (r * k * 2 if case["A"] == "given" else 16)
    return dict(bytes=b, flops=2 * T * r * (k + d))


# ------------------------------------------------------------------ the inputs
BETA1, BETA2, EPS, LR, STEP = 0.9, 0.999, 1e-8, 1e-3, 17


def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + salt)
    return g


def _rows(n, cols, dtype, mult=8):
    """An n x cols tensor whose rows start on 16-byte boundaries."""
    return torch.empty(n, -(-cols // mult) * mult, dtype=dtype, device="cuda")[:, :cols]


def _logits(case, seed):
    n, V = case["n"], case["V"]
    g = _gen(seed, 1)
    z = _rows(n, V, torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    for a in range(0, n, 512):
        z[a:a + 512].copy_(torch.randn(min(512, n - a), V, device="cuda", generator=g) * 3)
    # sampled tokens are likely ones: a raised logit at the target
    target = torch.randint(V, (n,), device="cuda", generator=g)
    lift = torch.rand(n, device="cuda", generator=g) * 12
    at = torch.arange(n, device="cuda")
    z[at, target] = (z[at, target].float() + lift).to(z.dtype)
    if case["mask"]:
        z[:, torch.rand(V, device="cuda", generator=g) < case["mask"]] = -math.inf
        z[at, target] = lift.to(z.dtype)          # the given token is never masked
    target[torch.rand(n, device="cuda", generator=g) < case["pad"]] = -100
    return z, target


def _encode(x, dither, keep):
    """(codes, block exponents) of the 8-bit form of x, blocks of 32 entries."""
    t = x.abs().contiguous().view(torch.int32)
    drop = 23 - keep
    t = t + dither
    E = (t >> 23).view(-1, 32).amax(1).clamp(16, 254)
    c = (t >> drop).view(-1, 32) - ((E - 15) << keep).unsqueeze(1)
    return c.clamp(min=0).reshape(-1), E


def _decode(c, E, keep):
    """Values of magnitudes c with block exponents E."""
    b = ((E.to(torch.int32) - 15) << 23).unsqueeze(1) + (c.view(-1, 32) << (23 - keep))
    x = b.view(torch.float32).reshape(-1)
    return torch.where(c > 0, x, torch.zeros_like(x))


def _dither(n, step, half, keep):
    """The counter-based dither of n entries: multiples of two odd constants near
    2^32 times irrationals, modulo 2^32; the top 23 - keep bits are used."""
    i = torch.arange(n, device="cuda")
    h = (i * 0x6A09E667 + step * 0x9E3779B9 + half) & 0xFFFFFFFF
    return (h >> (9 + keep)).to(torch.int32)


def _pack_m(m, step):
    c, E = _encode(m, _dither(m.numel(), step, 0, 3), 3)
    return (c + torch.where(m < 0, 128, 0)).to(torch.uint8), E.to(torch.uint8)


def _pack_v(v, step):
    root = v.sqrt()
    c, E = _encode(root, _dither(v.numel(), step, 0x80000000, 4), 4)
    return torch.where((root > 0) & (c < 1), 1, c).to(torch.uint8), E.to(torch.uint8)


def _prepare_adamw(case, seed):
    sizes = _sizes(case)
    starts, total = [], 0
    for s in sizes:                     # each tensor starts on a block of 32 entries
        starts.append(total)
        total += -(-s // 32) * 32
    g = _gen(seed, 2)
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    for a, s in zip(starts, sizes):
        live[a:a + s] = True

    def normal():
        return torch.randn(total, device="cuda", generator=g).mul_(live)

    scale = 1e-3 * torch.exp(normal().view(-1, 32)[:, :1]).expand(-1, 32).reshape(-1)
    pd, gd = (torch.bfloat16 if case[x] == "bf16" else torch.float32 for x in ("param", "grad"))
    w = normal() * 0.02
    st = dict(op="adamw", sizes=sizes, starts=starts, bits=case["bits"])
    st["p"] = w.to(pd)
    st["master"] = w if case["master"] else None
    st["g"] = (normal() * scale).to(gd)
    m, v = normal() * scale * 0.3, (normal() * 0.1 + 1).square() * scale.square() * live
    if case["bits"] == 8:
        st["m"], st["m_exp"] = _pack_m(m, STEP - 1)
        st["v"], st["v_exp"] = _pack_v(v, STEP - 1)
    else:
        st["m"], st["v"] = m, v
    # tensors of one axis (norms, biases) take no weight decay
    st["wd"] = [0.1 if s > 100000 else 0.0 for s in sizes]
    st["wd_of"] = torch.tensor(st["wd"], device="cuda")
    st["block_ends"] = torch.tensor([-(-s // 32) for s in sizes], device="cuda").cumsum(0)
    return st


def _signs(r, k, seed, stream):
    """The r x k sign basis of (seed, stream): row i, column j takes bit j & 63 of
    word (j >> 6) & 3 of the Philox4x64-10 block with counter (j >> 8, i, 0, 0)."""
    blocks = -(-k // 256)
    rows = np.empty((r, blocks * 4), np.uint64)
    for i in range(r):
        # (the generator steps its counter before each block)
        at = ((i << 64) - 1) % (1 << 256)
        gen = np.random.Philox(counter=at, key=seed + (stream << 64))
        rows[i] = gen.random_raw(blocks * 4)
    bits = np.unpackbits(rows.view(np.uint8), axis=1, bitorder="little")[:, :k]
    return 1.0 - 2.0 * bits.astype(np.float32)


def _prepare_adapter(case, seed):
    T, k, d, r, n = (case[x] for x in ("T", "k", "d", "r", "n"))
    g = _gen(seed, 3)
    rs = np.random.default_rng([seed, 4])
    st = dict(op="adapter")
    st["X"] = _rows(T, k, torch.bfloat16)
    st["X"].copy_(torch.randn(T, k, device="cuda", generator=g))
    st["Y"] = _rows(T, d, torch.bfloat16)
    st["Y"].copy_(torch.randn(T, d, device="cuda", generator=g))
    st["out"] = _rows(T, d, torch.bfloat16)
    st["U"] = (torch.randn(n, d, r, device="cuda", generator=g) * 15).to(
        torch.float32 if case["U"] == "fp32" else torch.bfloat16)
    # minus the step: -alpha eta
    st["scale"] = -(torch.rand(n, device="cuda", generator=g) + 0.5) * 2e-4
    if case["rows"] == "mixed":         # any order, the base policy (-1) among them
        ids = rs.integers(-1 if T > 1 else 0, n, T)
    else:                               # prompts of different lengths, packed
        cuts = np.sort(rs.integers(0, T + 1, 4 * n - 1))
        ids = np.repeat(rs.integers(0, n, 4 * n), np.diff(np.concatenate([[0], cuts, [T]])))
    st["adapter"] = torch.from_numpy(ids.astype(np.int32)).cuda()
    if case["A"] == "signs":
        keys = rs.integers(0, 1 << 62, (n, 2))
        keys[:, 1] = 0
        st["seeds"] = torch.from_numpy(keys).cuda()
        # the plain form has no generator: it gets the same signs spelled out
        A = np.stack([_signs(r, k, int(s), int(t)) for s, t in keys])
        st["A"] = torch.from_numpy(A).cuda().to(torch.bfloat16)
        st["unit"] = 1.0 / math.sqrt(r)
    else:
        st["A"] = (torch.randn(n, r, k, device="cuda", generator=g) / math.sqrt(r)).to(
            torch.bfloat16)
        st["seeds"], st["unit"] = None, 1.0
    return st


def prepare(case, seed):
    op = case["op"]
    if op == "adamw":
        return _prepare_adamw(case, seed)
    if op == "adapter":
        return _prepare_adapter(case, seed)
    z, target = _logits(case, seed)
    st = dict(op=op, z=z, target=target, tau=case["tau"], n_top=case.get("n_top", 0))
    if op == "logprob_grad":
        # what the forward pass left, and the loss's gradients (a policy ratio's
        # advantage and an entropy bonus, both over the mean of the batch)
        n = case["n"]
        g = _gen(seed, 5)
        st["lse"], st["entropy"] = (torch.empty(n, device="cuda") for _ in range(2))
        for a in range(0, n, 512):
            x = z[a:a + 512].double() / case["tau"]
            lse = x.logsumexp(1)
            st["lse"][a:a + 512] = lse
            lp = x - lse[:, None]
            st["entropy"][a:a + 512] = -torch.where(lp > -math.inf, lp.exp() * lp, 0.0).sum(1)
        st["d_logp"] = torch.randn(n, device="cuda", generator=g) / n
        st["d_entropy"] = torch.full((n,), -1e-2 / n, device="cuda")
    return st


# ------------------------------------------------------------------ one pass
def _plain_logprob(st):
    z, target, tau, n_top = st["z"], st["target"], st["tau"], st["n_top"]
    n, V = z.shape
    a = z.float() / tau
    lead = a.amax(1, keepdim=True)
    e = (a - lead).exp()
    total = e.sum(1, keepdim=True)
    lse = (lead + total.log()).squeeze(1)
    entropy = total.log().squeeze(1) - (torch.where(e > 0, e * (a - lead), 0.0).sum(1)
                                        / total.squeeze(1))
    ok = (target >= 0) & (target < V)
    logp = a[torch.arange(n, device=z.device), target.clamp(0, V - 1)] - lse
    out = [torch.where(ok, x, 0.0) for x in (logp, entropy, lse)]
    if n_top:
        # the order of the values, then of the indices: one whole number for both
        b = (z.float() + 0.0).view(torch.int32)
        key = (b ^ ((b >> 31) & 0x7FFFFFFF)).long() * (1 << 32)
        key += (1 << 32) - 1 - torch.arange(V, device=z.device)
        idx = (1 << 32) - 1 - (key.topk(n_top, dim=1).values & 0xFFFFFFFF)
        top = a.gather(1, idx) - lse[:, None]
        gone = ~ok[:, None] | (top == -math.inf)
        out += [torch.where(gone, -1, idx).int(), torch.where(gone, -math.inf, top)]
    return out


def _plain_logprob_grad(st):
    z, target, tau = st["z"], st["target"], st["tau"]
    V = z.shape[1]
    ok = ((target >= 0) & (target < V))[:, None]
    lp = z.float() / tau - st["lse"][:, None]
    p = lp.exp()
    dz = -st["d_logp"][:, None] * p
    dz -= st["d_entropy"][:, None] * torch.where(p > 0, p * (lp + st["entropy"][:, None]), 0.0)
    dz.scatter_add_(1, target.clamp(0, V - 1)[:, None], st["d_logp"][:, None])
    return torch.where(ok, dz / tau, 0.0).to(z.dtype)


def _plain_adamw(st):
    g = st["g"].float()
    w = st["p"].float() if st["master"] is None else st["master"]
    if st["bits"] == 8:
        c = st["m"].int()
        m = _decode(c & 127, st["m_exp"], 3)
        m = torch.where(c > 127, -m, m)
        v = _decode(st["v"].int(), st["v_exp"], 4).square()
    else:
        m, v = st["m"], st["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g * g
    at = torch.arange(g.numel() // 32, device=g.device)
    wd = st["wd_of"][torch.searchsorted(st["block_ends"], at, right=True)].unsqueeze(1)
    root = (v / (1 - BETA2 ** STEP)).sqrt() + EPS
    w = w - LR * ((m / (1 - BETA1 ** STEP)) / root + (wd * w.view(-1, 32)).view(-1))
    st["p"].copy_(w)
    if st["master"] is not None:
        st["master"].copy_(w)
    if st["bits"] == 32:
        st["m"].copy_(m)
        st["v"].copy_(v)
        return [x for x in (st["p"], st["master"], m, v) if x is not None]
    for name, (code, E) in (("m", _pack_m(m, STEP)), ("v", _pack_v(v, STEP))):
        st[name].copy_(code)
        st[name + "_exp"].copy_(E)
    c = st["m"].int()
    m = _decode(c & 127, st["m_exp"], 3)
    m = torch.where(c > 127, -m, m)
    root = _decode(st["v"].int(), st["v_exp"], 4)
    # (five significant bits: bf16 holds the values as they are)
    out = (st["p"], st["master"], m.to(torch.bfloat16), root.to(torch.bfloat16))
    return [x for x in out if x is not None]


def _plain_adapter(st):
    n, r, k = st["A"].shape
    d = st["U"].shape[1]
    a = st["adapter"][:, None]
    # every adapter's projection of every row, and the row's own one kept
    P = st["X"].float() @ st["A"].float().view(n * r, k).t()
    keep = torch.where(a == torch.arange(n, device=a.device), st["scale"] * st["unit"], 0.0)
    P = P.view(-1, n, r) * keep[:, :, None]
    delta = P.view(-1, n * r) @ st["U"].float().transpose(1, 2).reshape(n * r, d)
    return (st["Y"].float() + delta).to(torch.bfloat16)


def _own(st):
    import rank_gradient_sketching_amd as lg
    op = st["op"]
    if op == "logprob":
        out = lg.token_logprob(st["z"], st["target"], tau=st["tau"], n_top=st["n_top"])
        return [x for x in out if x is not None]
    if op == "logprob_grad":
        return lg.token_logprob_backward(st["z"], st["target"], st["lse"], st["entropy"],
                                         d_logp=st["d_logp"], d_entropy=st["d_entropy"],
                                         tau=st["tau"])
    if op == "adapter":
        return lg.adapter_apply(st["X"], st["Y"], st["adapter"], st["U"], st["scale"],
                                seeds=st["seeds"], A=None if st["seeds"] is not None else st["A"],
                                out=st["out"])
    if "bound" not in st:               # the handle a program keeps for its tensors
        def cut(x, block=1):
            return [x[a // block:(a + s + block - 1) // block] if block > 1 else x[a:a + s]
                    for a, s in zip(st["starts"], st["sizes"])]
        more = {}
        if st["master"] is not None:
            more["master"] = cut(st["master"])
        if st["bits"] == 8:
            more.update(m_exp=cut(st["m_exp"], 32), v_exp=cut(st["v_exp"], 32))
        st["bound"] = lg.adamw_bind(cut(st["p"]), cut(st["g"]), cut(st["m"]), cut(st["v"]),
                                    weight_decay=st["wd"], **more)
    lg.adamw_step(st["bound"], lr=LR, step=STEP, beta1=BETA1, beta2=BETA2, eps=EPS)
    if st["bits"] == 32:
        out = (st["p"], st["master"], st["m"], st["v"])
    else:
        out = (st["p"], st["master"], lg.adamw_state_values(st["m"], st["m_exp"], "m"),
               lg.adamw_state_values(st["v"], st["v_exp"], "v"))
    return [x for x in out if x is not None]


def run(state):
    if own:
        return _own(state)
    return {"logprob": _plain_logprob, "logprob_grad": _plain_logprob_grad,
            "adamw": _plain_adamw, "adapter": _plain_adapter}[state["op"]](state)


# ------------------------------------------------------------------ in 64 bits
def _exact_logprob(st):
    z, target, n_top = st["z"], st["target"], st["n_top"]
    n, V = z.shape
    parts = []
    for a in range(0, n, 256):
        t = target[a:a + 256]
        ok = (t >= 0) & (t < V)
        lp = torch.log_softmax(z[a:a + 256].double() / st["tau"], 1)
        lse = (z[a:a + 256].double() / st["tau"]).logsumexp(1)
        H = torch.special.entr(lp.exp()).sum(1)
        rows = [lp.gather(1, t.clamp(0, V - 1)[:, None])[:, 0], H, lse]
        rows = [x.masked_fill(~ok, 0) for x in rows]
        if n_top:
            val, idx = lp.sort(dim=1, descending=True, stable=True)
            val, idx = val[:, :n_top].clone(), idx[:, :n_top].clone()
            gone = (val == -math.inf) | ~ok[:, None]
            val[gone], idx[gone] = -math.inf, -1
            rows += [idx.int(), val]
        parts.append(rows)
    return [torch.cat(x) for x in zip(*parts)]


def _exact_logprob_grad(st):
    z, target = st["z"], st["target"]
    out = torch.empty(z.shape, dtype=torch.float64, device=z.device)
    for a in range(0, z.shape[0], 256):
        s = slice(a, a + 256)
        t = target[s]
        ok = (t >= 0) & (t < z.shape[1])
        lp = torch.log_softmax(z[s].double() / st["tau"], 1)
        p = lp.exp()
        H = torch.special.entr(p).sum(1, keepdim=True)
        one = torch.zeros_like(p)
        one[ok.nonzero()[:, 0], t[ok]] = 1
        g1, g2 = (st[x][s].double()[:, None] for x in ("d_logp", "d_entropy"))
        dz = g1 * (one - p) + g2 * (torch.special.entr(p) - p * H)
        out[s] = (dz / st["tau"]).masked_fill(~ok[:, None], 0)
    return out


def _exact_round(x, step, keep, half):
    """x >= 0 in the 8-bit form, by frexp and floor: with q the spacing of `keep`
    mantissa bits at x, floor(x / q + u) q for the dither u in [0, 1)."""
    x = x.float().double()
    i = torch.arange(x.numel(), device=x.device, dtype=torch.int64)
    u = torch.remainder(i * 0x6A09E667 + step * 0x9E3779B9 + half, 1 << 32) // (1 << (9 + keep))
    _, e = torch.frexp(x)
    q = torch.ldexp(torch.ones_like(x), e - 1 - keep)
    y = torch.floor(x / q + u.double() / (1 << (23 - keep))) * q
    y[x == 0] = 0
    _, e = torch.frexp(y.view(-1, 32).amax(1))
    least = torch.ldexp(torch.ones_like(e, dtype=torch.float64),
                        torch.clamp(e - 1, min=16 - 127) - 15)
    least = (least * (1 + 2.0 ** -keep)).repeat_interleave(32)
    small = y < least
    y[small] = 0
    return y, least


def _exact_adamw(case, st):
    out, sizes = [], st["sizes"]
    full = sum(-(-s // 32) * 32 for s in sizes)
    wd = torch.zeros(full, dtype=torch.float64, device="cuda")
    for a, s, x in zip(st["starts"], sizes, st["wd"]):
        wd[a:a + s] = x
    g = st["g"].double()
    w = (st["p"] if st["master"] is None else st["master"]).double()
    if case["bits"] == 8:
        def values(code, E, keep):
            c, E = code.double(), E.double().repeat_interleave(32)
            x = torch.exp2(E - 15 - 127 + torch.floor(c / 2 ** keep))
            return torch.where(c > 0, x * (1 + torch.remainder(c, 2 ** keep) / 2 ** keep), 0.0)
        neg = st["m"] >= 128
        m = values(torch.where(neg, st["m"] - 128, st["m"]), st["m_exp"], 3)
        m = torch.where(neg, -m, m)
        v = values(st["v"], st["v_exp"], 4) ** 2
    else:
        m, v = st["m"].double(), st["v"].double()
    m = m + (g - m) * (1 - BETA1)
    v = v + (g * g - v) * (1 - BETA2)
    step = m / (1 - BETA1 ** STEP) / (torch.sqrt(v / (1 - BETA2 ** STEP)) + EPS)
    w = w * (1 - LR * wd) - LR * step
    out = [w] + ([w] if st["master"] is not None else [])
    if case["bits"] == 32:
        return out + [m, v]
    ym, _ = _exact_round(m.abs(), STEP, 3, 0)
    yv, least = _exact_round(v.sqrt(), STEP, 4, 1 << 31)
    yv = torch.where((v.sqrt().float() > 0) & (yv == 0), least, yv)
    return out + [torch.where(m < 0, -ym, ym), yv]


def _exact_adapter(st):
    out = st["Y"].double()
    for a in range(st["U"].shape[0]):
        at = (st["adapter"] == a).nonzero()[:, 0]
        if at.numel():
            P = st["X"][at].double() @ st["A"][a].double().t().contiguous()
            c = float(st["scale"][a]) / (math.sqrt(st["A"].shape[1]) if st["seeds"] is not None
                                         else 1.0)
            out[at] += c * (P @ st["U"][a].double().t().contiguous())
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, st)
    return {"logprob": _exact_logprob, "logprob_grad": _exact_logprob_grad,
            "adapter": _exact_adapter}[case["op"]](st)
