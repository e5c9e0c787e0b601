"""Python binding of the operators around the sketch in one policy step
(include/logra_policy.h): log probabilities of given tokens with entropy and
top alternatives, their gradient down to the logits, AdamW over many tensors,
and the rank-r updates of several policies beside the projection they share.

Argument marshalling only, as in api.py: the work runs in the library's HIP
kernels on the tensors' device, asynchronously on torch's current stream of
that device.  Tensors must live on the GPU; nothing here falls back to the CPU.
"""
import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch

from . import _lib
from .api import _rows, _stream, _ws

MAX_TOP = 64         # LOGRA_MAX_TOP
STATE_BLOCK = 32     # LOGRA_STATE_BLOCK
_TYPES = {torch.bfloat16: 0, torch.float32: 1}   # LOGRA_BF16, LOGRA_F32
_same_device = contextlib.nullcontext()


def _need(t, name, dtypes, device=None, shape=None, ndim=None, contiguous=False):
    """Checks one tensor argument; dtypes: the types it may have."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device} (got {t.device})")
    if t.dtype not in dtypes:
        want = " or ".join(str(d) for d in dtypes)
        raise ValueError(f"{name} must be {want} (got {t.dtype})")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims (got {t.dim()})")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _on(device):
    """Launches go to the current device, so make it the tensors' own."""
    return (_same_device if device.index == torch.cuda.current_device()
            else torch.cuda.device(device))


def _matrix(t, name):
    """(rows, cols, row stride) of a 2-D tensor with contiguous rows; the stride
    of a single row (or of none) does not matter and is given a legal value."""
    rows, cols, ld = _rows(t, name)
    return rows, cols, ld if rows > 1 else -(-cols // 8) * 8


def _opt(t, name, n, device, dtype=torch.float32):
    """Address of an optional vector of n entries."""
    if t is None:
        return None
    _need(t, name, (dtype,), device, shape=(n,), contiguous=True)
    return t.data_ptr()


def _workspace(ws, need, device):
    if need == 0:
        return None, 0
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=device)
    elif isinstance(ws, torch.Tensor) and ws.device != device:
        raise ValueError(f"ws must be on {device} (got {ws.device})")
    return _ws(ws)


# ------------------------------------------------------------------ log probabilities
class TokenLogprob(NamedTuple):
    """Results of token_logprob, per row: logp, entropy and lse [n] fp32;
    top_idx [n, n_top] int32 and top_logp [n, n_top] fp32.  None: not asked for."""
    logp: Optional[torch.Tensor]
    entropy: Optional[torch.Tensor]
    lse: Optional[torch.Tensor]
    top_idx: Optional[torch.Tensor]
    top_logp: Optional[torch.Tensor]


def token_logprob_ws_bytes(n_tok, vocab, n_top=0):
    return int(_lib.lib().logra_token_logprob_ws_bytes(n_tok, vocab, n_top))


def token_logprob(z, target=None, tau=1.0, n_top=0, out=None, ws=None):
    """Log probability of target[t] under softmax(z[t] / tau), the entropy and
    log normaliser of that distribution, and its n_top most probable tokens
    (equal logits in the order of their index): a TokenLogprob.

    z: [n, vocab] bf16 or fp32, rows on 16-byte boundaries.  target: int64 [n];
    a row whose target lies outside [0, vocab) (e.g. -100) is left out: zeros,
    index -1 and -inf among the alternatives.  Without target there is no logp.
    -inf logits are tokens of probability zero and no alternatives.
    out: a TokenLogprob of contiguous tensors to write; its None entries are
    not computed (top_* are given exactly when n_top > 0).  ws: scratch of
    token_logprob_ws_bytes(n, vocab, n_top) bytes."""
    _need(z, "z", (torch.bfloat16, torch.float32), ndim=2)
    n, V, ld = _matrix(z, "z")
    dev = z.device
    n_top = int(n_top)
    if not 0 <= n_top <= MAX_TOP:
        raise ValueError(f"n_top must be between 0 and {MAX_TOP}")
    if out is None:
        rows = torch.empty((2 if target is None else 3, n), dtype=torch.float32, device=dev)
        top = ((torch.empty((n, n_top), dtype=torch.int32, device=dev),
                torch.empty((n, n_top), dtype=torch.float32, device=dev))
               if n_top else (None, None))
        out = TokenLogprob(None if target is None else rows[2], rows[0], rows[1], *top)
    if (out.top_idx is None) != (n_top == 0) or (out.top_logp is None) != (n_top == 0):
        raise ValueError("out.top_idx and out.top_logp go with n_top > 0")
    if n_top:
        _need(out.top_idx, "out.top_idx", (torch.int32,), dev, (n, n_top), contiguous=True)
        _need(out.top_logp, "out.top_logp", (torch.float32,), dev, (n, n_top), contiguous=True)
    if out.logp is not None and target is None:
        raise ValueError("logp needs target")
    ptrs = [_opt(getattr(out, x), f"out.{x}", n, dev) for x in ("logp", "entropy", "lse")]
    ptrs += [t.data_ptr() if n_top else None for t in (out.top_idx, out.top_logp)]
    t_ptr = _opt(target, "target", n, dev, torch.int64)
    ws_ptr, ws_n = _workspace(ws, token_logprob_ws_bytes(n, V, n_top), dev)
    with _on(dev):
        st = _lib.lib().logra_token_logprob(z.data_ptr(), _TYPES[z.dtype], n, V, ld, t_ptr,
                                            float(tau), n_top, *ptrs, ws_ptr, ws_n, _stream(z))
    _lib.check(st, "logra_token_logprob")
    return out


def token_logprob_backward(z, target, lse, entropy=None, d_logp=None, d_entropy=None, d_lse=None,
                           tau=1.0, dz=None):
    """The gradient of a loss with respect to z from its gradients with respect
    to logp, entropy and lse (fp32 [n] each, at least one given):
    dz_j = (d_logp ([j = target] - p_j) - d_entropy p_j (log p_j + entropy) +
    d_lse p_j) / tau.  lse (and entropy, with d_entropy) are those of
    token_logprob for the same z and tau.  Rows left out get zeros.  dz: a
    tensor like z to write (z itself: the gradient replaces the logits)."""
    _need(z, "z", (torch.bfloat16, torch.float32), ndim=2)
    n, V, ld = _matrix(z, "z")
    dev = z.device
    if dz is None:
        pad = 16 // z.element_size()
        dz = torch.empty((n, -(-V // pad) * pad), dtype=z.dtype, device=dev)[:, :V]
    _need(dz, "dz", (z.dtype,), dev, (n, V))
    ldz = _matrix(dz, "dz")[2]
    _need(lse, "lse", (torch.float32,), dev, (n,), contiguous=True)
    ptrs = [_opt(t, name, n, dev) for name, t in
            (("entropy", entropy), ("d_logp", d_logp), ("d_entropy", d_entropy),
             ("d_lse", d_lse))]
    t_ptr = _opt(target, "target", n, dev, torch.int64)
    with _on(dev):
        st = _lib.lib().logra_token_logprob_backward(
            z.data_ptr(), _TYPES[z.dtype], n, V, ld, t_ptr, float(tau), lse.data_ptr(), *ptrs,
            dz.data_ptr(), ldz, _stream(z))
    _lib.check(st, "logra_token_logprob_backward")
    return dz


# ------------------------------------------------------------------ AdamW
class _Bound:
    """Tensors of an AdamW step, checked and laid out once (adamw_bind)."""

    def __init__(self, items, device, keep):
        self.items, self.device = items, device
        self._keep = keep      # the bound storage lives as long as the addresses

    def __len__(self):
        return len(self.items)


def _lists(n, **named):
    out = []
    for name, x in named.items():
        if x is None:
            x = [None] * n
        if len(x) != n:
            raise ValueError(f"{name} must have {n} entries (got {len(x)})")
        out.append(list(x))
    return out


def _check_apart(spans):
    """spans: (low, high, written, name); raises where a written one overlaps."""
    spans.sort(key=lambda x: (x[0], x[1]))
    reach, by, w_reach, w_by = 0, None, 0, None      # the furthest of all, and of the written
    for lo, hi, written, name in spans:
        if hi <= lo:
            continue
        if lo < w_reach or (written and lo < reach):
            raise ValueError(f"{name} overlaps {w_by if lo < w_reach else by}")
        if hi > reach:
            reach, by = hi, name
        if written and hi > w_reach:
            w_reach, w_by = hi, name


def adamw_bind(params, grads, m, v, master=None, m_exp=None, v_exp=None, weight_decay=0.0):
    """Checks the tensors of an AdamW step once and returns a handle for
    adamw_step.  Lists of equal length: params (bf16 or fp32, updated in
    place), grads (bf16 or fp32), m and v (fp32, or uint8 codes of 8-bit states
    with their block exponents m_exp and v_exp: uint8, one per 32 entries; all
    zero is the zero state), master (fp32 weights behind bf16 params, or None
    entries); weight_decay: one number or a list.  All contiguous, on one GPU.
    The handle keeps the storage that the tensors have now and steps that:
    bind again after giving a tensor other storage (e.g. a new gradient)."""
    params = list(params)
    n = len(params)
    if n == 0:
        raise ValueError("params is empty")
    grads, m, v, master, m_exp, v_exp = _lists(n, grads=grads, m=m, v=v, master=master,
                                               m_exp=m_exp, v_exp=v_exp)
    decay = (list(weight_decay) if isinstance(weight_decay, (list, tuple))
             else [weight_decay] * n)
    if len(decay) != n:
        raise ValueError(f"weight_decay must have {n} entries (got {len(decay)})")
    items = (_lib.AdamWItem * n)()
    keep, spans, dev = [], [], None
    both = (torch.bfloat16, torch.float32)
    for i in range(n):
        p = params[i]
        _need(p, f"params[{i}]", both, dev, contiguous=True)
        dev = p.device
        k = p.numel()
        q = items[i]
        q.n, q.weight_decay = k, float(decay[i])
        q.p_type, q.g_type = _TYPES[p.dtype], 0
        state8 = m_exp[i] is not None or v_exp[i] is not None
        st = (torch.uint8,) if state8 else (torch.float32,)
        blocks = -(-k // STATE_BLOCK)
        for name, t, types, size, written in (
                ("p", p, both, k, True), ("g", grads[i], both, k, False),
                ("m", m[i], st, k, True), ("v", v[i], st, k, True),
                ("master", master[i], (torch.float32,), k, True),
                ("m_exp", m_exp[i], (torch.uint8,), blocks, True),
                ("v_exp", v_exp[i], (torch.uint8,), blocks, True)):
            if t is None:
                if name == "master" or (name.endswith("_exp") and not state8):
                    continue
                raise ValueError(f"{name}[{i}] is missing")
            _need(t, f"{name}[{i}]", types, dev, contiguous=True)
            if t.numel() != size:
                raise ValueError(f"{name}[{i}] must have {size} entries (got {t.numel()})")
            if name == "g":
                q.g_type = _TYPES[t.dtype]
            if name == "master" and p.dtype != torch.bfloat16:
                raise ValueError(f"master[{i}] needs a bf16 parameter")
            setattr(q, name, t.data_ptr())
            spans.append((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), written,
                          f"{name}[{i}]"))
            keep.append(t.detach())
    _check_apart(spans)
    return _Bound(items, dev, keep)


def adamw_step(bound, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=None):
    """One AdamW step over the tensors of a handle of adamw_bind, in place:
    m <- beta1 m + (1 - beta1) g, v <- beta2 v + (1 - beta2) g^2,
    w <- w - lr (m / b1 / (sqrt(v / b2) + eps) + weight_decay w), with the bias
    corrections b = 1 - beta^step; step counts from 1.  grad_scale: fp32 GPU
    tensor of one entry that scales every gradient (a loss scale's inverse, a
    clipping factor), read on the GPU.  For parameters that are not sketched;
    sketch_update steps a sketch.  Returns None."""
    if not isinstance(bound, _Bound):
        raise TypeError("bound must be a handle of adamw_bind")
    scale = None
    if grad_scale is not None:
        _need(grad_scale, "grad_scale", (torch.float32,), bound.device)
        if grad_scale.numel() != 1:
            raise ValueError("grad_scale must have one entry")
        scale = grad_scale.data_ptr()
    with _on(bound.device):
        st = _lib.lib().logra_adamw_step(len(bound.items), bound.items, float(lr), float(beta1),
                                         float(beta2), float(eps), int(step), scale,
                                         _stream(bound))
    _lib.check(st, "logra_adamw_step")


def adamw_state_values(codes, exps, which, out=None):
    """bf16 values of an 8-bit state: which "m", or "v" for sqrt(v).  codes uint8
    (any shape, contiguous), exps uint8 with one entry per 32 codes."""
    if which not in ("m", "v"):
        raise ValueError('which must be "m" or "v"')
    _need(codes, "codes", (torch.uint8,), contiguous=True)
    n = codes.numel()
    _need(exps, "exps", (torch.uint8,), codes.device, contiguous=True)
    if exps.numel() != -(-n // STATE_BLOCK):
        raise ValueError(f"exps must have {-(-n // STATE_BLOCK)} entries (got {exps.numel()})")
    if out is None:
        out = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
    _need(out, "out", (torch.bfloat16,), codes.device, codes.shape, contiguous=True)
    with _on(codes.device):
        st = _lib.lib().logra_adamw_state_values(0 if which == "m" else 1, codes.data_ptr(),
                                                 exps.data_ptr(), n, out.data_ptr(),
                                                 _stream(codes))
    _lib.check(st, "logra_adamw_state_values")
    return out


# ------------------------------------------------------------------ unmerged updates
def adapter_ws_bytes(T, d, k, r):
    return int(_lib.lib().logra_adapter_ws_bytes(T, d, k, r))


def adapter_apply(X, Y, adapter, U, scale, seeds=None, A=None, out=None, ws=None):
    """out[t] = Y[t] + c scale[a] (X[t] A_a^T) U_a^T, a = adapter[t]: the rank-r
    updates of several policies beside the projection Y = X W^T they share,
    W left alone; returns out (Y itself when None).

    X [T, k], Y and out [T, d] bf16; adapter int32 [T], rows with an index
    outside [0, n) keep Y's bits; U [n, d, r] fp32 or bf16 contiguous; scale
    fp32 [n] (minus alpha eta for the update W - alpha eta U A).  Bases: seeds
    int64 [n, 2] (seed and stream of each policy's sign basis; c = 1/sqrt(r)),
    or A [n, r, k] bf16 (c = 1), e.g. Gaussian ones from regen_A.  ws: scratch
    of adapter_ws_bytes(T, d, k, r) bytes."""
    _need(X, "X", (torch.bfloat16,), ndim=2)
    dev = X.device
    T, k, ldx = _matrix(X, "X")
    _need(Y, "Y", (torch.bfloat16,), dev, ndim=2)
    T2, d, ldy = _matrix(Y, "Y")
    if T2 != T:
        raise ValueError(f"X has {T} rows but Y has {T2}")
    if out is None:
        out = Y
    _need(out, "out", (torch.bfloat16,), dev, (T, d))
    ldo = _matrix(out, "out")[2]
    _need(U, "U", (torch.float32, torch.bfloat16), dev, ndim=3, contiguous=True)
    n, d2, r = U.shape
    if d2 != d:
        raise ValueError(f"Y has {d} columns but U is for {d2}")
    _need(adapter, "adapter", (torch.int32,), dev, (T,), contiguous=True)
    _need(scale, "scale", (torch.float32,), dev, (n,), contiguous=True)
    if (seeds is None) == (A is None):
        raise ValueError("give seeds (sign bases) or A")
    s_ptr = a_ptr = None
    lda = 0
    if seeds is not None:
        _need(seeds, "seeds", (torch.int64,), dev, (n, 2), contiguous=True)
        s_ptr = seeds.data_ptr()
    else:
        _need(A, "A", (torch.bfloat16,), dev, (n, r, k))
        rows = A.as_strided((n * r, k), (A.stride(1) if r > 1 else A.stride(0), A.stride(2)))
        if n > 1 and r > 1 and A.stride(0) != r * A.stride(1):
            raise ValueError("the policies of A must lie r rows apart")
        lda = _matrix(rows, "A")[2]
        a_ptr = A.data_ptr()
    ws_ptr, ws_n = _workspace(ws, adapter_ws_bytes(T, d, k, r), dev)
    with _on(dev):
        st = _lib.lib().logra_adapter_apply(
            X.data_ptr(), ldx, Y.data_ptr(), ldy, out.data_ptr(), ldo, T, d, k, r, n,
            adapter.data_ptr(), U.data_ptr(), _TYPES[U.dtype], s_ptr, a_ptr, lda,
            scale.data_ptr(), ws_ptr, ws_n, _stream(X))
    _lib.check(st, "logra_adapter_apply")
    return out
