"""Python binding of the operators around the sketch in one policy step
(include/logra_policy.h): log probabilities of given tokens with entropy and
top alternatives, their gradient down to the logits, AdamW over many tensors,
and the rank-r updates of several policies beside the projection they share.

Argument marshalling only, as in api.py: the work runs in the library's HIP
kernels on the tensors' device, asynchronously on torch's current stream of
that device.  Tensors must live on the GPU; nothing here falls back to the CPU.

Autograd sees none of it, as in the rest of the library: results are detached
(adapter_apply into Y adds no gradient of the update to Y's graph), and writes
into given tensors raise no version counter, so a tensor that autograd has saved
must not be one of them.  A program takes gradients by the calls themselves
(token_logprob_backward) or wraps them in a torch.autograd.Function of its own.
"""
import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from . import _lib
from .api import _rows, _stream, _ws

MAX_TOP = 64         # LOGRA_MAX_TOP
STATE_BLOCK = 32     # LOGRA_STATE_BLOCK
_BF16 = (torch.bfloat16,)
_F32 = (torch.float32,)
_EITHER = (torch.bfloat16, torch.float32)
_I32, _I64, _U8 = (torch.int32,), (torch.int64,), (torch.uint8,)
_TYPES = {torch.bfloat16: 0, torch.float32: 1}   # LOGRA_BF16, LOGRA_F32
# (the raw lookup spares torch.cuda.current_device's initialisation check: every
# tensor that gets here is on the GPU already)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _need(t, name, dtypes, dev=None, shape=None, ndim=None, contiguous=False):
    """Checks one tensor argument: dtypes it may have, device index, shape."""
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes
            and (dev is None or t.get_device() == dev) and (ndim is None or t.dim() == ndim)
            and (shape is None or t.shape == shape) and (not contiguous or t.is_contiguous())):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))} (got {t.dtype})")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} must be on GPU {dev} (got {t.device})")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims (got {t.dim()})")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    raise ValueError(f"{name} must be contiguous")


def _call(name, dev, *args):
    """One library call; launches go to the current device, so the tensors' own
    is made current."""
    fn = getattr(_lib.lib(), name)
    if dev == _current_device():
        st = fn(*args)
    else:
        with torch.cuda.device(dev):
            st = fn(*args)
    if st != 0:
        _lib.check(st, name)


def _matrix(t, name):
    """(rows, cols, row stride) of a 2-D tensor with contiguous rows; the stride
    of a single row (or of none) does not matter and is given a legal value."""
    rows, cols, ld = _rows(t, name)
    return rows, cols, ld if rows > 1 else -(-cols // 8) * 8


def _opt(t, name, n, dev, dtypes=_F32):
    """Address of an optional vector of n entries."""
    if t is None:
        return None
    _need(t, name, dtypes, dev, (n,), contiguous=True)
    return t.data_ptr()


def _workspace(ws, need, like):
    """(address, bytes, tensor) of scratch for a call; the tensor is held until
    the call is enqueued."""
    if need == 0:
        return None, 0, None
    if ws is None:
        ws = torch.empty(need, dtype=torch.uint8, device=like.device)
        return ws.data_ptr(), need, ws
    if isinstance(ws, torch.Tensor) and ws.is_cuda and ws.get_device() != like.get_device():
        raise ValueError(f"ws must be on {like.device} (got {ws.device})")
    return (*_ws(ws), ws)


# ------------------------------------------------------------------ log probabilities
class TokenLogprob(NamedTuple):
    """Results of token_logprob, per row: logp, entropy and lse [n] fp32;
    top_idx [n, n_top] int32 and top_logp [n, n_top] fp32.  None: not asked for."""
    logp: Optional[torch.Tensor]
    entropy: Optional[torch.Tensor]
    lse: Optional[torch.Tensor]
    top_idx: Optional[torch.Tensor]
    top_logp: Optional[torch.Tensor]


@functools.lru_cache(maxsize=256)
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
    _need(z, "z", _EITHER, ndim=2)
    n, V, ld = _matrix(z, "z")
    dev = z.get_device()
    n_top = int(n_top)
    if not 0 <= n_top <= MAX_TOP:
        raise ValueError(f"n_top must be between 0 and {MAX_TOP}")
    if out is None:
        rows = torch.empty((2 if target is None else 3, n), dtype=torch.float32,
                           device=z.device).unbind(0)
        idx = top = None
        if n_top:
            idx = torch.empty((n, n_top), dtype=torch.int32, device=z.device)
            top = torch.empty((n, n_top), dtype=torch.float32, device=z.device)
        out = TokenLogprob(None if target is None else rows[2], rows[0], rows[1], idx, top)
        ptrs = [None if t is None else t.data_ptr() for t in out]
    else:
        if (out.top_idx is None) != (n_top == 0) or (out.top_logp is None) != (n_top == 0):
            raise ValueError("out.top_idx and out.top_logp go with n_top > 0")
        if out.logp is not None and target is None:
            raise ValueError("logp needs target")
        ptrs = [_opt(getattr(out, x), f"out.{x}", n, dev) for x in ("logp", "entropy", "lse")]
        if n_top:
            _need(out.top_idx, "out.top_idx", _I32, dev, (n, n_top), contiguous=True)
            _need(out.top_logp, "out.top_logp", _F32, dev, (n, n_top), contiguous=True)
            ptrs += [out.top_idx.data_ptr(), out.top_logp.data_ptr()]
        else:
            ptrs += [None, None]
    t_ptr = _opt(target, "target", n, dev, _I64)
    ws_ptr, ws_n, ws = _workspace(ws, token_logprob_ws_bytes(n, V, n_top), z)
    _call("logra_token_logprob", dev, z.data_ptr(), _TYPES[z.dtype], n, V, ld, t_ptr, tau, n_top,
          *ptrs, ws_ptr, ws_n, _stream(z))
    return out


def token_logprob_backward(z, target, lse, entropy=None, d_logp=None, d_entropy=None, d_lse=None,
                           tau=1.0, dz=None):
    """The gradient of a loss with respect to z from its gradients with respect
    to logp, entropy and lse (fp32 [n] each, at least one given):
    dz_j = (d_logp ([j = target] - p_j) - d_entropy p_j (log p_j + entropy) +
    d_lse p_j) / tau.  lse (and entropy, with d_entropy) are those of
    token_logprob for the same z and tau.  Rows left out get zeros.  dz: a
    tensor like z to write (z itself: the gradient replaces the logits)."""
    _need(z, "z", _EITHER, ndim=2)
    n, V, ld = _matrix(z, "z")
    dev = z.get_device()
    if dz is None:
        pad = 16 // z.element_size()
        cols = -(-V // pad) * pad
        dz = torch.empty((n, cols), dtype=z.dtype, device=z.device)
        ldz = cols if n > 1 else -(-V // 8) * 8
        if cols != V:
            dz = dz[:, :V]
    else:
        _need(dz, "dz", (z.dtype,), dev, (n, V))
        ldz = _matrix(dz, "dz")[2]
    _need(lse, "lse", _F32, dev, (n,), contiguous=True)
    _call("logra_token_logprob_backward", dev, z.data_ptr(), _TYPES[z.dtype], n, V, ld,
          _opt(target, "target", n, dev, _I64), tau, lse.data_ptr(),
          _opt(entropy, "entropy", n, dev), _opt(d_logp, "d_logp", n, dev),
          _opt(d_entropy, "d_entropy", n, dev), _opt(d_lse, "d_lse", n, dev), dz.data_ptr(), ldz,
          _stream(z))
    return dz


# ------------------------------------------------------------------ AdamW
class _Bound:
    """Tensors of an AdamW step, checked and laid out once (adamw_bind)."""

    def __init__(self, n, table, table_dev, keep):
        self.n, self.table, self.table_dev = n, table, table_dev
        self.device = table_dev.device
        self.address = ctypes.addressof(table)
        self._keep = keep      # the bound storage lives as long as its addresses

    def __len__(self):
        return self.n


def _listed(x, n, name):
    x = [None] * n if x is None else list(x)
    if len(x) != n:
        raise ValueError(f"{name} must have {n} entries (got {len(x)})")
    return x


def _check_apart(spans):
    """spans: (low, high, written, name); raises where a written one overlaps."""
    spans.sort(key=lambda x: x[:2])
    reach, by, w_reach, w_by = 0, None, 0, None      # the furthest of all, and of the written
    for lo, hi, written, name in spans:
        if hi <= lo:
            continue
        if lo < w_reach or (written and lo < reach):
            raise ValueError("%s[%d] overlaps %s[%d]" % (name + (w_by if lo < w_reach else by)))
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
    bind again after giving a tensor other storage (e.g. a new gradient).  It
    copies a table to the GPU, so it is made outside a stream capture, and is
    kept until its steps have run (a captured one: as long as its graph)."""
    params = list(params)
    n = len(params)
    if n == 0:
        raise ValueError("params is empty")
    columns = [("p", params, _EITHER, 1), ("g", _listed(grads, n, "grads"), _EITHER, 1),
               ("m", _listed(m, n, "m"), _F32, 1), ("v", _listed(v, n, "v"), _F32, 1),
               ("master", _listed(master, n, "master"), _F32, 1),
               ("m_exp", _listed(m_exp, n, "m_exp"), _U8, STATE_BLOCK),
               ("v_exp", _listed(v_exp, n, "v_exp"), _U8, STATE_BLOCK)]
    decay = (list(weight_decay) if isinstance(weight_decay, (list, tuple))
             else [weight_decay] * n)
    if len(decay) != n:
        raise ValueError(f"weight_decay must have {n} entries (got {len(decay)})")
    items = (_lib.AdamWItem * n)()
    keep, spans, dev = [], [], None
    exps = columns[5][1], columns[6][1]
    for i in range(n):
        p = params[i]
        if not isinstance(p, torch.Tensor):
            raise TypeError(f"p[{i}] must be a torch.Tensor")
        if dev is None:
            _need(p, "p[0]", _EITHER)
            dev = p.get_device()
        k = p.numel()
        q = items[i]
        state8 = exps[0][i] is not None or exps[1][i] is not None
        for name, column, types, block in columns:
            t = column[i]
            if t is None:
                if name == "master" or (block > 1 and not state8):
                    continue
                raise ValueError(f"{name}[{i}] is missing")
            if state8 and name in ("m", "v"):
                types = _U8
            if not (isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() == dev
                    and t.dtype in types and t.is_contiguous()):
                _need(t, f"{name}[{i}]", types, dev, contiguous=True)
            size = t.numel()
            if size != -(-k // block):
                raise ValueError(f"{name}[{i}] must have {-(-k // block)} entries (got {size})")
            at = t.data_ptr()
            setattr(q, name, at)
            spans.append((at, at + size * t.element_size(), name != "g", (name, i)))
            keep.append(t)
        if q.master is not None and p.dtype != torch.bfloat16:
            raise ValueError(f"master[{i}] needs a bf16 parameter")
        q.n, q.weight_decay = k, decay[i]
        q.p_type, q.g_type = _TYPES[p.dtype], _TYPES[columns[1][1][i].dtype]
    _check_apart(spans)
    # (an alias each: a tensor given other storage does not free this one)
    keep = [t.detach() for t in keep]
    size = int(_lib.lib().logra_adamw_table_bytes(n))
    table = (ctypes.c_uint64 * (size // 8))()
    _lib.check(_lib.lib().logra_adamw_table(n, items, table, size), "logra_adamw_table")
    table_dev = torch.frombuffer(table, dtype=torch.uint8).to(params[0].device)
    return _Bound(n, table, table_dev, keep)


def adamw_step(bound, lr, step, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=None):
    """One AdamW step over the tensors of a handle of adamw_bind, in place:
    m <- beta1 m + (1 - beta1) g, v <- beta2 v + (1 - beta2) g^2,
    w <- w - lr (m / b1 / (sqrt(v / b2) + eps) + weight_decay w), with the bias
    corrections b = 1 - beta^step; step counts from 1.  grad_scale: fp32 GPU
    tensor of one entry that scales every gradient (a loss scale's inverse, a
    clipping factor), read on the GPU.  For parameters that are not sketched;
    sketch_update steps a sketch.  A captured call replays its lr and step: with
    8-bit states the same dither each time, which rounds with a bias, so those
    are stepped outside the graph.  Returns None."""
    if not isinstance(bound, _Bound):
        raise TypeError("bound must be a handle of adamw_bind")
    dev = bound.table_dev.get_device()
    scale = None
    if grad_scale is not None:
        _need(grad_scale, "grad_scale", _F32, dev)
        if grad_scale.numel() != 1:
            raise ValueError("grad_scale must have one entry")
        scale = grad_scale.data_ptr()
    _call("logra_adamw_step", dev, bound.address, bound.table_dev.data_ptr(), lr, beta1, beta2,
          eps, step, scale, _stream(bound))


def adamw_state_values(codes, exps, which, out=None):
    """bf16 values of an 8-bit state: which "m", or "v" for sqrt(v).  codes uint8
    (any shape, contiguous), exps uint8 with one entry per 32 codes."""
    if which not in ("m", "v"):
        raise ValueError('which must be "m" or "v"')
    _need(codes, "codes", _U8, contiguous=True)
    n = codes.numel()
    dev = codes.get_device()
    _need(exps, "exps", _U8, dev, contiguous=True)
    if exps.numel() != -(-n // STATE_BLOCK):
        raise ValueError(f"exps must have {-(-n // STATE_BLOCK)} entries (got {exps.numel()})")
    if out is None:
        out = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
    else:
        _need(out, "out", _BF16, dev, codes.shape, contiguous=True)
    _call("logra_adamw_state_values", dev, 0 if which == "m" else 1, codes.data_ptr(),
          exps.data_ptr(), n, out.data_ptr(), _stream(codes))
    return out


# ------------------------------------------------------------------ unmerged updates
@functools.lru_cache(maxsize=256)
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
    _need(X, "X", _BF16, ndim=2)
    dev = X.get_device()
    T, k, ldx = _matrix(X, "X")
    _need(Y, "Y", _BF16, dev, ndim=2)
    T2, d, ldy = _matrix(Y, "Y")
    if T2 != T:
        raise ValueError(f"X has {T} rows but Y has {T2}")
    if out is None:
        out, ldo = Y, ldy
    else:
        _need(out, "out", _BF16, dev, (T, d))
        ldo = _matrix(out, "out")[2]
    _need(U, "U", _EITHER, dev, ndim=3, contiguous=True)
    n, d2, r = U.shape
    if d2 != d:
        raise ValueError(f"Y has {d} columns but U is for {d2}")
    _need(adapter, "adapter", _I32, dev, (T,), contiguous=True)
    _need(scale, "scale", _F32, dev, (n,), contiguous=True)
    if (seeds is None) == (A is None):
        raise ValueError("give seeds (sign bases) or A")
    s_ptr = a_ptr = None
    lda = 0
    if seeds is not None:
        _need(seeds, "seeds", _I64, dev, (n, 2), contiguous=True)
        s_ptr = seeds.data_ptr()
    else:
        _need(A, "A", _BF16, dev, (n, r, k))
        if k > 1 and A.stride(2) != 1:
            raise ValueError("A must have contiguous rows")
        if n > 1 and r > 1 and A.stride(0) != r * A.stride(1):
            raise ValueError("the policies of A must lie r rows apart")
        lda = A.stride(1) if r > 1 else A.stride(0) if n > 1 else -(-k // 8) * 8
        a_ptr = A.data_ptr()
    ws_ptr, ws_n, ws = _workspace(ws, adapter_ws_bytes(T, d, k, r), X)
    _call("logra_adapter_apply", dev, X.data_ptr(), ldx, Y.data_ptr(), ldy, out.data_ptr(), ldo, T,
          d, k, r, n, adapter.data_ptr(), U.data_ptr(), _TYPES[U.dtype], s_ptr, a_ptr, lda,
          scale.data_ptr(), ws_ptr, ws_n, _stream(X))
    return out
