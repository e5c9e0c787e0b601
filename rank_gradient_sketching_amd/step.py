"""Python binding of the operators that close a policy step
(include/logra_step.h): drawing tokens from logits, the layer product with its
epilogue and its gradients, and the global gradient norm with clipping.

Argument marshalling only, as in api.py and policy.py: the work runs in the
library's HIP kernels on the tensors' device, asynchronously on torch's current
stream of that device; autograd sees none of it.
"""
import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from . import _lib
from .api import _stream
from .policy import (_BF16, _EITHER, _F32, _I32, _I64, _TYPES, _call, _check_apart, _listed,
                     _matrix, _need, _opt, _workspace)

ACTIVATIONS = (None, "relu", "silu", "gelu", "gelu_tanh")   # LOGRA_ACT_*
_ACT = {name: i for i, name in enumerate(ACTIVATIONS)}
_NORMS = {2: 0, 2.0: 0, "inf": 1, float("inf"): 1}          # LOGRA_NORM_*


# ------------------------------------------------------------------ sampling
class SampledTokens(NamedTuple):
    """Results of sample_tokens, per row: token [n] int64, logp and logq [n] fp32,
    kept [n] int32.  None: not asked for (token always is)."""
    token: torch.Tensor
    logp: Optional[torch.Tensor]
    logq: Optional[torch.Tensor]
    kept: Optional[torch.Tensor]


@functools.lru_cache(maxsize=256)
def sample_tokens_ws_bytes(n_tok, vocab):
    return int(_lib.lib().logra_sample_tokens_ws_bytes(n_tok, vocab))


def sample_tokens(z, u, tau=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None, ws=None):
    """One token per row of logits z [n, vocab] (bf16 or fp32, rows on 16-byte
    boundaries) from the random number u[t] (fp32 [n], uniform in [0, 1)): a
    SampledTokens.

    The tokens of a row stand in descending order of z (equal ones by their
    index); kept are the first top_k of them (0: all), of those the fewest with
    probability mass >= top_p (1: all), and those with a probability >= min_p of
    the largest one's; at least one.  The token is the first whose cumulative mass
    exceeds u times the kept ones'.  logp is its log probability under
    softmax(z / tau), as token_logprob gives it; logq that under the kept tokens
    alone; kept their number.

    tau, top_k, top_p, min_p: a number, or a tensor of one per row (fp32 [n];
    top_k int32 [n]).  A row with u outside [0, 1) (e.g. -1: an ended sequence)
    gives token -1, zeros and nothing kept; a row with a NaN or +inf logit, with
    none above -inf, or with a setting out of range (tau > 0 finite, 0 < top_p <=
    1, 0 <= min_p <= 1) token -1, NaN, NaN and 0.  out: a SampledTokens of
    contiguous tensors to write, whose None entries are not computed.  ws: scratch
    of sample_tokens_ws_bytes(n, vocab) bytes."""
    _need(z, "z", _EITHER, ndim=2)
    n, V, ld = _matrix(z, "z")
    dev = z.get_device()
    _need(u, "u", _F32, dev, (n,), contiguous=True)
    scalars, rows = [], []
    for name, x, dtypes, default in (("tau", tau, _F32, 1.0), ("top_k", top_k, _I32, 0),
                                     ("top_p", top_p, _F32, 1.0), ("min_p", min_p, _F32, 0.0)):
        per_row = isinstance(x, torch.Tensor)
        rows.append(_opt(x, name, n, dev, dtypes) if per_row else None)
        if not per_row and name == "top_k" and not 0 <= x < 1 << 31:
            raise ValueError(f"top_k must be between 0 and 2^31 - 1 (got {x})")
        scalars.append(default if per_row else x)
    if out is None:
        device = z.device
        out = SampledTokens(torch.empty(n, dtype=torch.int64, device=device),
                            torch.empty(n, dtype=torch.float32, device=device),
                            torch.empty(n, dtype=torch.float32, device=device),
                            torch.empty(n, dtype=torch.int32, device=device))
        ptrs = [t.data_ptr() for t in out]
    else:
        _need(out.token, "out.token", _I64, dev, (n,), contiguous=True)
        ptrs = [out.token.data_ptr(), _opt(out.logp, "out.logp", n, dev),
                _opt(out.logq, "out.logq", n, dev), _opt(out.kept, "out.kept", n, dev, _I32)]
    ws_ptr, ws_n, ws = _workspace(ws, sample_tokens_ws_bytes(n, V), z)
    _call("logra_sample_tokens", dev, z.data_ptr(), _TYPES[z.dtype], n, V, ld, u.data_ptr(),
          *scalars, *rows, *ptrs, ws_ptr, ws_n, _stream(z))
    return out


# ------------------------------------------------------------------ gradient norm
class GradNorm(NamedTuple):
    """Results of grad_norm: norm and scale [1] fp32, norms [n] fp32 or None."""
    norm: torch.Tensor
    scale: torch.Tensor
    norms: Optional[torch.Tensor]


class _BoundGrads:
    """Tensors of a gradient norm, checked and laid out once (grad_norm_bind)."""

    def __init__(self, n, table, table_dev, keep):
        self.n, self.table, self.table_dev = n, table, table_dev
        self.device = table_dev.device
        self.address = ctypes.addressof(table)
        self.ws_bytes = int(_lib.lib().logra_grad_norm_ws_bytes(self.address))
        self._keep = keep      # the bound storage lives as long as its addresses

    def __len__(self):
        return self.n


def _bound(bound):
    if not isinstance(bound, _BoundGrads):
        raise TypeError("bound must be a handle of grad_norm_bind")
    return bound.table_dev.get_device()


def grad_norm_bind(grads, out=None):
    """Checks gradients (bf16 or fp32, contiguous, on one GPU; sketches S among
    them) once and returns a handle for grad_norm and grad_clip.  out: tensors of
    the same sizes (bf16 or fp32) that grad_clip writes, or None entries: it
    writes the gradient itself.  No two of what is written may overlap, nor a
    gradient with another's out.  The handle keeps the storage that the tensors
    have now: bind again after giving one other storage.  It copies a table to the
    GPU, so it is made outside a stream capture, and is kept until its calls have
    run (a captured one: as long as its graph).  It takes the host about 1.2 us a
    tensor, so a program with many of them keeps its gradients' storage from step
    to step (zero_grad(set_to_none=False)) and binds once."""
    grads = list(grads)
    n = len(grads)
    if n == 0:
        raise ValueError("grads is empty")
    outs = _listed(out, n, "out")
    items = (_lib.GradItem * n)()
    keep, spans, dev = [], [], None
    for i, (g, o) in enumerate(zip(grads, outs)):
        _need(g, f"grads[{i}]", _EITHER, dev, contiguous=True)
        dev = g.get_device()
        q, at, k = items[i], g.data_ptr(), g.numel()
        q.g, q.n, q.g_type = at, k, _TYPES[g.dtype]
        keep.append(g.untyped_storage())
        in_place = o is None
        if not in_place:
            _need(o, f"out[{i}]", _EITHER, dev, contiguous=True)
            if o.numel() != k:
                raise ValueError(f"out[{i}] must have {k} entries (got {o.numel()})")
            to = o.data_ptr()
            q.out, q.out_type = to, _TYPES[o.dtype]
            keep.append(o.untyped_storage())
            in_place = to == at and o.dtype == g.dtype
            if not in_place:
                spans.append((to, to + k * o.element_size(), True, ("out", i)))
        spans.append((at, at + k * g.element_size(), in_place, ("grads", i)))
    _check_apart(spans)
    size = int(_lib.lib().logra_grad_table_bytes(n))
    if size == 0:
        raise ValueError(f"{n} tensors are too many for one handle")
    table = (ctypes.c_uint64 * (size // 8))()
    _lib.check(_lib.lib().logra_grad_table(n, items, table, size), "logra_grad_table")
    table_dev = torch.frombuffer(table, dtype=torch.uint8).to(grads[0].device)
    return _BoundGrads(n, table, table_dev, keep)


def grad_norm(bound, max_norm=None, grad_scale=None, norm_type=2, per_tensor=False, out=None,
              ws=None):
    """The norm of all gradients of a handle as one vector, times |grad_scale|, and
    the factor that clips it to max_norm (None: no clipping): a GradNorm.
    scale = grad_scale min(1, max_norm / norm) is adamw_step's grad_scale, read on
    the GPU.  grad_scale: fp32 GPU tensor of one entry (a loss scale's inverse).
    norm_type: 2, or "inf" for the largest magnitude.  per_tensor: each tensor's own
    norm too.  A NaN gradient makes norm and scale NaN, an infinite one norm infinite
    and scale zero.  out: a GradNorm to write.  ws: scratch of bound.ws_bytes bytes."""
    dev = _bound(bound)
    if norm_type not in _NORMS:
        raise ValueError('norm_type must be 2 or "inf"')
    s_ptr = None
    if grad_scale is not None:
        _need(grad_scale, "grad_scale", _F32, dev)
        if grad_scale.numel() != 1:
            raise ValueError("grad_scale must have one entry")
        s_ptr = grad_scale.data_ptr()
    like = bound.table_dev
    if out is None:
        device = bound.device      # (new tensors cost the host less than views of one)
        out = GradNorm(torch.empty(1, dtype=torch.float32, device=device),
                       torch.empty(1, dtype=torch.float32, device=device),
                       torch.empty(bound.n, dtype=torch.float32, device=device)
                       if per_tensor else None)
    else:
        for name in ("norm", "scale"):
            _need(getattr(out, name), f"out.{name}", _F32, dev, (1,))
        if (out.norms is not None) != bool(per_tensor):
            raise ValueError("out.norms goes with per_tensor")
    norms = _opt(out.norms, "out.norms", bound.n, dev)
    ws_ptr, ws_n, ws = _workspace(ws, bound.ws_bytes, like)
    _call("logra_grad_norm", dev, bound.address, like.data_ptr(), _NORMS[norm_type],
          float("inf") if max_norm is None else max_norm, s_ptr, out.norm.data_ptr(),
          out.scale.data_ptr(), norms, ws_ptr, ws_n, _stream(bound))
    return out


def grad_clip(bound, scale):
    """Every gradient of a handle times scale (fp32 GPU tensor of one entry, e.g.
    grad_norm's), rounded once to the type written: into its out, or in place
    (where a scale of 1 leaves it alone).  For what no optimizer step scales by
    itself (a sketch before sketch_update or merge).  Returns None."""
    dev = _bound(bound)
    _need(scale, "scale", _F32, dev)
    if scale.numel() != 1:
        raise ValueError("scale must have one entry")
    _call("logra_grad_clip", dev, bound.address, bound.table_dev.data_ptr(), scale.data_ptr(),
          _stream(bound))


# ------------------------------------------------------------------ layer product
@functools.lru_cache(maxsize=1024)
def linear_ws_bytes(T, d, k):
    return int(_lib.lib().logra_linear_ws_bytes(T, d, k))


@functools.lru_cache(maxsize=1024)
def linear_backward_act_ws_bytes(T, d):
    return int(_lib.lib().logra_linear_backward_act_ws_bytes(T, d))


def _act(act):
    if act not in _ACT:
        raise ValueError(f"act must be one of {ACTIVATIONS} (got {act!r})")
    return _ACT[act]


def _rows_out(rows, cols, dtype, like):
    """(tensor, row stride) of a new rows x cols result with rows on 16 bytes."""
    wide = -(-cols // 8) * 8
    t = torch.empty((rows, wide), dtype=dtype, device=like.device)
    return (t if wide == cols else t[:, :cols]), wide


def _given(t, name, dtypes, dev, rows, cols):
    """(address, row stride) of a matrix argument of known shape; None: (None, 0)."""
    if t is None:
        return None, 0
    _need(t, name, dtypes, dev, (rows, cols))
    return t.data_ptr(), _matrix(t, name)[2]


def linear(X, W, bias=None, act=None, residual=None, out=None, pre=None, out_dtype=None, ws=None):
    """out = act(X W^T + bias) + residual; returns out.

    X [T, k], W [d, k] bf16; bias bf16 or fp32 [d]; act one of ACTIVATIONS;
    residual bf16 [T, d].  out: bf16 or fp32 [T, d] to write (residual itself:
    added in place), else a new one of out_dtype (bf16).  pre: bf16 [T, d] to
    write X W^T + bias to, for linear_backward_act.  ws: scratch of
    linear_ws_bytes(T, d, k) bytes."""
    _need(X, "X", _BF16, ndim=2)
    dev = X.get_device()
    T, k, ldx = _matrix(X, "X")
    _need(W, "W", _BF16, dev, ndim=2)
    d, k2, ldw = _matrix(W, "W")
    if k2 != k:
        raise ValueError(f"X has {k} columns but W has {k2}")
    b_ptr = _opt(bias, "bias", d, dev, _EITHER)
    r_ptr, ldr = _given(residual, "residual", _BF16, dev, T, d)
    if out is None:
        if out_dtype not in (None, *_EITHER):
            raise ValueError(f"out_dtype must be bfloat16 or float32 (got {out_dtype})")
        out, ldo = _rows_out(T, d, out_dtype or torch.bfloat16, X)
        o_ptr = out.data_ptr()
    else:
        if out_dtype not in (None, out.dtype):
            raise ValueError(f"out is {out.dtype} but out_dtype {out_dtype}")
        o_ptr, ldo = _given(out, "out", _EITHER, dev, T, d)
    p_ptr, ldp = _given(pre, "pre", _BF16, dev, T, d)
    ws_ptr, ws_n, ws = _workspace(ws, linear_ws_bytes(T, d, k), X)
    _call("logra_linear", dev, X.data_ptr(), ldx, W.data_ptr(), ldw, T, d, k, b_ptr,
          0 if bias is None else _TYPES[bias.dtype], _act(act), r_ptr, ldr, o_ptr,
          _TYPES[out.dtype], ldo, p_ptr, ldp, ws_ptr, ws_n, _stream(X))
    return out


def linear_backward_act(d_out, pre=None, act=None, dY=None, d_bias=None, ws=None):
    """dY = d_out act'(pre) in bf16, and its sum over the rows before rounding, the
    bias's gradient; returns dY.

    d_out [T, d] bf16 or fp32; pre bf16 [T, d] of linear (None without act); dY:
    bf16 [T, d] to write (d_out or pre itself among them).  d_bias: fp32 [d] to
    write.  Without act and dY nothing but d_bias is computed and a bf16 d_out is
    returned as it is (an fp32 one is rounded).  dY is what sketch_accumulate,
    linear_backward_input and linear_backward_weight take.  ws: scratch of
    linear_backward_act_ws_bytes(T, d) bytes."""
    _need(d_out, "d_out", _EITHER, ndim=2)
    dev = d_out.get_device()
    T, d, ldd = _matrix(d_out, "d_out")
    a = _act(act)
    if (pre is None) != (a == 0):
        raise ValueError("pre goes with act")
    p_ptr, ldp = _given(pre, "pre", _BF16, dev, T, d)
    b_ptr = _opt(d_bias, "d_bias", d, dev)
    ldy = 0
    if dY is not None:
        y_ptr, ldy = _given(dY, "dY", _BF16, dev, T, d)
    elif a == 0 and d_out.dtype == torch.bfloat16:
        dY, y_ptr = d_out, None
        if d_bias is None:
            return dY
    else:
        dY, ldy = _rows_out(T, d, torch.bfloat16, d_out)
        y_ptr = dY.data_ptr()
    if T == 0 and d_bias is None:       # (no address, so no output that the library could see)
        return dY
    need = 0 if d_bias is None else linear_backward_act_ws_bytes(T, d)
    ws_ptr, ws_n, ws = _workspace(ws, need, d_out)
    _call("logra_linear_backward_act", dev, d_out.data_ptr(), _TYPES[d_out.dtype], ldd, p_ptr, ldp,
          a, T, d, y_ptr, ldy, b_ptr, ws_ptr, ws_n, _stream(d_out))
    return dY


def linear_backward_input(dY, W, residual=None, out=None, ws=None):
    """out = dY W + residual (bf16 [T, k]), the gradient of linear's X; returns out.
    residual: bf16 [T, k], a gradient that reaches X by another way (out itself:
    added in place).  ws: scratch of linear_ws_bytes(T, d, k) bytes."""
    _need(dY, "dY", _BF16, ndim=2)
    dev = dY.get_device()
    T, d, ldy = _matrix(dY, "dY")
    _need(W, "W", _BF16, dev, ndim=2)
    d2, k, ldw = _matrix(W, "W")
    if d2 != d:
        raise ValueError(f"dY has {d} columns but W has {d2} rows")
    r_ptr, ldr = _given(residual, "residual", _BF16, dev, T, k)
    if out is None:
        out, ldo = _rows_out(T, k, torch.bfloat16, dY)
        o_ptr = out.data_ptr()
    else:
        o_ptr, ldo = _given(out, "out", _BF16, dev, T, k)
    ws_ptr, ws_n, ws = _workspace(ws, linear_ws_bytes(T, d, k), dY)
    _call("logra_linear_backward_input", dev, dY.data_ptr(), ldy, W.data_ptr(), ldw, T, d, k,
          r_ptr, ldr, o_ptr, ldo, ws_ptr, ws_n, _stream(dY))
    return out


def linear_backward_weight(dY, X, dW=None, accumulate=False, ws=None):
    """dW = dY^T X (or dW += with accumulate, fp32 only), the full gradient of a
    weight that is not sketched; returns dW ([d, k] bf16 or fp32; a new one is
    fp32).  ws: scratch of linear_ws_bytes(T, d, k) bytes."""
    _need(dY, "dY", _BF16, ndim=2)
    dev = dY.get_device()
    T, d, ldy = _matrix(dY, "dY")
    _need(X, "X", _BF16, dev, ndim=2)
    T2, k, ldx = _matrix(X, "X")
    if T2 != T:
        raise ValueError(f"dY has {T} rows but X has {T2}")
    if dW is None:
        if accumulate:
            raise ValueError("accumulate needs dW")
        dW, ldw = _rows_out(d, k, torch.float32, dY)
        w_ptr = dW.data_ptr()
    else:
        w_ptr, ldw = _given(dW, "dW", _F32 if accumulate else _EITHER, dev, d, k)
    ws_ptr, ws_n, ws = _workspace(ws, linear_ws_bytes(T, d, k), dY)
    _call("logra_linear_backward_weight", dev, dY.data_ptr(), ldy, X.data_ptr(), ldx, T, d, k,
          1 if accumulate else 0, w_ptr, _TYPES[dW.dtype], ldw, ws_ptr, ws_n, _stream(dY))
    return dW
