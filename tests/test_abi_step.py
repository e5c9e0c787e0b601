"""The boundary of include/logra_step.h on the CPU: exported names, workspace
queries, and the refusals of every entry point (status codes before any HIP
call, so no device is needed) and of the Python binding."""
import ctypes
import subprocess

import pytest
import torch

import rank_gradient_sketching_amd as lg
from rank_gradient_sketching_amd import _lib

OK, EINVAL, EWS = _lib.OK, _lib.EINVAL, _lib.EWORKSPACE
# 256-byte-aligned stand-in addresses far apart; never dereferenced
A, B, C, D, E, F, G, H, I, W = (0x10000000000 * i for i in range(1, 11))
NAN, INF = float("nan"), float("inf")
INT64_MIN = -(1 << 63)
FAR = dict(T=(1 << 24) + 1)      # with strides of 2^39 elements: past the address space


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def test_exports_every_declared_symbol(L):
    declared = _lib.header_symbols(_lib.STEP_HEADER_PATH)
    assert len(declared) == 13
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    for name in declared:
        assert name in exported and name in _lib.SIGNATURES, name


def test_struct_layout(L):
    # two pointers, a 64-bit count and two 32-bit types
    assert ctypes.sizeof(_lib.GradItem) == 2 * 8 + 8 + 2 * 4


# ------------------------------------------------------------------ sampling
def _sample(L, **kw):
    a = dict(z=A, dtype=0, n=8, V=10000, ld=10000, u=B, tau=1.0, top_k=50, top_p=0.9, min_p=0.0,
             tau_rows=None, top_k_rows=None, top_p_rows=None, min_p_rows=None, token=C, logp=D,
             logq=E, kept=F, ws=W, ws_bytes=1 << 30, s=None)
    a.update(kw)
    return L.logra_sample_tokens(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(z=None), EINVAL), (dict(z=A + 8), EINVAL), (dict(dtype=2), EINVAL),
    (dict(dtype=-1), EINVAL), (dict(n=-1), EINVAL), (dict(n=1 << 31), EINVAL), (dict(V=0), EINVAL),
    (dict(V=1 << 31, ld=1 << 31), EINVAL), (dict(ld=9992), EINVAL), (dict(ld=10004), EINVAL),
    (dict(dtype=1, ld=10002), EINVAL), (dict(u=None), EINVAL), (dict(u=B + 2), EINVAL),
    (dict(tau=0.0), EINVAL), (dict(tau=-1.0), EINVAL), (dict(tau=NAN), EINVAL),
    (dict(tau=INF), EINVAL), (dict(top_k=-1), EINVAL), (dict(top_p=0.0), EINVAL),
    (dict(top_p=1.01), EINVAL), (dict(top_p=NAN), EINVAL), (dict(min_p=-0.1), EINVAL),
    (dict(min_p=1.5), EINVAL), (dict(min_p=NAN), EINVAL),
    (dict(token=None), EINVAL), (dict(token=C + 4), EINVAL), (dict(logp=D + 2), EINVAL),
    (dict(logq=E + 1), EINVAL), (dict(kept=F + 2), EINVAL), (dict(tau_rows=G + 2), EINVAL),
    (dict(top_k_rows=G + 2), EINVAL), (dict(top_p_rows=G + 1), EINVAL),
    (dict(min_p_rows=G + 3), EINVAL), (dict(ws=None), EWS), (dict(ws_bytes=64), EWS),
    (dict(ws=W + 16), EWS),
    # outputs that overlap each other, the logits, the settings or the workspace
    (dict(logp=C), EINVAL), (dict(kept=D + 28), EINVAL), (dict(logq=B), EINVAL),
    (dict(token=A), EINVAL), (dict(tau_rows=D), EINVAL), (dict(min_p_rows=W), EINVAL),
    (dict(kept=W + 256), EINVAL), (dict(ws=A), EINVAL),
    # strides whose last row lies past the address space
    (dict(n=(1 << 24) + 1, ld=1 << 39), EINVAL), (dict(n=1 << 30, ld=1 << 39, dtype=1), EINVAL),
])
def test_sample_rejects(L, kw, status):
    assert _sample(L, **kw) == status


def test_sample_empty_and_sizes(L):
    none = dict(n=0, z=None, u=None, token=None, logp=None, logq=None, kept=None, ws=None,
                ws_bytes=0)
    assert _sample(L, **none) == OK
    assert _sample(L, **{**none, "tau": 0.0}) == EINVAL       # scalars are still checked
    # ... but not those that the rows give themselves
    assert _sample(L, **{**none, "tau": 0.0, "tau_rows": G, "top_k": -3, "top_k_rows": G,
                         "top_p": 7.0, "top_p_rows": G, "min_p": NAN, "min_p_rows": G}) == OK
    size = L.logra_sample_tokens_ws_bytes
    assert size(512, 152064) == 0                             # rows fill the chip
    assert 0 < size(1, 152064) < size(8, 152064) and size(8, 152064) % 256 == 0
    assert size(0, 152064) == 0 and size(8, 0) == 0 and size(-1, 10) == 0 and size(1 << 31, 8) == 0


# ------------------------------------------------------------------ gradient norm
def _table(L, n=1, items=1, table=True, short=0, **kw):
    arr = (_lib.GradItem * max(1, n))()
    for q in arr:
        q.g, q.n, q.g_type = A, 100, 1
        for k, v in kw.items():
            setattr(q, k, v)
    size = max(L.logra_grad_table_bytes(n), 256)
    buf = (ctypes.c_uint64 * (size // 8))()
    st = L.logra_grad_table(n, arr if items else None, buf if table else None, size - short)
    return st, buf


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), EINVAL), (dict(n=(1 << 20) + 1), EINVAL), (dict(items=0), EINVAL),
    (dict(table=False), EINVAL), (dict(short=256), EWS), (dict(g_type=2), EINVAL),
    (dict(g_type=-1), EINVAL), (dict(out=B, out_type=2), EINVAL), (dict(g=None), EINVAL),
    (dict(g=A + 2), EINVAL), (dict(g=A + 1, g_type=0), EINVAL), (dict(out=B + 2, out_type=1), EINVAL),
    (dict(out=B + 1, out_type=0), EINVAL), (dict(out=A, out_type=0), EINVAL),
    (dict(out=A, out_type=1), OK), (dict(out=B, out_type=0), OK), (dict(g=A + 2, g_type=0), OK),
    (dict(n=0, items=0), OK), (dict(n=3), OK),
])
def test_grad_table_rejects(L, kw, status):
    assert _table(L, **kw)[0] == status


def test_grad_table_sizes(L):
    assert L.logra_grad_table_bytes(-1) == 0 and L.logra_grad_table_bytes((1 << 20) + 1) == 0
    assert L.logra_grad_table_bytes(0) > 0 and L.logra_grad_table_bytes(1 << 20) > 0
    arr = (_lib.GradItem * 1)()
    q = arr[0]
    q.g, q.g_type = A, 1
    buf = (ctypes.c_uint64 * 64)()
    for n, st in ((-1, EINVAL), (1 << 40, EINVAL), (INT64_MIN, EINVAL), (0, OK), (1 << 38, OK),
                  ((1 << 40) - 1, OK)):
        q.n = n
        assert L.logra_grad_table(1, arr, buf, 512) == st, n
        ws = L.logra_grad_norm_ws_bytes(ctypes.addressof(buf))
        assert ws % 256 == 0 and (ws > 0 or st != OK)


def _norm(L, table, dev=W, kind=0, max_norm=1.0, grad_scale=None, norm=B, scale=C, norms=D, ws=E,
          ws_bytes=1 << 30):
    return L.logra_grad_norm(table, dev, kind, max_norm, grad_scale, norm, scale, norms, ws,
                             ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dev=None), EINVAL), (dict(dev=W + 4), EINVAL), (dict(kind=2), EINVAL),
    (dict(kind=-1), EINVAL), (dict(max_norm=-1.0), EINVAL), (dict(max_norm=NAN), EINVAL),
    (dict(norm=None, scale=None, norms=None), EINVAL), (dict(grad_scale=F + 2), EINVAL),
    (dict(norm=B + 1), EINVAL), (dict(scale=C + 2), EINVAL), (dict(norms=D + 2), EINVAL),
    (dict(ws=None), EWS), (dict(ws_bytes=8), EWS), (dict(ws=E + 8), EWS),
    (dict(scale=B), EINVAL), (dict(norms=B), EINVAL), (dict(norm=W), EINVAL),
    (dict(grad_scale=C), EINVAL), (dict(norm=E), EINVAL), (dict(ws=W), EINVAL),
])
def test_grad_norm_rejects(L, kw, status):
    st, buf = _table(L)
    assert st == OK
    assert _norm(L, ctypes.addressof(buf), **kw) == status


def test_grad_norm_and_clip_need_a_table(L):
    buf = (ctypes.c_uint64 * 256)()
    at = ctypes.addressof(buf)
    assert _norm(L, None) == EINVAL and _norm(L, at) == EINVAL
    assert L.logra_grad_norm_ws_bytes(at) == 0 and L.logra_grad_norm_ws_bytes(None) == 0
    assert L.logra_grad_clip(at, W, C, None) == EINVAL
    assert L.logra_grad_clip(None, W, C, None) == EINVAL
    st, buf = _table(L)
    at = ctypes.addressof(buf)
    assert st == OK
    for dev, scale in ((W, None), (W, C + 2), (None, C), (W + 4, C)):
        assert L.logra_grad_clip(at, dev, scale, None) == EINVAL
    assert _norm(L, at + 4) == EINVAL
    # a refused table is no table
    arr = (_lib.GradItem * 1)()
    arr[0].g, arr[0].n, arr[0].g_type = A, 100, 9
    assert L.logra_grad_table(1, arr, (ctypes.c_uint64 * 64)(), 512) == EINVAL
    # no tensors, or none with entries: nothing to clip, nothing to look at on the device
    st, buf = _table(L, n=2, g=None)
    assert st == EINVAL
    arr = (_lib.GradItem * 2)()
    buf = (ctypes.c_uint64 * 64)()
    assert L.logra_grad_table(2, arr, buf, 512) == OK
    assert L.logra_grad_clip(ctypes.addressof(buf), None, C, None) == OK
    assert L.logra_grad_table(0, None, buf, 512) == OK
    assert _norm(L, ctypes.addressof(buf), dev=None, norm=None, scale=None) == OK


# ------------------------------------------------------------------ layer product
def _linear(L, **kw):
    a = dict(X=A, ldx=256, W=B, ldw=256, T=8, d=512, k=256, bias=C, bias_type=0, act=2, residual=D,
             ldr=512, out=E, out_type=0, ldo=512, pre=F, ldp=512, ws=W, ws_bytes=1 << 30, s=None)
    a.update(kw)
    return L.logra_linear(*a.values())


LINEAR_BAD = [
    (dict(X=None), EINVAL), (dict(X=A + 8), EINVAL), (dict(W=None), EINVAL),
    (dict(W=B + 2), EINVAL), (dict(T=-1), EINVAL), (dict(T=1 << 31), EINVAL), (dict(d=0), EINVAL),
    (dict(d=1 << 31, ldo=1 << 31, ldr=1 << 31, ldp=1 << 31), EINVAL), (dict(k=0), EINVAL),
    (dict(k=-5), EINVAL), (dict(ldx=248), EINVAL), (dict(ldx=260), EINVAL), (dict(ldw=255), EINVAL),
    (dict(ldw=1 << 40), EINVAL), (dict(bias=C + 1), EINVAL), (dict(bias=C + 2, bias_type=1), EINVAL),
    (dict(bias_type=2), EINVAL), (dict(act=5), EINVAL), (dict(act=-1), EINVAL),
    (dict(residual=D + 8), EINVAL), (dict(ldr=504), EINVAL), (dict(ldr=516), EINVAL),
    (dict(out=None), EINVAL), (dict(out=E + 8), EINVAL), (dict(out_type=2), EINVAL),
    (dict(ldo=511), EINVAL), (dict(out_type=1, ldo=514), EINVAL), (dict(pre=F + 4), EINVAL),
    (dict(ldp=508), EINVAL),
    # out over the residual with another stride, partly, or as fp32; over the inputs; pre too
    (dict(out=D, ldo=520), EINVAL), (dict(out=D + 16), EINVAL), (dict(out=D, out_type=1), EINVAL),
    (dict(out=A), EINVAL), (dict(out=B), EINVAL), (dict(out=C), EINVAL), (dict(pre=D), EINVAL),
    (dict(pre=E), EINVAL), (dict(pre=A), EINVAL), (dict(pre=C - 16), EINVAL),
    # strides whose last row lies past the address space
    (dict(**FAR, ldx=1 << 39), EINVAL), (dict(**FAR, ldo=1 << 39, residual=None), EINVAL),
    (dict(d=(1 << 24) + 1, ldw=1 << 39, ldo=1 << 25, ldr=1 << 25, ldp=1 << 25), EINVAL),
    (dict(**FAR, ldr=1 << 39), EINVAL), (dict(**FAR, ldp=1 << 39), EINVAL),
    # more than one launch covers
    (dict(T=(1 << 31) - 1, d=1 << 20, k=8, ldx=8, ldw=8, ldo=1 << 20, residual=None, pre=None,
          out=1 << 61), EINVAL),
]


@pytest.mark.parametrize("kw,status", LINEAR_BAD)
def test_linear_rejects(L, kw, status):
    assert _linear(L, **kw) == status


def _split(L, form):
    """A T, d, k whose product is split, so that it needs the workspace."""
    T, d, k = {"forward": (64, 64, 1 << 20), "input": (64, 1 << 20, 64),
               "weight": (1 << 20, 64, 64)}[form]
    assert L.logra_linear_ws_bytes(T, d, k) > 0 and L.logra_linear_ws_bytes(T, d, k) % 256 == 0
    return T, d, k


def test_linear_workspace(L):
    T, d, k = _split(L, "forward")
    a = dict(T=T, d=d, k=k, ldx=k, ldw=k, residual=None, pre=None)
    for kw in (dict(ws=None), dict(ws_bytes=256), dict(ws=W + 16)):
        assert _linear(L, **a, **kw) == EWS
    for kw in (dict(ws=A), dict(ws=B), dict(ws=C), dict(ws=E)):
        assert _linear(L, **a, **kw) == EINVAL


def test_linear_empty_and_sizes(L):
    none = dict(T=0, X=None, W=None, out=None, bias=None, residual=None, pre=None, ws=None,
                ws_bytes=0)
    assert _linear(L, **none) == OK
    assert _linear(L, **{**none, "act": 7}) == EINVAL
    assert _linear(L, **{**none, "ldo": 100}) == EINVAL
    for bad in ((-1, 8, 8), (8, 0, 8), (8, 8, 0), (1 << 31, 8, 8), (8, 1 << 31, 8), (0, 8, 8)):
        assert L.logra_linear_ws_bytes(*bad) == 0
    assert L.logra_linear_ws_bytes(8192, 4096, 4096) >= 0
    assert L.logra_linear_backward_act_ws_bytes(-1, 8) == 0
    assert L.logra_linear_backward_act_ws_bytes(8, 0) == 0
    assert L.logra_linear_backward_act_ws_bytes(8192, 4096) % 256 == 0
    # few rows are added up by one launch, without scratch (which is then not looked at)
    assert L.logra_linear_backward_act_ws_bytes(1000, 512) == 0
    assert L.logra_linear_backward_act_ws_bytes(2000, 512) > 0


def _act(L, **kw):
    a = dict(d_out=A, d_out_type=0, ldd=512, pre=B, ldp=512, act=2, T=2000, d=512, dY=C, ldy=512,
             d_bias=D, ws=W, ws_bytes=1 << 30, s=None)
    a.update(kw)
    return L.logra_linear_backward_act(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(d_out=None), EINVAL), (dict(d_out=A + 8), EINVAL), (dict(d_out_type=2), EINVAL),
    (dict(d_out_type=1, ldd=514), EINVAL), (dict(ldd=504), EINVAL), (dict(pre=None), EINVAL),
    (dict(pre=B + 2), EINVAL), (dict(ldp=500), EINVAL), (dict(act=5), EINVAL),
    (dict(act=0), EINVAL),                            # pre without an activation
    (dict(T=-1), EINVAL), (dict(T=1 << 31), EINVAL), (dict(d=0), EINVAL),
    (dict(dY=C + 8), EINVAL), (dict(ldy=508), EINVAL), (dict(dY=None, d_bias=None), EINVAL),
    (dict(d_bias=D + 2), EINVAL), (dict(ws=None), EWS), (dict(ws_bytes=16), EWS),
    (dict(ws=W + 8), EWS),
    # dY over d_out or pre with another stride, partly, or over an fp32 d_out
    (dict(dY=A, ldy=520), EINVAL), (dict(dY=A + 16), EINVAL), (dict(dY=B, ldy=520), EINVAL),
    (dict(dY=A, d_out_type=1), EINVAL), (dict(d_bias=A), EINVAL), (dict(d_bias=B + 64), EINVAL),
    (dict(d_bias=C), EINVAL), (dict(d_bias=W), EINVAL), (dict(ws=C), EINVAL), (dict(ws=A), EINVAL),
    (dict(**FAR, ldd=1 << 39), EINVAL), (dict(**FAR, ldp=1 << 39), EINVAL),
    (dict(**FAR, ldy=1 << 39), EINVAL),
])
def test_backward_act_rejects(L, kw, status):
    assert _act(L, **kw) == status


def test_backward_act_empty(L):
    assert _act(L, T=0, d_out=None, pre=None, dY=None, d_bias=None) == EINVAL
    assert _act(L, T=0, d_out=None, pre=None, d_bias=None) == OK


def _input(L, **kw):
    a = dict(dY=A, ldy=512, W=B, ldw=256, T=8, d=512, k=256, residual=C, ldr=256, dX=D, ldx=256,
             ws=W, ws_bytes=1 << 30, s=None)
    a.update(kw)
    return L.logra_linear_backward_input(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dY=None), EINVAL), (dict(dY=A + 8), EINVAL), (dict(ldy=504), EINVAL),
    (dict(W=None), EINVAL), (dict(W=B + 4), EINVAL), (dict(ldw=250), EINVAL), (dict(T=-1), EINVAL),
    (dict(d=0), EINVAL), (dict(k=1 << 31), EINVAL), (dict(residual=C + 8), EINVAL),
    (dict(ldr=248), EINVAL), (dict(dX=None), EINVAL), (dict(dX=D + 2), EINVAL),
    (dict(ldx=255), EINVAL), (dict(dX=C, ldx=264), EINVAL), (dict(dX=C + 16), EINVAL),
    (dict(dX=A), EINVAL), (dict(dX=B), EINVAL), (dict(**FAR, ldy=1 << 39), EINVAL),
    (dict(**FAR, ldx=1 << 39), EINVAL), (dict(**FAR, ldr=1 << 39), EINVAL),
    (dict(T=0, dX=None, dY=None, W=None), OK), (dict(T=0, ldw=3), EINVAL),
])
def test_backward_input_rejects(L, kw, status):
    assert _input(L, **kw) == status


def _weight(L, **kw):
    a = dict(dY=A, ldy=512, X=B, ldx=256, T=8, d=512, k=256, flags=0, dW=C, dw_type=1, ldw=256,
             ws=W, ws_bytes=1 << 30, s=None)
    a.update(kw)
    return L.logra_linear_backward_weight(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dY=None), EINVAL), (dict(dY=A + 2), EINVAL), (dict(ldy=511), EINVAL),
    (dict(X=None), EINVAL), (dict(X=B + 8), EINVAL), (dict(ldx=252), EINVAL), (dict(T=-2), EINVAL),
    (dict(d=1 << 31), EINVAL), (dict(k=0), EINVAL), (dict(flags=2), EINVAL),
    (dict(flags=1, dw_type=0), EINVAL), (dict(dw_type=3), EINVAL), (dict(dW=None), EINVAL),
    (dict(dW=C + 8), EINVAL), (dict(ldw=254), EINVAL), (dict(dW=A), EINVAL), (dict(dW=B), EINVAL),
    (dict(**FAR, ldy=1 << 39), EINVAL), (dict(**FAR, ldx=1 << 39), EINVAL),
    (dict(d=(1 << 23) + 1, ldw=1 << 39, ldy=1 << 24), EINVAL),
    (dict(T=0, flags=1, dY=None, X=None), OK), (dict(T=0, flags=1, dW=None), EINVAL),
])
def test_backward_weight_rejects(L, kw, status):
    assert _weight(L, **kw) == status


def test_gradients_workspaces(L):
    T, d, k = _split(L, "input")
    a = dict(T=T, d=d, k=k, ldy=d, ldw=k, ldr=k, ldx=k)
    for kw in (dict(ws=None), dict(ws_bytes=256), dict(ws=W + 128)):
        assert _input(L, **a, **kw) == EWS
    for ws in (A, B, C, D):
        assert _input(L, **a, ws=ws) == EINVAL
    T, d, k = _split(L, "weight")
    a = dict(T=T, d=d, k=k, ldy=d, ldw=k, ldx=k)
    for kw in (dict(ws=None), dict(ws_bytes=256), dict(ws=W + 128)):
        assert _weight(L, **a, **kw) == EWS
    for ws in (A, B, C):
        assert _weight(L, **a, ws=ws) == EINVAL


# ------------------------------------------------------------------ binding
def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    f = torch.zeros(4)
    for call in (lambda: lg.sample_tokens(x, f), lambda: lg.grad_norm_bind([f]),
                 lambda: lg.linear(x, x), lambda: lg.linear_backward_act(x),
                 lambda: lg.linear_backward_input(x, x), lambda: lg.linear_backward_weight(x, x)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_binding_refuses_what_is_no_handle():
    f = torch.zeros(4)
    with pytest.raises(ValueError, match="empty"):
        lg.grad_norm_bind([])
    with pytest.raises(TypeError, match="grad_norm_bind"):
        lg.grad_norm([f])
    with pytest.raises(TypeError, match="grad_norm_bind"):
        lg.grad_clip(f, f)


def test_sizes_of_the_binding():
    assert lg.sample_tokens_ws_bytes(512, 152064) == 0 < lg.sample_tokens_ws_bytes(8, 152064)
    assert lg.linear_ws_bytes(64, 64, 1 << 20) > 0
    assert lg.linear_backward_act_ws_bytes(8192, 4096) > 0
