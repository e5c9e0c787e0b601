"""The boundary of include/logra_policy.h on the CPU: exported names, workspace
queries, and the refusals of every entry point (status codes before any HIP
call, so no device is needed) and of the Python binding."""
import ctypes
import subprocess

import pytest
import torch

import rank_gradient_sketching_amd as lg
from rank_gradient_sketching_amd import _lib, policy

OK, EINVAL, EWS = _lib.OK, _lib.EINVAL, _lib.EWORKSPACE
# 256-byte-aligned stand-in addresses far apart; never dereferenced
Z, T, A, B, C, D, E, W = (0x10000000000 * i for i in range(1, 9))
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def test_exports_every_declared_symbol(L):
    declared = _lib.header_symbols(_lib.POLICY_HEADER_PATH)
    assert len(declared) == 9
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = {line.split()[-1] for line in out.splitlines() if line.strip()}
    for name in declared:
        assert name in exported and name in _lib.SIGNATURES, name


def test_struct_layout(L):
    # seven pointers, a 64-bit count, a float and two 32-bit types
    assert ctypes.sizeof(_lib.AdamWItem) == 7 * 8 + 8 + 3 * 4 + 4


# ------------------------------------------------------------------ log probabilities
def _lp(L, **kw):
    a = dict(z=Z, dtype=0, n=64, V=10000, ld=10000, target=T, tau=1.0, n_top=4, logp=A, H=B, lse=C,
             idx=D, top=E, ws=W, ws_bytes=1 << 30, s=None)
    a.update(kw)
    return L.logra_token_logprob(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(z=None), EINVAL), (dict(z=Z + 8), EINVAL), (dict(dtype=2), EINVAL),
    (dict(dtype=-1), EINVAL), (dict(n=-1), EINVAL), (dict(n=1 << 31), EINVAL),
    (dict(V=0), EINVAL), (dict(V=1 << 31, ld=1 << 31), EINVAL), (dict(ld=9992), EINVAL),
    (dict(ld=10004), EINVAL), (dict(dtype=1, ld=10002), EINVAL), (dict(target=None), EINVAL),
    (dict(target=T + 4), EINVAL), (dict(tau=0.0), EINVAL), (dict(tau=NAN), EINVAL),
    (dict(tau=INF), EINVAL), (dict(tau=-1.0), EINVAL), (dict(n_top=-1), EINVAL),
    (dict(tau=1e-39), EINVAL),                      # log2(e) / tau past fp32
    (dict(n_top=65), EINVAL), (dict(logp=A + 2), EINVAL), (dict(H=B + 1), EINVAL),
    (dict(lse=C + 2), EINVAL), (dict(idx=None), EINVAL), (dict(top=None), EINVAL),
    (dict(idx=D + 2), EINVAL), (dict(ws=None), EWS), (dict(ws_bytes=64), EWS),
    (dict(ws=W + 16), EWS),
    # outputs that overlap each other, the logits or the workspace
    (dict(H=A), EINVAL), (dict(lse=A + 4), EINVAL), (dict(logp=Z), EINVAL),
    (dict(top=D), EINVAL), (dict(top=W), EINVAL), (dict(logp=T), EINVAL),
    # strides whose last row lies past the address space
    (dict(n=1 << 30, ld=1 << 39, dtype=1, n_top=0), EINVAL),
    (dict(n=(1 << 24) + 1, ld=1 << 39, n_top=0), EINVAL),
])
def test_logprob_rejects(L, kw, status):
    assert _lp(L, **kw) == status


def test_logprob_empty_and_sizes(L):
    assert _lp(L, n=0, z=None, target=None, logp=None, ws=None, ws_bytes=0) == OK
    assert _lp(L, n=0, tau=0.0) == EINVAL            # scalars are still checked
    assert L.logra_token_logprob_ws_bytes(4096, 152064, 0) == 0     # rows fill the chip
    few = L.logra_token_logprob_ws_bytes(4, 152064, 0)
    assert 0 < few < L.logra_token_logprob_ws_bytes(4, 152064, 8)
    assert L.logra_token_logprob_ws_bytes(4, 0, 0) == 0
    assert L.logra_token_logprob_ws_bytes(4, 10, 65) == 0


def _grad(L, **kw):
    a = dict(z=Z, dtype=0, n=64, V=1000, ld=1000, target=T, tau=1.0, lse=A, H=B, dl=C, dh=D,
             ds=E, dz=W, ldz=1000, s=None)
    a.update(kw)
    return L.logra_token_logprob_backward(*a.values())


@pytest.mark.parametrize("kw", [
    dict(z=None), dict(dz=None), dict(lse=None), dict(z=Z + 2), dict(dz=W + 2), dict(ldz=999),
    dict(ldz=1004), dict(dl=None, dh=None, ds=None), dict(target=None), dict(H=None),
    dict(dtype=3), dict(n=-1), dict(V=0), dict(tau=0.0), dict(tau=1e-39), dict(lse=A + 2), dict(dl=C + 1),
    dict(target=T + 4),
    # dz over the logits with another stride, or partly, or over a row vector
    dict(dz=Z, ldz=1008), dict(dz=Z + 16), dict(lse=W), dict(dl=W + 4), dict(target=W),
    # strides whose last row lies past the address space
    dict(n=(1 << 24) + 1, ld=1 << 39), dict(n=(1 << 24) + 1, ldz=1 << 39),
    dict(n=(1 << 24) + 1, ldz=1 << 39, ld=1 << 39, dz=Z),
])
def test_logprob_grad_rejects(L, kw):
    assert _grad(L, **kw) == EINVAL


def test_logprob_grad_empty(L):
    assert _grad(L, n=0, z=None, dz=None, lse=None) == OK
    assert _grad(L, n=0, ldz=999) == EINVAL


# ------------------------------------------------------------------ AdamW
def _table(L, n=1, items=1, table=True, short=0, **kw):
    arr = (_lib.AdamWItem * max(1, n))()
    for q in arr:
        q.p, q.g, q.m, q.v, q.n, q.p_type, q.g_type = A, B, C, D, 100, 1, 1
        for k, v in kw.items():
            setattr(q, k, v)
    size = max(L.logra_adamw_table_bytes(n), 256)
    buf = (ctypes.c_uint64 * (size // 8))()
    st = L.logra_adamw_table(n, arr if items else None, buf if table else None, size - short)
    return st, buf


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), EINVAL), (dict(items=0), EINVAL), (dict(table=False), EINVAL),
    (dict(short=256), EWS), (dict(p_type=2), EINVAL), (dict(g_type=-1), EINVAL),
    (dict(weight_decay=NAN), EINVAL), (dict(m_exp=E), EINVAL), (dict(v_exp=E), EINVAL),
    (dict(master=W), EINVAL), (dict(p=None), EINVAL), (dict(g=None), EINVAL),
    (dict(m=None), EINVAL), (dict(v=None), EINVAL), (dict(p=A + 2), EINVAL),
    (dict(g=B + 2), EINVAL), (dict(m=C + 1), EINVAL), (dict(v=D + 2), EINVAL),
    (dict(p_type=0, p=A + 1), EINVAL), (dict(p_type=0, master=W + 2), EINVAL),
    (dict(n=2, p_type=0, m_exp=E, v_exp=W, m=C + 1, v=D + 3), OK),
    (dict(p_type=0, p=A + 2, g=B + 4), OK),
    # sizes, also past what one launch can take
    (dict(**{"n": 1}, weight_decay=0.1), OK),
])
def test_adamw_table_rejects(L, kw, status):
    assert _table(L, **kw)[0] == status


def test_adamw_table_sizes(L):
    assert L.logra_adamw_table_bytes(-1) == 0 and L.logra_adamw_table_bytes(1 << 25) == 0
    assert L.logra_adamw_table_bytes(0) > 0
    assert L.logra_adamw_table_bytes(1000) >= 1000 * 84
    arr = (_lib.AdamWItem * 1)()
    q = arr[0]
    q.p, q.g, q.m, q.v, q.p_type, q.g_type = A, B, C, D, 1, 1
    buf = (ctypes.c_uint64 * 256)()
    for n, st in ((-1, EINVAL), (1 << 40, EINVAL), (1 << 37, EINVAL), ((1 << 36) - 4096, OK)):
        q.n = n
        assert L.logra_adamw_table(1, arr, buf, 2048) == st, n


def _step(L, table, dev=W, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, step=1, scale=None):
    return L.logra_adamw_step(table, dev, lr, b1, b2, eps, step, scale, None)


@pytest.mark.parametrize("kw", [
    dict(lr=-1.0), dict(lr=NAN), dict(lr=INF), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0),
    dict(b2=NAN), dict(b2=1.0 - 1e-12), dict(eps=-1e-8), dict(eps=INF), dict(step=0),
    dict(scale=E + 2), dict(dev=None), dict(dev=W + 4),
])
def test_adamw_step_rejects(L, kw):
    st, buf = _table(L)
    assert st == OK
    assert _step(L, ctypes.addressof(buf), **kw) == EINVAL


@pytest.mark.parametrize("kw", [dict(lr=1e39), dict(eps=1e39), dict(lr=-1e-300), dict(b1=-1e-300)])
def test_adamw_step_rejects_scalars_past_fp32(L, kw):
    """The kernels take fp32 scalars: an lr that is infinite there would turn entries
    without a step into NaN."""
    st, buf = _table(L)
    assert st == OK
    assert _step(L, ctypes.addressof(buf), **kw) == EINVAL


def test_adamw_step_needs_a_table_and_work(L):
    assert _step(L, None) == EINVAL
    buf = (ctypes.c_uint64 * 256)()
    assert _step(L, ctypes.addressof(buf)) == EINVAL          # not a table
    for kw in (dict(n=0, items=0), dict(n=3, p=None, g=None, m=None, v=None)):
        arr_n = kw.pop("n")
        arr = (_lib.AdamWItem * 3)()
        st = L.logra_adamw_table(arr_n, arr, buf, 2048)       # (no entries in any tensor)
        assert st == OK
        assert _step(L, ctypes.addressof(buf), dev=None) == OK
    # a refused table is no table
    arr = (_lib.AdamWItem * 1)()
    q = arr[0]
    q.p, q.g, q.m, q.v, q.p_type, q.g_type, q.n = A, B, C, D, 1, 1, 1 << 37
    assert L.logra_adamw_table(1, arr, buf, 2048) == EINVAL
    assert _step(L, ctypes.addressof(buf)) == EINVAL


@pytest.mark.parametrize("args,status", [
    ((2, A, B, 10, C, None), EINVAL), ((0, None, B, 10, C, None), EINVAL),
    ((0, A, None, 10, C, None), EINVAL), ((0, A, B, 10, None, None), EINVAL),
    ((0, A, B, 10, C + 1, None), EINVAL), ((0, A, B, -1, C, None), EINVAL),
    ((0, A, B, 10, A + 2, None), EINVAL), ((1, A, B, 10, B, None), EINVAL),
    ((1, None, None, 0, None, None), OK),
])
def test_state_values_rejects(L, args, status):
    assert L.logra_adamw_state_values(*args) == status


# ------------------------------------------------------------------ unmerged updates
def _ad(L, **kw):
    a = dict(X=Z, ldx=256, Y=T, ldy=512, out=A, ldo=512, T=100, d=512, k=256, r=16, n=4,
             adapter=B, U=C, u_type=1, seeds=D, A=None, lda=0, scale=E, ws=W, ws_bytes=1 << 30,
             s=None)
    a.update(kw)
    return L.logra_adapter_apply(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), EINVAL), (dict(Y=None), EINVAL), (dict(out=None), EINVAL),
    (dict(adapter=None), EINVAL), (dict(U=None), EINVAL), (dict(scale=None), EINVAL),
    (dict(seeds=None), EINVAL), (dict(A=Z, lda=256), EINVAL), (dict(seeds=None, A=D), EINVAL),
    (dict(seeds=None, A=D + 1, lda=256), EINVAL), (dict(seeds=None, A=D, lda=255), EINVAL),
    (dict(T=-1), EINVAL), (dict(T=1 << 31), EINVAL), (dict(d=0), EINVAL), (dict(k=0), EINVAL),
    (dict(r=0), EINVAL), (dict(r=257), EINVAL), (dict(n=0), EINVAL), (dict(n=1 << 31), EINVAL),
    (dict(u_type=2), EINVAL), (dict(ldx=255), EINVAL), (dict(ldx=260), EINVAL),
    (dict(ldy=504), EINVAL), (dict(ldo=508), EINVAL), (dict(X=Z + 2), EINVAL),
    (dict(Y=T + 8), EINVAL), (dict(out=A + 8), EINVAL), (dict(adapter=B + 2), EINVAL),
    (dict(U=C + 2), EINVAL), (dict(u_type=0, U=C + 1), EINVAL), (dict(seeds=D + 4), EINVAL),
    (dict(scale=E + 1), EINVAL), (dict(ws=None), EWS), (dict(ws_bytes=100), EWS),
    (dict(ws=W + 64), EWS),
    # out over Y with another stride or partly, over X, U, the ids, the scratch
    (dict(out=T, ldo=520), EINVAL), (dict(out=T + 16), EINVAL), (dict(out=Z), EINVAL),
    (dict(out=C + 16), EINVAL), (dict(adapter=A), EINVAL), (dict(ws=A), EINVAL),
    (dict(ws=Z), EINVAL), (dict(ws=T), EINVAL), (dict(scale=W + 64), EINVAL),
    # sizes and strides that pass the address space
    (dict(T=(1 << 24) + 1, ldx=1 << 39, d=8, ldy=8, ldo=8, ws_bytes=1 << 38), EINVAL),
    (dict(T=(1 << 24) + 1, ldy=1 << 39, ldo=1 << 39, out=T, d=8, ws_bytes=1 << 38), EINVAL),
    (dict(n=1 << 30, d=1 << 26, ldy=1 << 26, ldo=1 << 26), EINVAL),
    (dict(seeds=None, A=D, lda=1 << 39, n=1 << 21), EINVAL),
])
def test_adapter_rejects(L, kw, status):
    assert _ad(L, **kw) == status


def test_adapter_empty_and_sizes(L):
    assert _ad(L, T=0, X=None, Y=None, out=None, ws=None, ws_bytes=0) == OK
    assert _ad(L, T=0, r=0) == EINVAL
    assert L.logra_adapter_ws_bytes(0, 8, 8, 8) == 0
    assert L.logra_adapter_ws_bytes(8, 8, 8, 257) == 0
    assert L.logra_adapter_ws_bytes(8192, 4096, 4096, 64) >= 8192 * 64 * 4
    # flat grids past their limit are refused
    assert L.logra_adapter_ws_bytes((1 << 31) - 1, 4096, 64, 1) == 0
    assert _ad(L, T=(1 << 31) - 1, d=4096, ldy=4096, ldo=4096, out=T) == EINVAL
    # ... also those of few rows and a very wide layer
    assert L.logra_adapter_ws_bytes(1, 1 << 30, 64, 1) == 0
    assert L.logra_adapter_ws_bytes(1, 1 << 28, 64, 1) > 0
    assert L.logra_adapter_ws_bytes(8192, 1 << 25, 64, 1) > 0


# ------------------------------------------------------------------ binding
def test_binding_refuses_cpu_tensors():
    z = torch.zeros(4, 16, dtype=torch.bfloat16)
    f = torch.zeros(4)
    with pytest.raises(ValueError, match="GPU"):
        lg.token_logprob(z)
    with pytest.raises(ValueError, match="GPU"):
        lg.token_logprob_backward(z, None, f, d_lse=f)
    with pytest.raises(ValueError, match="GPU"):
        lg.adapter_apply(z, z, f, z, f)
    with pytest.raises(ValueError, match="GPU"):
        lg.adamw_bind([f], [f], [f], [f])
    with pytest.raises(ValueError, match="GPU"):
        lg.adamw_state_values(z, f, "m")
    with pytest.raises(ValueError, match="which"):
        lg.adamw_state_values(z, f, "w")
    with pytest.raises(ValueError, match="empty"):
        lg.adamw_bind([], [], [], [])
    with pytest.raises(TypeError, match="adamw_bind"):
        lg.adamw_step([f], 1e-3, 1)


@pytest.mark.parametrize("spans,ok", [
    ([(0, 10, True, ("a", 0)), (10, 20, True, ("b", 0))], True),
    ([(0, 10, False, ("a", 0)), (0, 10, False, ("b", 0))], True),       # shared inputs
    ([(0, 10, True, ("a", 0)), (0, 10, False, ("b", 0))], False),
    ([(0, 10, False, ("a", 0)), (4, 6, True, ("b", 0))], False),
    ([(0, 100, False, ("a", 0)), (10, 20, False, ("b", 0)), (90, 95, True, ("c", 0))], False),
    ([(0, 100, True, ("a", 0)), (10, 20, False, ("b", 0))], False),
    ([(0, 0, True, ("a", 0)), (0, 10, True, ("b", 0))], True),          # empty tensors
])
def test_overlap_check(spans, ok):
    if ok:
        policy._check_apart(list(spans))
    else:
        with pytest.raises(ValueError, match="overlaps"):
            policy._check_apart(list(spans))
