"""Argument checks of the operators around the block through the C ABI, on the
CPU: every call below fails validation before any HIP call."""
import ctypes

import pytest

import mixed_gemm_amd as mg

FAKE = 1 << 20
ARG, SHAPE, DTYPE, ALIGN, UNSUPPORTED = -1, -2, -3, -4, -5


def _norm(**over):
    n = mg.mg_norm(FAKE, FAKE, 0, 0, 1e-6)
    for k, v in over.items():
        setattr(n, k, v)
    return n


def _mod(**over):
    m = mg.mg_mod(FAKE, FAKE, FAKE, None, 8, 64, 1, 0)
    for k, v in over.items():
        setattr(m, k, v)
    return m


def _norm_mod(norm=None, mod=None, X=FAKE, dtype=0, ldx=64, M=8, K=64, H=FAKE, h_dtype=1, ldh=64):
    n, m = norm or _norm(), mod or _mod()
    return mg.lib().mg_norm_mod(ctypes.byref(n), ctypes.byref(m), X, dtype, ldx, M, K, H, h_dtype, ldh, None)


@pytest.mark.parametrize("kw,code", [
    (dict(norm=_norm(kind=2)), ARG),
    (dict(norm=_norm(eps=-1.0)), ARG),
    (dict(norm=_norm(eps=float("nan"))), ARG),
    (dict(norm=_norm(dtype=5)), DTYPE),
    (dict(norm=_norm(weight=FAKE + 1)), ALIGN),
    (dict(norm=_norm(bias=FAKE + 2)), ALIGN),
    (dict(mod=_mod(dtype=2)), DTYPE),
    (dict(mod=_mod(rows=0)), SHAPE),
    (dict(mod=_mod(group=0)), SHAPE),
    (dict(mod=_mod(group=7)), SHAPE),           # 8 rows in groups of 7 need 2 modulation rows
    (dict(mod=_mod(rows=2, ld=63)), SHAPE),
    (dict(mod=_mod(scale=FAKE + 2)), ALIGN),
    (dict(mod=_mod(index=FAKE + 1)), ALIGN),
    (dict(X=None), ARG),
    (dict(X=FAKE + 2), ALIGN),
    (dict(H=None), ARG),
    (dict(H=FAKE + 1), ALIGN),
    (dict(dtype=2), DTYPE),
    (dict(h_dtype=-1), DTYPE),
    (dict(ldx=63), SHAPE),
    (dict(ldh=63), SHAPE),
    (dict(M=-1), SHAPE),
    (dict(M=1 << 31, mod=_mod(group=1 << 40)), UNSUPPORTED),
    (dict(K=0), SHAPE),
    (dict(K=65537, ldx=70000, ldh=70000), UNSUPPORTED),
])
def test_norm_mod_refuses(kw, code):
    assert _norm_mod(**kw) == code
    assert mg.lib().mg_last_error()


def test_zero_rows_are_accepted_without_pointers():
    assert _norm_mod(M=0, X=None, H=None) == 0
    assert mg.lib().mg_norm_mod(None, None, None, 0, 64, 0, 64, None, 0, 64, None) == ARG     # but not without a norm


def _res(**over):
    n = _norm()
    a = mg.mg_residual(FAKE, FAKE, FAKE, FAKE, 64, 64, 64, 64, 0, 1, 1, 0, None, None, ctypes.pointer(n), None)
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(reserved=1), ARG),
    (dict(X=None), ARG),
    (dict(Y=None), ARG),
    (dict(O=None), ARG),
    (dict(H=None), ARG),
    (dict(Y=FAKE + 1), ALIGN),
    (dict(O=FAKE + 2), ALIGN),
    (dict(dtype=3), DTYPE),
    (dict(y_dtype=3), DTYPE),
    (dict(h_dtype=3), DTYPE),
    (dict(ldo=60), SHAPE),
    (dict(ldy=60), SHAPE),
    (dict(norm=None), ARG),                     # H without a norm
    (dict(norm=None, H=None, mod=ctypes.pointer(_mod())), ARG),
    (dict(gate=ctypes.pointer(_mod(gate=FAKE + 2))), ALIGN),
    (dict(post=ctypes.pointer(_norm(kind=7))), ARG),
    (dict(mod=ctypes.pointer(_mod(group=1))), SHAPE),
])
def test_residual_refuses(kw, code):
    a = _res(**kw)
    assert mg.lib().mg_residual_norm(ctypes.byref(a), 8, 64, None) == code
    assert mg.lib().mg_last_error()


def test_residual_refuses_null():
    assert mg.lib().mg_residual_norm(None, 8, 64, None) == ARG


def _plan(K=64, N=64, k=4):
    return mg.mg_plan(mg.make_desc(K, N, k, 0.5), FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0, FAKE)


def _ep(**over):
    e = mg.mg_epilogue(FAKE, FAKE, None, 64, 0, 0, 0, 0)
    for k, v in over.items():
        setattr(e, k, v)
    return e


def _gemm(ep=None, M=8, Y=FAKE, y_dtype=1, act=True, plan=None):
    p, a, e = plan or _plan(), mg.mg_act(FAKE, FAKE, FAKE), ep or _ep()
    return [f for f in (
        mg.lib().mg_dual_gemm_ep(ctypes.byref(p), ctypes.byref(a) if act else None, M, ctypes.byref(e), Y, y_dtype, None),
        mg.lib().mg_forward_ep(ctypes.byref(p), FAKE, 1, M, ctypes.byref(a) if act else None, ctypes.byref(e), Y,
                               y_dtype, None))]


@pytest.mark.parametrize("kw,code", [
    (dict(ep=_ep(reserved=1)), ARG),
    (dict(ep=_ep(act=3)), ARG),
    (dict(ep=_ep(bias=FAKE + 4)), ALIGN),
    (dict(ep=_ep(bias_dtype=9)), DTYPE),
    (dict(ep=_ep(residual=FAKE + 8)), ALIGN),
    (dict(ep=_ep(residual_dtype=9)), DTYPE),
    (dict(ep=_ep(ldr=56)), SHAPE),
    (dict(ep=_ep(ldr=68)), ALIGN),
    (dict(ep=_ep(mod=ctypes.pointer(_mod(gate=FAKE + 4)))), ALIGN),
    (dict(ep=_ep(mod=ctypes.pointer(_mod(rows=2, ld=68)))), ALIGN),
    (dict(ep=_ep(mod=ctypes.pointer(_mod(group=3)))), SHAPE),
    (dict(M=-1), SHAPE),
    (dict(Y=None), ARG),
    (dict(Y=FAKE + 2), ALIGN),
    (dict(y_dtype=4), DTYPE),
    (dict(act=False), ARG),
    (dict(plan=_plan(K=48)), SHAPE),
    (dict(M=1 << 27), UNSUPPORTED),
])
def test_gemm_epilogue_refuses(kw, code):
    assert _gemm(**kw) == [code, code]
    assert mg.lib().mg_last_error()


def test_forward_ep_refuses_its_own_input():
    p, a = _plan(), mg.mg_act(FAKE, FAKE, FAKE)
    for X, dt, code in ((None, 1, ARG), (FAKE + 2, 1, ALIGN), (FAKE, 8, DTYPE)):
        assert mg.lib().mg_forward_ep(ctypes.byref(p), X, dt, 8, ctypes.byref(a), None, FAKE, 1, None) == code


def test_norm_quantize_refuses():
    p, a, n, m = _plan(), mg.mg_act(FAKE, FAKE, FAKE), _norm(), _mod()

    def call(p=p, n=n, m=m, X=FAKE, dtype=1, ldx=64, M=8, a=a):
        r = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
        return mg.lib().mg_norm_quantize_act(r(p), r(n), r(m), X, dtype, ldx, M, r(a), None)

    assert call(p=None) == ARG and call(n=None) == ARG and call(a=None) == ARG and call(X=None) == ARG
    assert call(X=FAKE + 1) == ALIGN and call(dtype=2) == DTYPE and call(ldx=32) == SHAPE and call(M=-1) == SHAPE
    assert call(m=_mod(group=1)) == SHAPE and call(a=mg.mg_act(FAKE + 4, FAKE, FAKE)) == ALIGN
    assert call(M=0, X=None, a=None) == 0
