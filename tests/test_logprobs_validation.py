"""Argument checks of the log-probability and distillation entry points on the
CPU: the binding's (nothing reaches the library) and the library's (answered
before anything is enqueued)."""
import ctypes

import pytest
import torch

import linear_layers_b200 as tpl
from linear_layers_b200 import build as tpbuild

BF, F32, I64, I32 = torch.bfloat16, torch.float32, torch.int64, torch.int32
T, V, K, H = 6, 40, 5, 16


def t(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


def passes(fn, *a, **k):
    with pytest.raises(RuntimeError, match="no CPU path"):
        fn(*a, **k)


def rejected(fn, *a, **k):
    with pytest.raises((ValueError, TypeError)):
        fn(*a, **k)


X, Y, R = t(T, V), t(T, dtype=I64), t(T)


def test_logprobs_fwd_binding():
    f = tpl.vp_logprobs_fwd
    passes(f, X, Y, 4)
    passes(f, X.bfloat16(), None, 4, top_k=3)
    rejected(f, X.half(), Y, 4)
    rejected(f, X.t(), t(V, dtype=I64), 4)                       # not contiguous
    rejected(f, X, t(T, dtype=I32), 4)
    rejected(f, X, t(T + 1, dtype=I64), 4)
    rejected(f, X, None, 4, logprob=R)
    rejected(f, X, Y, 4, entropy=t(T, dtype=BF))
    rejected(f, X, Y, 4, top_k=3, top_idx=t(T, 3, dtype=I64))
    rejected(f, X, Y, 4, top_k=3, top_logprob=t(T, 4))
    rejected(f, X, Y, 4, top_idx=t(T, 3, dtype=I32))             # without top_k
    rejected(f, X, Y, 4, dev_status=t(1, dtype=I64))


def test_logprobs_bwd_binding():
    f = tpl.vp_logprobs_bwd
    passes(f, X, Y, R, R, R, R, 4)
    passes(f, X, Y, R, None, R, None, 4, dlogits=X)              # in place
    passes(f, X, None, R, R, None, R, 4)
    rejected(f, X, Y, R, R, None, None, 4)                       # nothing to differentiate
    rejected(f, X, None, R, R, R, None, 4)
    rejected(f, X, Y, R, None, None, R, 4)
    rejected(f, X, Y, R[:3], R, R, R, 4)
    rejected(f, X, Y, R, R, t(T, 1), R, 4)
    rejected(f, X, Y, R, R, R, R, 4, dlogits=t(T, V + 1))
    rejected(f, X, Y, R, R, R, R, 4, grad_dtype=torch.float16)


def test_distill_binding():
    f, ids, tl = tpl.vp_distill, t(T, K, dtype=I32), t(T, K)
    passes(f, X, ids, tl, 4)
    passes(f, X.bfloat16(), ids, tl, 4, weight=R, with_grad=False, renormalize=False)
    rejected(f, X, ids.long(), tl, 4)
    rejected(f, X, ids, tl.bfloat16(), 4)
    rejected(f, X, ids, t(T, K + 1), 4)
    rejected(f, X, ids[:3], tl, 4)
    rejected(f, X, ids, tl, 4, weight=t(T, 1))
    rejected(f, X, ids, tl, 4, loss_sum=t(2))
    rejected(f, X, ids, tl, 4, dlogits=t(T, V - 1))
    rejected(f, X, ids, tl, 4, grad_dtype=torch.float16)


def test_linear_logprobs_binding():
    h, E = t(T, H, dtype=BF), t(V, H, dtype=BF)
    f, g = tpl.tp_linear_logprobs_fwd, tpl.tp_linear_logprobs_dlogits
    passes(f, h, E, Y, 4)
    passes(f, h, E, None, 4)
    rejected(f, h.float(), E, Y, 4)
    rejected(f, h, t(V, H + 8, dtype=BF), Y, 4)
    rejected(f, h, E, None, 4, logprob=R)
    passes(g, h, E, Y, R, R, R, R, 4)
    passes(g, h, E, Y, R, None, R, None, 4)
    rejected(g, h, E, Y, R, None, R, R, 4)
    rejected(g, h, E, Y, R, R, None, None, 4)
    rejected(g, h, E, Y, R, R, R, R, 4, dlogits=t(T, V))         # must be bf16


@pytest.fixture(scope="module")
def L():
    tpbuild.build()
    return tpl.lib()


P = ctypes.c_void_p(1 << 20)                                     # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 4)
OK, NULL, SHAPE, ALIGN, DTYPE, UNSUPPORTED, WORKSPACE, DEVICE = 0, 1, 2, 3, 4, 5, 7, 8


def call(fn, names, defaults, **kw):
    a = dict(zip(names.split(), defaults))
    assert set(kw) <= set(a)
    a.update(kw)
    return fn(*a.values())


def test_logprobs_abi(L):
    f = lambda **k: call(L.vp_logprobs_fwd, "x dt y T v N scale k lp ent lse ti tl st stream",  # noqa: E731
                         (P, 1, P, 4, 300, 2, 1.0, 0, P, P, P, None, None, None, None), **k)
    assert f(x=None) == NULL and f(y=None) == NULL
    assert f(y=None, lp=None, ent=None, lse=None) == NULL        # nothing asked for
    assert f(k=3) == NULL and f(k=3, ti=P) == NULL
    assert f(dt=2) == DTYPE
    assert f(T=0) == f(v=0) == f(T=(1 << 30) + 1) == f(N=7) == f(N=0) == SHAPE
    assert f(k=-1, ti=P, tl=P) == f(k=301, ti=P, tl=P) == SHAPE
    assert f(k=129, ti=P, tl=P) == UNSUPPORTED
    for s in (0.0, -1.0, float("inf"), float("nan")):
        assert f(scale=s) == SHAPE
    assert f(x=ODD) == f(y=ODD) == f(lse=ctypes.c_void_p((1 << 20) + 2)) == ALIGN
    g = lambda **k: call(L.vp_logprobs_bwd, "x dt y lse ent g e T v N scale d gdt st stream",  # noqa: E731
                         (P, 1, P, P, P, P, P, 4, 300, 2, 1.0, ctypes.c_void_p(1 << 21), 0, None,
                          None), **k)
    assert g(x=None) == g(lse=None) == g(d=None) == g(y=None) == g(ent=None) == NULL
    assert g(g=None, e=None) == NULL
    assert g(gdt=5) == g(dt=-1) == DTYPE
    assert g(v=-1) == g(N=7) == g(scale=0.0) == SHAPE
    assert g(d=ODD) == ALIGN
    assert g(d=P) == UNSUPPORTED                                 # in place needs one type


def test_distill_abi(L):
    f = lambda **k: call(L.vp_distill,  # noqa: E731
                         "x dt ids t w T v K N re scale gs loss sum lse d gdt ws wsb st stream",
                         (P, 1, P, P, None, 4, 300, 8, 2, 1, 1.0, 1.0, P, P, None, None, 0, P, 320,
                          None, None), **k)
    assert f(x=None) == f(ids=None) == f(t=None) == f(loss=None) == NULL
    assert f(dt=3) == f(d=ctypes.c_void_p(1 << 21), gdt=9) == DTYPE
    assert f(K=0) == f(T=0) == f(v=0) == f(N=7) == f(scale=float("nan")) == SHAPE
    assert f(K=257) == UNSUPPORTED and f(d=P) == UNSUPPORTED
    D = ctypes.c_void_p(1 << 21)
    assert f(v=337922, d=D) == UNSUPPORTED and f(v=337922, dt=0, d=D) == UNSUPPORTED
    assert f(x=ODD) == f(d=ODD) == f(ws=ODD) == ALIGN
    assert tpl.tp_workspace_bytes(tpl.OP_DISTILL, 4, 8, 300, 2) >= 4 * (16 + 8 * 8) == 320
    assert f(ws=None) == f(wsb=319) == WORKSPACE


def test_linear_logprobs_abi(L):
    wsb = tpl.tp_workspace_bytes(tpl.OP_LINEAR_LOGPROBS, 4, 64, 300, 2)
    assert wsb >= 3 * 3 * 4 * 4 + 4 * 4
    f = lambda **k: call(L.tp_linear_logprobs_fwd, "H E y T h v N scale lp ent lse ws wsb st stream",  # noqa: E731
                         (P, P, P, 4, 64, 300, 2, 1.0, P, P, P, P, wsb, None, None), **k)
    assert f(H=None) == f(E=None) == f(y=None) == NULL
    assert f(y=None, lp=None, ent=None, lse=None) == NULL
    assert f(T=0) == f(N=7) == f(scale=0.0) == SHAPE
    assert f(h=60) == f(H=ODD) == ALIGN
    assert f(ws=None) == f(wsb=wsb - 1) == WORKSPACE
    g = lambda **k: call(L.tp_linear_logprobs_dlogits,  # noqa: E731
                         "H E y lse ent g e T h v N scale d st stream",
                         (P, P, P, P, P, P, P, 4, 64, 304, 2, 1.0, P, None, None), **k)
    assert g(d=None) == g(y=None) == g(ent=None) == g(g=None, e=None) == NULL
    assert g(v=300) == g(h=60) == ALIGN
    assert g(scale=-1.0) == g(N=3) == SHAPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="a device answers instead")
def test_no_device_no_fallback(L):
    assert L.vp_logprobs_fwd(P, 1, P, 4, 300, 2, 1.0, 0, P, P, P, None, None, None, None) == DEVICE
    assert L.vp_distill(P, 1, P, P, None, 4, 300, 8, 2, 1, 1.0, 1.0, P, P, None, None, 0, P,
                        320, None, None) == DEVICE
