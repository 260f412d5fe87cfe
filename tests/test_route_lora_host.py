"""Refusals of the routing, row and adapter calls, checked on the host: no call
here reaches a kernel launch.  And the plain gradient that the GPU tests compare
with, against differences."""
import ctypes
import os

import numpy as np
import pytest

import gemv_fp16_amd as gf
from tests import route_plain as plain


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gf.LIB_PATH):
        from gemv_fp16_amd import build
        build.build()
    return gf.lib()


P = ctypes.c_void_p(0x10000)      # never dereferenced
ODD = ctypes.c_void_p(0x10001)
TWO = ctypes.c_void_p(0x10002)
FOUR = ctypes.c_void_p(0x10004)
NULL = ctypes.c_void_p(0)
BAD, OK = gf.GF_ERR_INVALID_ARG, gf.GF_OK


def cfg(score=0, renorm=1, groups=1, top_groups=1, group_best=1, scale=1.0):
    return ctypes.byref(gf.RouteCfg(score, renorm, groups, top_groups, group_best, scale))


def test_route_topk_refusals(L):
    need = L.route_workspace_bytes(65, 8, 2)
    assert need > 0

    def f(x=P, f32=0, bias=NULL, T=4, E=8, k=2, c=cfg(), ids=P, w=P, off=P, at=P, ws=P, n=1 << 20):
        return L.route_topk(x, f32, bias, T, E, k, c, ids, w, off, at, ws, n, NULL)
    for bad in (dict(T=-1), dict(E=0), dict(E=-8), dict(k=0), dict(k=-1), dict(k=9), dict(f32=2), dict(f32=-1),
                dict(E=1025), dict(E=1024, k=65), dict(T=2 ** 30 + 1, E=1, k=1), dict(T=2 ** 21, E=1024),
                dict(c=None), dict(c=cfg(score=2)), dict(c=cfg(score=-1)), dict(c=cfg(renorm=2)),
                dict(c=cfg(groups=0)), dict(c=cfg(groups=3)), dict(c=cfg(groups=2, top_groups=3)),
                dict(c=cfg(groups=2, top_groups=0)), dict(c=cfg(group_best=0)), dict(c=cfg(group_best=3)),
                dict(c=cfg(groups=8), k=2), dict(E=65 * 2, c=cfg(groups=65)), dict(c=cfg(scale=float("nan"))),
                dict(x=ODD), dict(x=TWO, f32=1), dict(x=NULL), dict(bias=TWO), dict(ids=NULL), dict(ids=TWO), dict(w=NULL),
                dict(w=TWO), dict(off=NULL), dict(at=NULL), dict(off=TWO), dict(at=TWO), dict(T=65, ws=NULL),
                dict(T=65, ws=TWO), dict(T=65, n=need - 1)):
        assert f(**bad) == BAD, bad
    assert f(T=0, x=NULL, ids=NULL, w=NULL, off=NULL, at=NULL, ws=NULL, n=0) == OK
    assert L.route_workspace_bytes(16, 8, 2) == 0
    assert L.route_workspace_bytes(2 ** 30, 1, 1) >= 2 ** 30 // 65535 * 2      # no chunk past 16 bits
    assert L.route_workspace_bytes(-1, 8, 2) == 0


def test_route_rows_refusals(L):
    def f(ids=P, T=4, k=2, E=8, off=P, at=P, ws=P, n=1 << 20):
        return L.route_rows(ids, T, k, E, off, at, ws, n, NULL)
    for bad in (dict(T=-1), dict(k=0), dict(E=0), dict(E=1025), dict(T=2 ** 30 + 1, k=1), dict(T=2 ** 30, k=2),
                dict(ids=NULL), dict(ids=TWO), dict(off=NULL), dict(off=TWO), dict(at=NULL), dict(at=ODD),
                dict(T=4097, k=1, ws=NULL), dict(T=4097, k=1, n=100)):
        assert f(**bad) == BAD, bad


def test_route_topk_bwd_refusals(L):
    def f(x=P, f32=0, ids=P, dw=P, T=4, E=8, k=2, c=cfg(), dx=P):
        return L.route_topk_bwd(x, f32, ids, dw, T, E, k, c, dx, NULL)
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=9), dict(E=1025), dict(f32=3), dict(c=None), dict(c=cfg(score=5)),
                dict(x=NULL), dict(x=ODD), dict(x=TWO, f32=1), dict(dx=NULL), dict(dx=TWO, f32=1), dict(ids=TWO),
                dict(ids=NULL), dict(dw=NULL), dict(dw=TWO), dict(T=2 ** 28)):
        assert f(**bad) == BAD, bad
    assert f(T=0, x=NULL, ids=NULL, dw=NULL, dx=NULL) == OK


def test_rows_refusals(L):
    def d(X=P, at=P, A=P, T=4, k=2, R=8, D=16):
        return L.dispatch_f16(X, at, A, T, k, R, D, NULL)

    def c(C=P, at=P, w=P, Y=P, T=4, k=2, R=8, D=16):
        return L.combine_f16(C, at, w, Y, T, k, R, D, NULL)

    def b(dY=P, C=P, at=P, w=P, dC=P, dw=P, T=4, k=2, R=8, D=16):
        return L.combine_f16_bwd(dY, C, at, w, dC, dw, T, k, R, D, NULL)
    for f in (d, c, b):
        for bad in (dict(T=-1), dict(k=0), dict(k=65), dict(R=-1), dict(D=-1), dict(T=2 ** 30 + 1, D=1), dict(at=NULL),
                    dict(at=TWO), dict(T=65536, D=65536), dict(R=65536, D=65536), dict(T=2 ** 30, D=1, k=2),
                    dict(D=2 ** 30 + 1, T=1, R=1), dict(R=2 ** 30 + 1, D=1)):
            assert f(**bad) == BAD, bad
        assert f(T=0) == OK
    assert d(D=0) == OK and c(D=0) == OK and d(R=0, A=NULL) == OK
    for bad in (dict(X=ODD), dict(X=NULL), dict(A=ODD), dict(A=NULL)):
        assert d(**bad) == BAD, bad
    for bad in (dict(C=ODD), dict(C=NULL), dict(Y=ODD), dict(Y=NULL), dict(w=TWO)):
        assert c(**bad) == BAD, bad
    for bad in (dict(dY=ODD), dict(dY=NULL), dict(C=NULL), dict(C=ODD), dict(dC=NULL), dict(dC=ODD), dict(w=NULL),
                dict(w=TWO), dict(dw=NULL), dict(dw=TWO)):
        assert b(**bad) == BAD, bad


def test_lora_refusals(L):
    need = L.lora_workspace_bytes(4, 16, 64, 8)
    assert need > 0

    def add(A=P, ids=P, Dn=P, Up=P, s=NULL, C=P, M=4, N=16, K=64, r=8, n=2, ws=P, b=1 << 30):
        return L.lora_add_f16(A, ids, Dn, Up, s, C, M, N, K, r, n, ws, b, NULL)

    def gemm(A=P, B=P, ids=P, Dn=P, Up=P, s=NULL, C=P, M=4, N=16, K=64, r=8, n=2, ws=P, b=1 << 30):
        return L.gemm_f16_nt_lora(A, B, ids, Dn, Up, s, C, M, N, K, r, n, ws, b, NULL)
    for f in (add, gemm):
        for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(r=0), dict(r=257), dict(r=-8), dict(n=-1),
                    dict(M=65536, K=65536), dict(N=65536, K=65536), dict(M=65536, N=65536), dict(K=2 ** 30 + 8, M=1, N=1, r=1),
                    dict(K=2 ** 28, M=1, N=1, r=16), dict(M=2 ** 25, r=64, K=8, N=8), dict(A=NULL), dict(A=ODD),
                    dict(ids=NULL), dict(ids=TWO), dict(Dn=NULL), dict(Dn=ODD), dict(Up=NULL), dict(Up=ODD), dict(s=TWO),
                    dict(C=NULL), dict(C=ODD), dict(ws=NULL), dict(ws=FOUR), dict(b=need - 1), dict(b=0)):
            assert f(**bad) == BAD, bad
        assert f(M=0, A=NULL, ids=NULL, C=NULL, ws=NULL, b=0) == OK
        assert f(N=0, Up=NULL, C=NULL, ws=NULL, b=0) == OK
    assert gemm(B=ODD) == BAD and gemm(B=NULL) == BAD
    assert add(n=0, Dn=NULL, Up=NULL) == OK
    for bad in ((-1, 1, 1, 1), (1, -1, 1, 1), (1, 1, -1, 1), (1, 1, 1, 0), (1, 1, 1, 257)):
        assert L.lora_workspace_bytes(*bad) == 0


def test_binding_refusals():
    """The binding's own checks come before the library is called."""
    torch = pytest.importorskip("torch")
    h = lambda *s: torch.zeros(s, dtype=torch.float16)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    f = lambda *s: torch.zeros(s)
    for call in (lambda: gf.route_topk(f(4), 1), lambda: gf.route_rows(i(4), 3),
                 lambda: gf.route_topk_bwd(f(4, 8), i(3, 2), f(3, 2)), lambda: gf.route_topk_bwd(f(4, 8), i(4, 2), f(4, 3)),
                 lambda: gf.dispatch_f16(h(4, 8), i(3, 2)), lambda: gf.dispatch_f16(h(4), i(4, 2)),
                 lambda: gf.combine_f16(h(4, 8), i(2)), lambda: gf.combine_f16(h(4, 8), i(2, 2), f(2, 3)),
                 lambda: gf.combine_f16_bwd(h(2, 8), h(4, 9), i(2, 2), f(2, 2)),
                 lambda: gf.combine_f16_bwd(h(2, 8), h(4, 8), i(2, 2), f(2, 1)),
                 lambda: gf.gemm_f16_nt_lora(h(2, 8), h(4, 8), i(3), h(2, 4, 8), h(2, 4, 4)),
                 lambda: gf.gemm_f16_nt_lora(h(2, 8), h(4, 8), i(2), h(2, 4, 9), h(2, 4, 4)),
                 lambda: gf.gemm_f16_nt_lora(h(2, 8), h(5, 8), i(2), h(2, 4, 8), h(2, 4, 4)),
                 lambda: gf.gemm_f16_nt_lora(h(2, 8), h(4, 8), i(2), h(2, 4, 8), h(2, 4, 4), f(3)),
                 lambda: gf.gemm_f16_nt_lora(h(2, 8), h(4, 8), i(2), h(2, 300, 8), h(2, 4, 300)),
                 lambda: gf.lora_add_f16(h(2, 8), i(2), h(2, 4, 8), h(2, 4, 4), None),
                 lambda: gf.lora_add_f16(h(2, 8), i(2), h(2, 4, 8), h(2, 4, 4), h(2, 5)),
                 lambda: gf.lora_add_f16(h(2, 8), i(2), h(3, 4, 8), h(2, 4, 4), h(2, 4))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: gf.route_topk(f(4, 8), 2), lambda: gf.dispatch_f16(h(4, 8), i(4, 2)),
                 lambda: gf.combine_f16(h(4, 8), i(2, 2))):
        with pytest.raises(TypeError):         # host tensors
            call()


@pytest.fixture
def _meta(monkeypatch):
    monkeypatch.setattr(gf, "_ptr", lambda t, dtype, name: 0x10000)

    def launch(name, tensors, stream, *args):
        raise AssertionError("%s reached with %s" % (name, args))

    monkeypatch.setattr(gf, "_launch", launch)
    torch = pytest.importorskip("torch")
    return lambda *shape, dtype=torch.float16: torch.empty(shape, dtype=dtype, device="meta")


def test_options_and_sizes_refused_by_the_binding(_meta):
    x = _meta(4, 8)
    for opt in (dict(score="tanh"), dict(scale=float("nan")), dict(bias=_meta(7)), dict(rows=False, offsets=_meta(9)),
                dict(ids=_meta(4, 3)), dict(offsets=_meta(8)), dict(place=_meta(3, 2)), dict(workspace=_meta(2, 2))):
        with pytest.raises(ValueError):
            gf.route_topk(x, 2, **opt)
    for k in (0, 9, -1):
        with pytest.raises(ValueError):
            gf.route_topk(x, k)
    with pytest.raises(ValueError):
        gf.route_topk(_meta(100, 8), 2, workspace=_meta(100))
    big = 2 ** 32 + 8
    for call in (lambda: gf.route_topk(_meta(big, 8), 2), lambda: gf.route_rows(_meta(big, 2), 4),
                 lambda: gf.route_rows(_meta(4, 2), big), lambda: gf.route_topk_bwd(_meta(big, 8), _meta(big, 2), _meta(big, 2)),
                 lambda: gf.dispatch_f16(_meta(big, 8), _meta(big, 1)), lambda: gf.dispatch_f16(_meta(2, 8), _meta(2, 1), A=_meta(big, 8)),
                 lambda: gf.combine_f16(_meta(big, 8), _meta(4, 2)),
                 lambda: gf.combine_f16_bwd(_meta(4, big), _meta(8, big), _meta(4, 2), _meta(4, 2)),
                 lambda: gf.gemm_f16_nt_lora(_meta(big, 8), _meta(4, 8), _meta(big), _meta(2, 4, 8), _meta(2, 4, 4)),
                 lambda: gf.lora_add_f16(_meta(2, 8), _meta(2), _meta(big, 4, 8), _meta(big, 4, 4), _meta(2, 4)),
                 lambda: gf.route_workspace_bytes(big, 8, 2), lambda: gf.lora_workspace_bytes(big, 8, 8, 8)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


# ---- the plain gradient ---------------------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_plain_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(2)
    for E, k in ((1, 1), (9, 3), (20, 20)):
        x, dw = rng.standard_normal(E), rng.standard_normal(k)
        ids = plain.choose(x, k, None, score)
        got, h = plain.grad(x, ids, dw, score, renorm, 1.7), 1e-5
        for e in range(E):
            up, dn = x.copy(), x.copy()
            up[e] += h
            dn[e] -= h
            diff = (dw * (plain.weights(up, ids, score, renorm, 1.7) - plain.weights(dn, ids, score, renorm, 1.7))).sum() / (2 * h)
            assert abs(diff - got[e]) <= 1e-8, (E, k, e)


def test_plain_choice_by_hand():
    x = [0.0, 2.0, 2.0, -np.inf, 1.0, 3.0]
    assert plain.choose(x, 3, None, "softmax") == [5, 1, 2]
    assert plain.choose(x, 6, None, "sigmoid") == [5, 1, 2, 4, 0, -1]
    assert plain.choose(x, 2, [9.0, 0, 0, 9.0, 0, 0], "sigmoid") == [0, 5]
    assert plain.choose(x, 2, None, "softmax", 3, 1, 1) == [5, 4]
    assert plain.choose([2.0, -5.0, 1.5, 1.4], 1, None, "sigmoid", 2, 1, 2) == [2]
    off, at = plain.rows([[1, 0], [2, 1], [-1, 1]], 3)
    assert list(off) == [0, 1, 4, 5] and at.tolist() == [[1, 0], [4, 2], [-1, 3]]
