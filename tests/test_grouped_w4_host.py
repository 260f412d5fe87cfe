"""Refusals of the grouped and 4-bit calls, checked on the host: no call here
reaches a kernel launch (every one fails validation or is a documented no-op),
and the plain forms the GPU tests compare with, against brute force."""
import ctypes
import os

import numpy as np
import pytest

import gemv_fp16_amd as gf
from tests import w4_plain as plain


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gf.LIB_PATH):
        from gemv_fp16_amd import build
        build.build()
    return gf.lib()


P = ctypes.c_void_p(0x10000)      # never dereferenced
ODD = ctypes.c_void_p(0x10001)
TWO = ctypes.c_void_p(0x10002)
NULL = ctypes.c_void_p(0)
BAD, OK = gf.GF_ERR_INVALID_ARG, gf.GF_OK


@pytest.mark.parametrize("name", ["gemm_f16_grouped_nt", "gemm_f16_grouped_nn"])
def test_grouped_rows_refusals(L, name):
    f = getattr(L, name)
    assert f(P, P, P, P, -1, 2, 8, 8, NULL) == BAD
    assert f(P, P, P, P, 4, -2, 8, 8, NULL) == BAD
    assert f(P, P, P, P, 4, 2, -8, 8, NULL) == BAD
    assert f(P, P, P, P, 4, 2, 8, -8, NULL) == BAD
    assert f(ODD, P, P, P, 4, 2, 8, 8, NULL) == BAD
    assert f(P, ODD, P, P, 4, 2, 8, 8, NULL) == BAD
    assert f(P, P, ODD, P, 4, 2, 8, 8, NULL) == BAD
    assert f(P, P, P, TWO, 4, 2, 8, 8, NULL) == BAD
    assert f(NULL, P, P, P, 4, 2, 8, 8, NULL) == BAD
    assert f(P, NULL, P, P, 4, 2, 8, 8, NULL) == BAD
    assert f(P, P, NULL, P, 4, 2, 8, 8, NULL) == BAD
    assert f(P, P, P, NULL, 4, 2, 8, 8, NULL) == BAD
    assert f(P, P, P, P, 65536, 2, 8, 65536, NULL) == BAD     # A of 2^32 elements
    assert f(P, P, P, P, 65536, 2, 65536, 8, NULL) == BAD     # C
    assert f(P, P, P, P, 4, 2, 65536, 65536, NULL) == BAD     # one group's B
    assert f(NULL, P, NULL, P, 0, 2, 8, 8, NULL) == OK        # no rows
    assert f(P, NULL, P, NULL, 4, 0, 8, 8, NULL) == OK        # no groups
    assert f(P, NULL, NULL, P, 4, 2, 0, 8, NULL) == OK        # no columns


def test_grouped_tn_refusals(L):
    f = L.gemm_f16_grouped_tn
    for T, E, M, N in ((-1, 2, 8, 8), (4, -2, 8, 8), (4, 2, -8, 8), (4, 2, 8, -8)):
        assert f(P, P, P, P, T, E, M, N, 0, NULL) == BAD
    assert f(P, P, P, P, 4, 2, 8, 8, 2, NULL) == BAD
    assert f(P, P, TWO, P, 4, 2, 8, 8, 1, NULL) == BAD        # float C off its grid
    assert f(P, P, ODD, P, 4, 2, 8, 8, 0, NULL) == BAD
    assert f(NULL, P, P, P, 4, 2, 8, 8, 0, NULL) == BAD
    assert f(P, NULL, P, P, 4, 2, 8, 8, 0, NULL) == BAD
    assert f(P, P, P, P, 4, 2, 65536, 65536, 0, NULL) == BAD
    assert f(P, P, NULL, NULL, 4, 0, 8, 8, 0, NULL) == OK
    assert f(P, P, NULL, P, 4, 2, 0, 8, 0, NULL) == OK


def test_w4_refusals(L):
    for f in (L.w4_quantize_f16, L.w4_dequantize_f16):
        for N, K, g in ((4, 12, 32), (4, 64, 16), (4, 64, 0), (-1, 64, 32), (4, -8, 32)):
            assert f(P, P, P, P, N, K, g, NULL) == BAD
        assert f(NULL, NULL, NULL, NULL, 0, 64, 32, NULL) == OK
        assert f(NULL, NULL, NULL, NULL, 4, 0, 32, NULL) == OK
    assert L.w4_quantize_f16(ODD, P, P, P, 4, 64, 32, NULL) == BAD
    assert L.w4_quantize_f16(P, TWO, P, P, 4, 64, 32, NULL) == BAD
    assert L.w4_dequantize_f16(TWO, P, P, P, 4, 64, 32, NULL) == BAD
    assert L.w4_dequantize_f16(P, ODD, P, P, 4, 64, 32, NULL) == BAD
    assert L.w4_dequantize_f16(P, P, P, ODD, 4, 64, 32, NULL) == BAD

    f = L.gemm_w4_f16_nt
    for M, N, K, g in ((-1, 4, 64, 32), (4, -1, 64, 32), (4, 4, 60, 32), (4, 4, 64, 48), (65536, 4, 65536, 32),
                       (4, 65536, 65536, 32), (65536, 65536, 8, 32)):
        assert f(P, P, P, P, P, M, N, K, g, NULL) == BAD
    assert f(ODD, P, P, P, P, 4, 4, 64, 32, NULL) == BAD
    assert f(P, TWO, P, P, P, 4, 4, 64, 32, NULL) == BAD
    assert f(P, P, ODD, P, P, 4, 4, 64, 32, NULL) == BAD
    assert f(P, P, P, P, ODD, 4, 4, 64, 32, NULL) == BAD
    assert f(P, P, P, P, NULL, 4, 4, 64, 32, NULL) == BAD
    assert f(NULL, P, P, P, P, 4, 4, 64, 32, NULL) == BAD
    assert f(NULL, P, P, P, NULL, 0, 4, 64, 32, NULL) == OK
    assert f(P, NULL, NULL, NULL, NULL, 4, 0, 64, 32, NULL) == OK
    assert L.gemv_w4_f16(P, P, P, P, P, 4, 60, 32, NULL) == BAD
    assert L.gemv_w4_f16(NULL, P, P, P, P, 4, 64, 32, NULL) == BAD

    f = L.gemm_w4_f16_grouped_nt
    assert f(P, P, P, P, P, P, 4, 2, 8, 60, 32, NULL) == BAD
    assert f(P, P, P, P, P, P, -4, 2, 8, 64, 32, NULL) == BAD
    assert f(P, P, P, P, P, P, 4, -2, 8, 64, 32, NULL) == BAD
    assert f(P, P, P, P, P, TWO, 4, 2, 8, 64, 32, NULL) == BAD
    assert f(P, P, P, P, P, NULL, 4, 2, 8, 64, 32, NULL) == BAD
    assert f(P, NULL, P, P, P, P, 4, 2, 8, 64, 32, NULL) == BAD
    assert f(NULL, P, P, P, NULL, P, 0, 2, 8, 64, 32, NULL) == OK
    assert f(P, P, P, P, P, NULL, 4, 0, 8, 64, 32, NULL) == OK


def test_sizes_past_the_limits(L):
    """What the kernels round up in 32 bits, and how many groups they look through."""
    big = 2 ** 30 + 8
    for f in (L.gemm_f16_grouped_nt, L.gemm_f16_grouped_nn):
        assert f(P, P, P, P, big, 1, 1, 1, NULL) == BAD
        assert f(P, P, P, P, 1, 1, big, 1, NULL) == BAD
        assert f(P, P, P, P, 1, 1, 1, big, NULL) == BAD
        assert f(P, P, P, P, 1, 65537, 1, 1, NULL) == BAD
    assert L.gemm_f16_grouped_tn(P, P, P, P, big, 1, 1, 1, 0, NULL) == BAD
    assert L.gemm_f16_grouped_tn(P, P, P, P, 1, 65537, 1, 1, 0, NULL) == BAD
    assert L.gemm_w4_f16_nt(P, P, P, P, P, 1, 1, big, 32, NULL) == BAD
    assert L.gemm_w4_f16_nt(P, P, P, P, P, 1, big, 0, 32, NULL) == BAD
    assert L.gemm_w4_f16_nt(P, P, P, P, P, big, 1, 0, 32, NULL) == BAD
    assert L.gemm_w4_f16_grouped_nt(P, P, P, P, P, P, 1, 65537, 1, 8, 32, NULL) == BAD
    assert L.gemm_w4_f16_grouped_nt(P, P, P, P, P, P, big, 1, 1, 0, 32, NULL) == BAD
    assert L.w4_quantize_f16(P, P, P, P, 1, big, 32, NULL) == BAD


def test_binding_refusals():
    """The binding's own checks come before the library is called."""
    torch = pytest.importorskip("torch")
    h = lambda *s: torch.zeros(s, dtype=torch.float16)
    with pytest.raises(ValueError):
        gf.gemm_f16_grouped_nt(h(4, 8), h(2, 8, 16), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        gf.gemm_f16_grouped_nn(h(4, 8), h(2, 16, 8), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        gf.gemm_f16_grouped_tn(h(4, 8), h(5, 8), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        gf.w4_quantize_f16(h(4, 12))
    with pytest.raises(ValueError):
        gf.w4_quantize_f16(h(4, 16), group=48)
    with pytest.raises(ValueError):
        gf.w4_quantize_f16(h(4, 16), symmetric=True, Z=torch.zeros((4, 1), dtype=torch.uint8))
    with pytest.raises(TypeError):                    # host tensors
        gf.w4_quantize_f16(h(4, 16))
    Q = torch.zeros((4, 8), dtype=torch.int32)
    with pytest.raises(ValueError):                   # S of another group size
        gf.gemm_w4_f16_nt(h(1, 64), Q, h(4, 2), None, group=64)
    with pytest.raises(TypeError):
        gf.gemm_w4_f16_nt(h(1, 64), Q, h(4, 1), None, group=64)


# ---- the plain forms themselves -------------------------------------------

def test_pack_and_unpack():
    rng = np.random.default_rng(0)
    q = rng.integers(0, 16, (3, 24)).astype(np.uint8)
    w = plain.pack(q)
    assert w.shape == (3, 3)
    for n in range(3):
        for k in range(24):
            assert (int(w[n, k // 8]) >> (4 * (k % 8))) & 15 == q[n, k]
    assert np.array_equal(plain.unpack(w), q)


@pytest.mark.parametrize("symmetric", [True, False])
def test_plain_quantize_against_fractions(symmetric):
    """Entry by entry in exact rational arithmetic, ties to even."""
    from fractions import Fraction
    rng = np.random.default_rng(1)
    W = np.concatenate([(rng.standard_normal((6, 40)) * 0.1), rng.integers(-15, 16, (4, 40)) / 2]).astype(np.float16)
    q, S, Z = plain.quantize(W, 32, symmetric)

    def nearest(x):
        f = x.numerator // x.denominator
        r = x - f
        return f + (1 if r > Fraction(1, 2) or (r == Fraction(1, 2) and f % 2) else 0)

    for n in range(W.shape[0]):
        for g, (k0, k1) in enumerate(((0, 32), (32, 40))):
            w = [Fraction(float(v)) for v in W[n, k0:k1]]
            lo, hi = min(w + [Fraction(0)]), max(w + [Fraction(0)])
            t = max(hi, -lo) / 7 if symmetric else (hi - lo) / 15
            assert float(S[n, g]) == float(np.float16(np.float32(float(t))))
            s = Fraction(float(S[n, g]))
            z = 8 if symmetric else min(15, nearest(-lo / s))
            if not symmetric:
                assert Z[n, g] == z
            for i, v in enumerate(w):
                assert q[n, k0 + i] == max(0, min(15, nearest(v / s) + z))


def test_bound_counts_half_a_step():
    x = np.float64(1.0) + 2.0 ** -11 * 0.999
    plain.check(np.array([np.float16(1.0)]), np.array([x]), np.array([1.0]), 1, plain.F16)
    with pytest.raises(AssertionError):
        plain.check(np.array([np.float16(1.0) + np.float16(2.0 ** -10)]), np.array([1.0]), np.array([1.0]), 1, plain.F16)
