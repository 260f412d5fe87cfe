"""4-bit products whose K ends inside a step: what fills the step adds nothing.

The scales are so large that code 0 (8 below the zero point) stands for a weight
past the fp16 range while every real weight is finite, and some are infinite.
Results are held to the product of the weights as w4_dequantize_f16 gives them,
within the product's own roundings."""
import sys

import numpy as np
import pytest

import gemv_fp16_amd as gf
from tests import w4_plain as plain
from tests.util import dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gf.lib()
    yield
    torch.cuda.synchronize()


def _say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def _rows(rng, M, K):
    """Positive, far from zero and small: products with weights up to 60000 stay finite."""
    return (rng.uniform(0.5, 1.0, (M, K)) * 2.0 ** -13).astype(np.float16)


def _large_weights(rng, N, K, group):
    """Symmetric codes of weights up to 60000 in every group (a scale of 8568:
    codes 1 to 15 stand for -59976 to 59976, code 0 would for -68544)."""
    W = np.clip(rng.standard_normal((N, K)) * 15000, -59000, 59000).astype(np.float16)
    W[:, ::group] = np.where(rng.integers(0, 2, W[:, ::group].shape), 60000, -60000)
    return W


def _check(C, A, back, what):
    """C against A . back^T in float64, where back are fp16 weights."""
    a, w = A.astype(np.float64), back.astype(np.float64)
    with np.errstate(all="ignore"):
        plain.check(C, a @ w.T, np.abs(a) @ np.abs(w).T, A.shape[1], plain.F16, what)


# few rows, then tiles of 32 x 128, 64 x 128, 128 x 128, 128 x 256 and 256 x 256
SIZES = [(20, 50), (70, 50), (100, 8204), (700, 4000), (1500, 4357), (2900, 4100)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("K", [72, 104, 120, 296])
@pytest.mark.parametrize("M,N", SIZES)
def test_padding_past_the_fp16_range(M, N, K, group):
    rng = np.random.default_rng(M + K + group)
    A, W = _rows(rng, M, K), _large_weights(rng, N, K, group)
    _say("padding", M, N, K, group)
    Q, S, Z = gf.w4_quantize_f16(dev(W), group, symmetric=True)
    back = gf.w4_dequantize_f16(Q, S, Z, group).cpu().numpy()
    assert np.isfinite(back).all()
    C = gf.gemm_w4_f16_nt(dev(A), Q, S, Z, group=group).cpu().numpy()
    assert np.isfinite(C).all()
    if M <= 64:                                            # the weights are not rounded
        back = plain.weights(plain.unpack(Q.cpu().numpy()), S.cpu().numpy(), None, group)
    _check(C, A, back, "padding")


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("K", [72, 104, 296])
def test_padding_of_infinite_weights(K, zeros, group):
    """Columns whose last group has an infinite scale, or weights past the fp16
    range: all of one sign, so that the column is infinite and not NaN."""
    rng = np.random.default_rng(K + group)
    M, N, G = 70, 50, plain.groups_of(K, group)
    A, q = _rows(rng, M, K), rng.integers(0, 16, (N, K)).astype(np.uint8)
    S = rng.uniform(0.5, 1.5, (N, G)).astype(np.float16)
    Z = rng.integers(2, 13, (N, G)).astype(np.uint8) if zeros else None
    last = (G - 1) * group
    for n, s, code in ((3, np.inf, 15), (4, np.inf, 1), (5, 40000, 15), (6, -np.inf, 15), (7, 40000, 1)):
        S[n, -1] = np.float16(s)
        q[n, last:] = code
        if zeros:
            Z[n, -1] = 8
    S[9, -1] = np.float16("nan")
    _say("infinite padding", K, zeros, group)
    dQ, dS, dZ = dev(plain.pack(q)), dev(S), None if Z is None else dev(Z)
    with np.errstate(all="ignore"):
        back = plain.weights(q, S, Z, group).astype(np.float16)
    C = gf.gemm_w4_f16_nt(dev(A), dQ, dS, dZ, group=group).cpu().numpy()
    assert (C[:, [3, 5]] == np.inf).all() and (C[:, [4, 6, 7]] == -np.inf).all() and np.isnan(C[:, 9]).all()
    _check(C, A, back, "infinite padding")


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("K", [72, 104, 296])
@pytest.mark.parametrize("sizes,N", [((40, 0, 33, 31), 2309), ((150, 1, 99, 0), 2309), ((400, 0, 130, 257), 2309)])
def test_grouped_padding_past_the_fp16_range(sizes, N, K, group):
    """By expert: tiles of 32, 64 and 128 rows."""
    rng = np.random.default_rng(K + group)
    E, T, off = len(sizes), sum(sizes), plain.offsets_of(sizes)
    A, W = _rows(rng, T, K), _large_weights(rng, E * N, K, group).reshape(E, N, K)
    _say("grouped padding", sizes, K, group)
    Q, S, Z = gf.w4_quantize_f16(dev(W), group, symmetric=True)
    back = gf.w4_dequantize_f16(Q, S, Z, group).cpu().numpy()
    C = gf.gemm_w4_f16_grouped_nt(dev(A), Q, S, Z, dev(off), group=group).cpu().numpy()
    assert np.isfinite(C).all()
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if sizes[e]:
            _check(C[r], A[r], back[e], "group %d" % e)
