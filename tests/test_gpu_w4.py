"""4-bit weights on the GPU against plain 64-bit forms.

Codes, scales, zero points and the weights they stand for are compared bit for
bit.  Products are held to half a step of their fp16 result plus the fp32
roundings of the sum (w4_plain.bound)."""
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


def _f16(rng, shape, scale=1.0):
    return (rng.standard_normal(shape) * scale).astype(np.float16)


def _codes(rng, N, K, group, zeros):
    """Random codes, scales of both signs and sizes, zero points."""
    G = plain.groups_of(K, group)
    q = rng.integers(0, 16, (N, K)).astype(np.uint8)
    S = (rng.uniform(-1, 1, (N, G)) * 2.0 ** rng.integers(-8, 2, (N, G))).astype(np.float16)
    Z = rng.integers(0, 16, (N, G)).astype(np.uint8) if zeros else None
    return q, S, Z


def _shifted(t, elems):
    """A contiguous copy of t whose first element lies `elems` past an allocation."""
    flat = torch.empty(t.numel() + elems, dtype=t.dtype, device=t.device)
    out = flat[elems:].view(t.shape)
    out.copy_(t)
    return out


# ---- quantize -------------------------------------------------------------

def _weights_case(rng, N, K):
    """Rows of different spread, and rows of special values."""
    W = (rng.standard_normal((N, K)) * 2.0 ** rng.integers(-12, 8, (N, 1))).astype(np.float16)
    if N >= 8:
        W[0] = 0
        W[1] = np.float16(0.25)                       # constant
        W[2] = -np.abs(W[2])                          # one sign
        W[3] = (rng.integers(-40, 40, K) * 2.0 ** -24).astype(np.float16)     # subnormals: s may be 0
        W[4] = rng.integers(-15, 16, K).astype(np.float16) / 2                # many ties
        W[5, 0] = np.float16(65504)
        W[5, -1] = np.float16(-65504)
        W[6, rng.integers(0, K)] = np.float16("inf")
        W[7, rng.integers(0, K)] = np.float16("nan")
    return W


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [False, True])
@pytest.mark.parametrize("N,K", [(1, 8), (9, 32), (33, 136), (10, 1000), (130, 2056), (300, 4096)])
def test_quantize_is_exact(group, symmetric, N, K):
    rng = np.random.default_rng(N * 10007 + K + group)
    W = _weights_case(rng, N, K)
    q, S, Z = plain.quantize(W, group, symmetric)
    _say("quantize", N, K, group, symmetric)
    for shift in (0, 1):
        gQ, gS, gZ = gf.w4_quantize_f16(_shifted(dev(W), shift), group, symmetric)
        gW = gf.w4_dequantize_f16(gQ, gS, gZ, group, W=_shifted(torch.zeros((N, K), dtype=torch.float16, device="cuda"), shift))
        torch.cuda.synchronize()
        got = gS.cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(S))
        assert np.array_equal(got[~np.isnan(S)].view(np.uint16), S[~np.isnan(S)].view(np.uint16))
        if not symmetric:
            assert np.array_equal(gZ.cpu().numpy(), Z)
        assert np.array_equal(plain.unpack(gQ.cpu().numpy()), q)
        back = plain.weights(q, S, Z, group).astype(np.float16)
        gW = gW.cpu().numpy()
        assert np.array_equal(np.isnan(gW), np.isnan(back))
        assert np.array_equal(gW[~np.isnan(back)], back[~np.isnan(back)])


def test_quantize_every_tie_and_neighbour():
    """Quotients at and one fp16 step beside every k + 1/2, over many scales."""
    rng = np.random.default_rng(5)
    rows = []
    for _ in range(400):
        s = np.float16(2.0 ** rng.uniform(-14, 6))
        top = np.float16(7 * np.float64(s))           # sets the scale near s
        t = ((np.arange(-7, 7) + 0.5) * np.float64(s)).astype(np.float16)
        row = np.concatenate([t, np.nextafter(t, np.float16(np.inf)), [top, -top, 0, s]]).astype(np.float16)
        rows.append(row)
    W = np.stack(rows)
    assert W.shape[1] == 32
    for symmetric in (True, False):
        q, S, Z = plain.quantize(W, 32, symmetric)
        gQ, gS, gZ = gf.w4_quantize_f16(dev(W), 32, symmetric)
        assert np.array_equal(gS.cpu().numpy().view(np.uint16), S.view(np.uint16))
        assert np.array_equal(plain.unpack(gQ.cpu().numpy()), q)


def test_quantize_experts_as_one():
    rng = np.random.default_rng(6)
    W = _f16(rng, (3, 40, 256), 0.05)
    Q, S, Z = gf.w4_quantize_f16(dev(W), 64)
    Q2, S2, Z2 = gf.w4_quantize_f16(dev(W.reshape(120, 256)), 64)
    assert torch.equal(Q.view(120, -1), Q2) and torch.equal(S.view(120, -1), S2) and torch.equal(Z.view(120, -1), Z2)
    assert torch.equal(gf.w4_dequantize_f16(Q, S, Z, 64).view(120, 256), gf.w4_dequantize_f16(Q2, S2, Z2, 64))


# ---- products -------------------------------------------------------------

def _product(A, q, S, Z, group, shift_a=0, shift_q=0):
    N, K = q.shape
    dA, dQ = _shifted(dev(A), shift_a), _shifted(dev(plain.pack(q)), shift_q)
    return dA, dQ, dev(S), None if Z is None else dev(Z)


def _check_product(C, A, q, S, Z, group, what):
    W = plain.weights(q, S, Z, group)
    a = A.astype(np.float64)
    with np.errstate(all="ignore"):
        absum = np.abs(a) @ np.abs(W).T
        plain.check(C, a @ W.T, absum, A.shape[1], plain.F16, what, _extra(A, absum))


def _extra(A, absum):
    """From 65 rows of A on, weights are rounded to fp16 before the product."""
    if A.shape[0] <= 64:
        return 0.0
    return plain.rounded_weights(absum, np.abs(A.astype(np.float64)).sum(1, keepdims=True))


SHAPES = [(1, 1, 8), (1, 16, 32), (1, 100, 4096), (2, 33, 136), (3, 64, 1000), (15, 15, 256), (16, 48, 128),
          (17, 31, 640), (33, 130, 2056), (64, 64, 2048), (65, 200, 1024), (130, 77, 512), (200, 300, 416),
          (66, 40, 32), (300, 520, 160), (1700, 7000, 96), (1, 50, 5128), (20, 8200, 264), (50, 8200, 520),
          (65, 70, 64), (90, 40, 72), (100, 150, 104), (130, 140, 1112), (1700, 7000, 120), (1, 16, 1536),
          (1, 8200, 1024), (16, 9000, 512), (9, 33, 8192), (12, 2000, 4608), (32, 130, 4096), (5, 17, 512)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_w4(M, N, K, group, zeros):
    rng = np.random.default_rng(M * 1009 + N * 31 + K + group)
    A, (q, S, Z) = _f16(rng, (M, K)), _codes(rng, N, K, group, zeros)
    _say("gemm_w4", M, N, K, group, zeros)
    dA, dQ, dS, dZ = _product(A, q, S, Z, group)
    C = gf.gemm_w4_f16_nt(dA, dQ, dS, dZ, group=group)
    again = gf.gemm_w4_f16_nt(dA, dQ, dS, dZ, group=group)
    torch.cuda.synchronize()
    assert torch.equal(C.view(torch.int16), again.view(torch.int16))
    _check_product(C.cpu().numpy(), A, q, S, Z, group, "gemm_w4 %dx%dx%d" % (M, N, K))
    if M == 1:
        y = gf.gemv_w4_f16(dQ, dS, dZ, dA.view(-1), group=group)
        assert torch.equal(y.view(1, -1).view(torch.int16), C.view(torch.int16))


@pytest.mark.parametrize("shift_a,shift_q", [(1, 0), (0, 1), (3, 3)])
@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_gemm_w4_off_the_16_byte_grid(M, shift_a, shift_q):
    rng = np.random.default_rng(M + shift_a)
    N, K, group = 70, 512, 64
    A, (q, S, Z) = _f16(rng, (M, K)), _codes(rng, N, K, group, True)
    _say("gemm_w4 shifted", M, shift_a, shift_q)
    C = gf.gemm_w4_f16_nt(*_product(A, q, S, Z, group, shift_a, shift_q), group=group)
    _check_product(C.cpu().numpy(), A, q, S, Z, group, "shifted")


@pytest.mark.parametrize("M", [1, 4, 30, 70, 300])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("K", [8 * 37, 32 * 9, 512])      # the first two with a short last group
def test_gemm_w4_infinities_and_nan(M, group, K):
    """An infinite or NaN entry of A or S shows in its row or column as the
    formula has it, and nowhere else; the group behind the last is not read."""
    rng = np.random.default_rng(M)
    N = 50
    A, (q, S, Z) = _f16(rng, (M, K)), _codes(rng, N, K, group, True)
    A[0, 5], A[M - 1, K - 1] = np.float16("inf"), np.float16("nan")
    q[:, 5] = np.where(q[:, 5] == Z[:, 0], (Z[:, 0] + 1) % 16, q[:, 5])     # inf * 0 apart
    q[7, 5] = Z[7, 0]                                 # and once on purpose
    S[3, -1], S[4, 0] = np.float16("inf"), np.float16("nan")
    _say("gemm_w4 special", M, group)
    W = plain.weights(q, S, Z, group)
    C = gf.gemm_w4_f16_nt(*_product(A, q, S, Z, group), group=group).cpu().numpy()
    a = A.astype(np.float64)
    # column 3: the infinite scale multiplies the group's sum, which the formula's
    # products spell as inf or NaN (an infinite sum of both signs): not finite is what counts
    with np.errstate(all="ignore"):
        exact, absum = a @ W.T, np.abs(a) @ np.abs(W).T
    keep = [n for n in range(N) if n != 3]
    assert not np.isfinite(C[:, 3].astype(np.float64)).any()
    extra = _extra(A, absum)
    plain.check(C[:, keep], exact[:, keep], absum[:, keep], K, plain.F16, "special",
                extra if np.isscalar(extra) else extra[:, keep])


def test_gemm_w4_empty_and_k0():
    z = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt, device="cuda")
    C = torch.full((3, 5), 7.0, dtype=torch.float16, device="cuda")
    gf.gemm_w4_f16_nt(z(3, 0), z(5, 0, dt=torch.int32), z(5, 0), None, C)
    assert torch.equal(C, torch.zeros_like(C)) and not torch.signbit(C).any()
    assert gf.gemm_w4_f16_nt(z(0, 64), z(5, 8, dt=torch.int32), z(5, 1), None).shape == (0, 5)
    assert gf.gemm_w4_f16_nt(z(2, 64), z(0, 8, dt=torch.int32), z(0, 1), None).shape == (2, 0)
    Q, S, Z = gf.w4_quantize_f16(z(0, 64))
    assert Q.shape == (0, 8) and gf.w4_dequantize_f16(Q, S, Z).shape == (0, 64)


@pytest.mark.parametrize("M,N,K", [(1, 8192, 8192), (8, 4096, 14336), (24, 11008, 4096), (300, 2048, 4096),
                                   (2048, 1024, 2048)])
def test_gemm_w4_full_size(M, N, K):
    """Every output at serving sizes, against float64 on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(M)
    W = (torch.randn((N, K), generator=g, device="cuda") * 0.02).half()
    A = torch.randn((M, K), generator=g, device="cuda").half()
    _say("gemm_w4 full", M, N, K)
    Q, S, Z = gf.w4_quantize_f16(W, 128)
    C = gf.gemm_w4_f16_nt(A, Q, S, Z)
    q, Sn, Zn = plain.unpack(Q.cpu().numpy()), S.cpu().numpy(), Z.cpu().numpy()
    Wd = torch.from_numpy(plain.weights(q, Sn, Zn, 128)).cuda()
    a = A.double()
    exact, absum = a @ Wd.t(), a.abs() @ Wd.abs().t()
    absum = absum.cpu().numpy()
    plain.check(C.cpu().numpy(), exact.cpu().numpy(), absum, K, plain.F16, "full", _extra(A.cpu().numpy(), absum))


@pytest.mark.parametrize("group", [32, 64, 128])
def test_gemm_w4_of_many_rows_is_the_product_of_the_weights_read_back(group):
    """From 65 rows on, within the product's own roundings."""
    rng = np.random.default_rng(group)
    M, N, K = 300, 264, 608
    A, (q, S, Z) = _f16(rng, (M, K)), _codes(rng, N, K, group, True)
    dA, dQ, dS, dZ = _product(A, q, S, Z, group)
    C = gf.gemm_w4_f16_nt(dA, dQ, dS, dZ, group=group).cpu().numpy().astype(np.float64)
    W = gf.w4_dequantize_f16(dQ, dS, dZ, group).cpu().numpy().astype(np.float64)
    a = A.astype(np.float64)
    plain.check(C, a @ W.T, np.abs(a) @ np.abs(W).T, K, plain.F16, "read back")
