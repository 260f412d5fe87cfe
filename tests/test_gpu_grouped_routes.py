"""Routes at their limits, for every form that walks them: offsets against the
contract stay inside the operands, a group's infinities and NaN stay in its own
rows, and no rows or no contraction give the empty sum."""
import sys

import numpy as np
import pytest

import gemv_fp16_amd as gf
from tests import w4_plain as plain
from tests.util import dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SENTINEL = 0x3A55


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gf.lib()
    yield
    torch.cuda.empty_cache()


def _say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def _half(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.float16, device="cuda").normal_(0.0, scale, generator=g)


def _sentinel(shape):
    return torch.full(shape, SENTINEL, dtype=torch.int16, device="cuda").view(torch.float16)


def _broken(T, E):
    """Routes of E groups over T rows against the contract: decreasing, negative,
    past T, overlapping, and at random."""
    rng = np.random.default_rng(T + E)
    yield np.linspace(T, 0, E + 1)
    yield np.where(np.arange(E + 1) % 2 == 0, 0, T)
    yield np.where(np.arange(E + 1) % 2 == 0, -2 ** 31, 2 ** 31 - 1)
    yield rng.integers(-T, 2 * T, E + 1)
    yield rng.integers(-2 ** 31, 2 ** 31 - 1, E + 1)


# a streaming form's mean of rows, in passes of 16 and 32 rows, and K in each number of parts of A; more
# groups than a wave's lanes; the launch in two parts (more than 256 tiles of 256 x 256); 128 x 128 tiles
ROUTES = [(12, 4, 72, 512), (44, 4, 72, 512), (40, 4, 72, 4096), (40, 4, 72, 8192), (200, 130, 48, 512),
          (700, 130, 48, 512), (2700, 2, 7000, 1032), (1300, 4, 2309, 1032)]


@pytest.mark.parametrize("T,E,N,K", ROUTES)
def test_offsets_against_the_contract(T, E, N, K):
    """The rows and weights beside the operands' in memory keep their contents."""
    A, B, D = _half(1, T, K), _half(2, E, N, K, scale=0.05), _half(3, T, N)
    codes = [(g, gf.w4_quantize_f16(B, g)) for g in (32, 64, 128)]
    whole, back = _sentinel((3 * T, N)), _sentinel((3 * T, K))
    dw = torch.full((3 * E, N, K), 7.0, dtype=torch.float16, device="cuda")
    for off in _broken(T, E):
        o = dev(off.astype(np.int64).clip(-2 ** 31, 2 ** 31 - 1).astype(np.int32))
        _say("broken offsets", T, E, N, K, off[:5])
        gf.gemm_f16_grouped_nt(A, B, o, whole[T:2 * T])
        for g, (Q, S, Z) in codes:
            gf.gemm_w4_f16_grouped_nt(A, Q, S, Z, o, whole[T:2 * T], g)
        gf.gemm_f16_grouped_nn(D, B, o, back[T:2 * T])
        gf.gemm_f16_grouped_tn(D, A, o, dw[E:2 * E])
        torch.cuda.synchronize()
        for t in (whole, back):
            v = t.view(torch.int16)
            assert (v[:T] == SENTINEL).all() and (v[2 * T:] == SENTINEL).all()
        assert (dw[:E] == 7).all() and (dw[2 * E:] == 7).all()


@pytest.mark.parametrize("sizes,N,K", [((3, 5, 2), 72, 512), ((3, 5, 2), 72, 264), ((20, 1, 33), 136, 512),
                                       ((70, 45, 90), 264, 328), ((70, 45, 90), 264, 512), ((70, 45, 90), 261, 77)])
def test_other_groups_infinities_and_nan_stay_there(sizes, N, K):
    """The rows of every group but the middle one, and its weights, are infinite or NaN."""
    E, T, off = len(sizes), sum(sizes), plain.offsets_of(sizes)
    A, B, D = _half(4, T, K), _half(5, E, N, K, scale=0.05), _half(6, T, N)
    r = slice(int(off[1]), int(off[2]))
    a, b, d = A[r].clone(), B[1].clone(), D[r].clone()
    for t in (A, D):
        t[:] = float("nan")
        t[::2] = float("inf")
    B[0], B[2] = float("inf"), float("nan")
    A[r], B[1], D[r] = a, b, d
    o = dev(off)
    _say("isolated", sizes, N, K)
    C, dA, dB = gf.gemm_f16_grouped_nt(A, B, o), gf.gemm_f16_grouped_nn(D, B, o), gf.gemm_f16_grouped_tn(D, A, o)

    def check(got, x, y, depth, what, extra=0.0):
        x, y = x.double(), y.double().contiguous()
        absum = x.abs() @ y.abs()
        plain.check(got.cpu().numpy(), (x @ y).cpu().numpy(), absum.cpu().numpy(), depth, plain.F16, what, extra)

    check(C[r], a, b.t(), K, "nt")
    check(dA[r], d, b, N, "nn")
    check(dB[1], d.t().contiguous(), a, sizes[1], "tn")
    if K % 8 == 0:
        for group in (32, 64, 128):
            Q, S, Z = gf.w4_quantize_f16(B, group)
            assert torch.isnan(S[0]).all() and torch.isnan(S[2]).all()
            C = gf.gemm_w4_f16_grouped_nt(A, Q, S, Z, o, group=group)
            w = plain.weights(plain.unpack(Q[1].cpu().numpy()), S[1].cpu().numpy(), Z[1].cpu().numpy(), group)
            w = torch.from_numpy(w).cuda()
            extra = plain.rounded_weights((a.double().abs() @ w.abs().t()).cpu().numpy(),
                                          a.double().abs().sum(1, keepdim=True).cpu().numpy())
            check(C[r], a, w.t(), K, "w4", extra)


def test_no_rows_and_no_contraction():
    z = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt, device="cuda")
    o = dev(np.array([0, 0, 0], dtype=np.int32))
    for f32 in (False, True):
        C = torch.full((2, 40, 24), 7.0, dtype=torch.float32 if f32 else torch.float16, device="cuda")
        gf.gemm_f16_grouped_tn(z(0, 40), z(0, 24), o, C)
        assert not C.any() and not torch.signbit(C).any()
    assert gf.gemm_f16_grouped_nt(z(0, 64), z(2, 24, 64), o).shape == (0, 24)
    assert gf.gemm_w4_f16_grouped_nt(z(0, 64), z(2, 24, 8, dt=torch.int32), z(2, 24, 2), None, o, group=32).shape == (0, 24)
    o = dev(np.array([1, 3, 4], dtype=np.int32))
    for T in (5, 300):                                     # groups of no k: rows 1 to 3 are zero, the others untouched
        C = _sentinel((T, 24))
        gf.gemm_w4_f16_grouped_nt(z(T, 0), z(2, 24, 0, dt=torch.int32), z(2, 24, 0), None, o, C, group=32)
        assert not C[1:4].view(torch.int16).any()
        assert (C[:1].view(torch.int16) == SENTINEL).all() and (C[4:].view(torch.int16) == SENTINEL).all()


def _check_groups(C, A, B, off, groups, depth, what):
    for e in groups:
        r = slice(int(off[e]), int(off[e + 1]))
        a, b = A[r].double(), B[e].double().contiguous()
        plain.check(C[r].cpu().numpy(), (a @ b).cpu().numpy(), (a.abs() @ b.abs()).cpu().numpy(), depth, plain.F16,
                    "%s group %d" % (what, e))


def test_as_many_groups_as_may_be():
    """65536 groups of no, one or two rows; sampled groups, the first and the last."""
    E, N, K = 65536, 16, 32
    rng = np.random.default_rng(7)
    off = plain.offsets_of(rng.integers(0, 3, E), 1)
    T = int(off[-1]) + 2
    A, B, D, o = _half(8, T, K), _half(9, E, N, K), _half(10, T, N), dev(off)
    groups = [0, 1, 63, 64, E - 65, E - 64, E - 2, E - 1] + [int(e) for e in rng.integers(0, E, 40)]
    _say("65536 groups")
    C = gf.gemm_f16_grouped_nt(A, B, o, _sentinel((T, N)))
    dA = gf.gemm_f16_grouped_nn(D, B, o, _sentinel((T, K)))
    dB = gf.gemm_f16_grouped_tn(D, A, o)
    torch.cuda.synchronize()
    for t in (C, dA):
        v = t.view(torch.int16)
        assert (v[:1] == SENTINEL).all() and (v[-2:] == SENTINEL).all() and not (v[1:-2] == SENTINEL).all(1).any()
    _check_groups(C, A, B.transpose(1, 2), off, groups, K, "nt")
    _check_groups(dA, D, B, off, groups, N, "nn")
    for e in groups:
        r = slice(int(off[e]), int(off[e + 1]))
        d, a = D[r].double(), A[r].double()
        plain.check(dB[e].cpu().numpy(), (d.t() @ a).cpu().numpy(), (d.abs().t() @ a.abs()).cpu().numpy(),
                    max(1, r.stop - r.start), plain.F16, "tn group %d" % e)
    for group in (32, 128):
        Q, S, Z = gf.w4_quantize_f16(B, group)
        C = gf.gemm_w4_f16_grouped_nt(A, Q, S, Z, o, _sentinel((T, N)), group)
        torch.cuda.synchronize()
        at = torch.tensor(groups, device="cuda")
        q = plain.unpack(Q[at].flatten(0, 1).cpu().numpy())
        W = plain.weights(q, S[at].flatten(0, 1).cpu().numpy(), Z[at].flatten(0, 1).cpu().numpy(), group)
        W = torch.from_numpy(W).cuda().view(len(groups), N, K).transpose(1, 2)
        _check_groups(C, A, dict(zip(groups, W)), off, groups, K, "w4")


@pytest.mark.parametrize("form", ["nt", "nn"])
def test_rounds_of_tiles_over_more_groups_than_lanes(form):
    """The launch in two parts, with the scan over the groups in two passes."""
    E, N, K = 70, 700, 1032
    sizes = np.random.default_rng(11).integers(0, 430, E)
    sizes[[0, 63, 64, 69]] = 257, 1, 0, 400
    sizes[5] += 196 * E - min(int(sizes.sum()), 196 * E)    # a mean of 196 rows at least
    off, T = plain.offsets_of(sizes), int(sizes.sum())
    A, B = _half(12, T, K), _half(13, E, *((N, K) if form == "nt" else (K, N)), scale=0.03)
    _say("rounds", form, T)
    C = (gf.gemm_f16_grouped_nt if form == "nt" else gf.gemm_f16_grouped_nn)(A, B, dev(off), _sentinel((T, N)))
    torch.cuda.synchronize()
    _check_groups(C, A, B.transpose(1, 2) if form == "nt" else B, off, [e for e in range(E) if sizes[e]], K, form)
