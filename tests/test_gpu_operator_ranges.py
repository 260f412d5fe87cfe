"""Grouped and 4-bit products where the launch changes with the sizes, and where
offsets pass 32 bits, against 64-bit forms on the GPU."""
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
    torch.cuda.empty_cache()


def _say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def _half(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=torch.float16, device="cuda")
    return t.normal_(0.0, scale, generator=g)


def _ints(seed, lo, hi, shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").random_(lo, hi, generator=g)


def _shifted(t, elems):
    flat = torch.empty(t.numel() + elems, dtype=t.dtype, device=t.device)
    out = flat[elems:].view(t.shape)
    out.copy_(t)
    return out


def _check(got, a, b, depth, what, kind=plain.F16, rounded=False):
    """got against a . b in float64 (tensors on the GPU)."""
    a, b = a.double(), b.double()
    absum = (a.abs() @ b.abs()).cpu().numpy()
    extra = 0.0
    if rounded:
        extra = plain.rounded_weights(absum, a.abs().sum(1, keepdim=True).cpu().numpy())
    plain.check(got.cpu().numpy(), (a @ b).cpu().numpy(), absum, depth, kind, what, extra)


def _codes(seed, lead, K, group, zeros=True):
    G = plain.groups_of(K, group)
    Q = _ints(seed, -2 ** 31, 2 ** 31 - 1, lead + (K // 8,), torch.int32)
    S = _half(seed + 1, *(lead + (G,)), scale=0.05)
    Z = _ints(seed + 2, 0, 16, lead + (G,), torch.uint8) if zeros else None
    return Q, S, Z


def _weights(Q, S, Z, group):
    """float64 weights (rows, K) of codes (rows, K/8) on the GPU."""
    q = torch.stack([(Q >> (4 * i)) & 15 for i in range(8)], -1).flatten(1).double()
    K = q.shape[1]
    spread = lambda t: t.double().repeat_interleave(group, 1)[:, :K]
    return (q - (8.0 if Z is None else spread(Z))) * spread(S)


# ---- launches of the fp16 products ----------------------------------------

# the last round of 256 x 256 tiles at most half full (308 tiles), fuller (420), one round (224)
@pytest.mark.parametrize("sizes", [(1500, 0, 700, 300), (1800, 0, 1100, 300), (300, 0, 900, 400)])
@pytest.mark.parametrize("form", ["nt", "nn"])
@pytest.mark.parametrize("shift", [0, 1])
def test_rounds_of_tiles(form, sizes, shift):
    T, E, N, K = sum(sizes), len(sizes), 7000, 1032
    off = plain.offsets_of(sizes)
    A = _half(1, T, K)
    B = _half(2, E, *((N, K) if form == "nt" else (K, N)), scale=0.03)
    _say("rounds", form, sizes, shift)
    fn = gf.gemm_f16_grouped_nt if form == "nt" else gf.gemm_f16_grouped_nn
    C = fn(_shifted(A, shift), B, dev(off))
    torch.cuda.synchronize()
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        _check(C[r], A[r], B[e].t().contiguous() if form == "nt" else B[e], K, "group %d" % e)


@pytest.mark.parametrize("group", [0, 32, 64, 128])       # 0: fp16 weights
@pytest.mark.parametrize("N,K", [(200, 1024), (1000, 4096), (90, 512)])
def test_decode_batch_with_most_rows_in_one_group(group, N, K):
    """The streaming forms, chosen by the mean, with several passes of rows."""
    sizes = [1, 0, 53, 1, 1, 0, 0, 2]
    E, T, off = len(sizes), sum(sizes), plain.offsets_of(sizes)
    A = _half(3, T, K)
    _say("skewed", group, N, K)
    if group:
        Q, S, Z = _codes(4, (E, N), K, group)
        C = gf.gemm_w4_f16_grouped_nt(A, Q, S, Z, dev(off), group=group)
        W = [_weights(Q[e], S[e], Z[e], group) for e in range(E)]
    else:
        B = _half(4, E, N, K)
        C = gf.gemm_f16_grouped_nt(A, B, dev(off))
        W = [B[e] for e in range(E)]
    torch.cuda.synchronize()
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if sizes[e]:
            _check(C[r], A[r], W[e].double().t().contiguous(), K, "group %d" % e)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("sizes", [(900, 1, 0, 700), (33, 31, 32, 0), (1, 95, 0, 2)])
def test_weight_gradients_shallow_and_deep(sizes, f32):
    """256 x 256 tiles where the groups are deep, 128 x 128 in 32-row steps else."""
    off, E, T = plain.offsets_of(sizes), len(sizes), sum(sizes)
    A, B = _half(5, T, 2056), _half(6, T, 2048)
    _say("gradients", sizes, f32)
    C = gf.gemm_f16_grouped_tn(A, B, dev(off), out_f32=f32)
    torch.cuda.synchronize()
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        _check(C[e], A[r].t().contiguous(), B[r], sizes[e], "group %d" % e, plain.F32 if f32 else plain.F16)


@pytest.mark.parametrize("sizes,N,K", [((700, 584), 448, 1032), ((90, 0, 200, 110), 300, 2048), ((400, 0, 3, 700), 2309, 200)])
@pytest.mark.parametrize("shift", [0, 1])
def test_groups_of_many_rows_and_few_tiles(sizes, N, K, shift):
    """64 x 64 tiles where 128 x 128 ones are few, and a case with enough of those."""
    T, E, off = sum(sizes), len(sizes), plain.offsets_of(sizes)
    A, B = _half(26, T, K), _half(27, E, N, K, scale=0.03)
    _say("few tiles", sizes, N, K, shift)
    C = gf.gemm_f16_grouped_nt(_shifted(A, shift), B, dev(off))
    torch.cuda.synchronize()
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if sizes[e]:
            _check(C[r], A[r], B[e].t().contiguous(), K, "group %d" % e)


# ---- launches of the 4-bit products ---------------------------------------

# 256 x 256, 128 x 256, 128 x 128, 64 x 128, 32 x 128; the general form; K by windows of 256 and not
@pytest.mark.parametrize("M,N", [(2900, 4100), (1500, 4357), (700, 4000), (100, 8204), (100, 4104), (100, 500)])
@pytest.mark.parametrize("K", [512, 328])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_tiles(M, N, K, group):
    A, (Q, S, Z) = _half(7, M, K), _codes(8, (N,), K, group, zeros=group != 64)
    _say("w4 tiles", M, N, K, group)
    C = gf.gemm_w4_f16_nt(A, Q, S, Z, group=group)
    torch.cuda.synchronize()
    _check(C, A, _weights(Q, S, Z, group).t().contiguous(), K, "tiles", rounded=True)


# the general form, then 32, 64 and 128 rows
@pytest.mark.parametrize("sizes,N", [((40, 0, 33, 31), 333), ((40, 0, 33, 31), 2309), ((150, 1, 99, 0), 2309),
                                     ((400, 0, 130, 257), 2309)])
@pytest.mark.parametrize("K", [512, 328])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_grouped_tiles(sizes, N, K, group):
    E, T, off = len(sizes), sum(sizes), plain.offsets_of(sizes)
    A, (Q, S, Z) = _half(9, T, K), _codes(10, (E, N), K, group, zeros=group != 64)
    _say("w4 grouped tiles", sizes, K, group)
    C = gf.gemm_w4_f16_grouped_nt(A, Q, S, Z, dev(off), group=group)
    torch.cuda.synchronize()
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if sizes[e]:
            W = _weights(Q[e], S[e], None if Z is None else Z[e], group)
            _check(C[r], A[r], W.t().contiguous(), K, "group %d" % e, rounded=True)


@pytest.mark.parametrize("M,N,K", [(m, n, k) for m in (9, 17, 33, 48, 64) for n, k in (
    (17, 512), (1000, 2048), (9000, 4096), (3000, 8192), (300, 1536), (9000, 2008))] +
    [(65, 4096, 2048), (512, 1000, 4096), (300, 500, 8192), (1024, 500, 2048), (700, 16, 4096), (1024, 17, 8192),
     (300, 900, 2008), (1000, 200, 7072)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_passes_of_rows(M, N, K, group):
    """Up to 64 rows, or few blocks of C: passes of 16 and 32 rows in the streaming form, and the general one."""
    A, (Q, S, Z) = _half(20, M, K), _codes(21, (N,), K, group, zeros=group != 32)
    _say("w4 passes", M, N, K, group)
    C = gf.gemm_w4_f16_nt(A, Q, S, Z, group=group)
    torch.cuda.synchronize()
    _check(C, A, _weights(Q, S, Z, group).t().contiguous(), K, "passes")


@pytest.mark.parametrize("sizes", [(10, 12, 0, 15), (40, 0, 33, 31), (1, 99, 0, 2), (200, 0, 300, 77)])
@pytest.mark.parametrize("N,K", [(200, 4096), (700, 8192), (70, 512), (300, 4008)])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_grouped_passes_of_rows(sizes, N, K, group):
    E, T, off = len(sizes), sum(sizes), plain.offsets_of(sizes)
    A, (Q, S, Z) = _half(22, T, K), _codes(23, (E, N), K, group, zeros=group != 64)
    _say("w4 grouped passes", sizes, N, K, group)
    C = gf.gemm_w4_f16_grouped_nt(A, Q, S, Z, dev(off), group=group)
    torch.cuda.synchronize()
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if sizes[e]:
            W = _weights(Q[e], S[e], None if Z is None else Z[e], group)
            _check(C[r], A[r], W.t().contiguous(), K, "group %d" % e, rounded=T > 16 * E)


# ---- offsets past 32 bits -------------------------------------------------

def _columns(N):
    return torch.tensor([0, 1, 15, 16, N // 2 + 3, N - 17, N - 2, N - 1], device="cuda")


@pytest.mark.parametrize("sizes", [(2, 1, 3), (0, 40, 30)])                 # streaming, tiles
def test_grouped_weights_past_32_bits(sizes):
    E, N, K = 3, 250000, 8192                             # 12.3 GB, 4.1 GB a group
    off, T = plain.offsets_of(sizes), sum(sizes)
    A, B, n = _half(11, T, K), _half(12, E, N, K), _columns(N)
    _say("past 32 bits", sizes)
    C = gf.gemm_f16_grouped_nt(A, B, dev(off))
    torch.cuda.synchronize()
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if sizes[e]:
            _check(C[r][:, n], A[r], B[e][n].t().contiguous(), K, "nt group %d" % e)
    D = _half(13, T, K)
    C = gf.gemm_f16_grouped_nn(D, B.view(E, K, N), dev(off))
    torch.cuda.synchronize()
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if sizes[e]:
            _check(C[r][:, n], D[r], B.view(E, K, N)[e][:, n].contiguous(), K, "nn group %d" % e)
    X = _half(14, T, N)
    gf.gemm_f16_grouped_tn(X, A, dev(off), B)             # the gradient over the weights
    torch.cuda.synchronize()
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        _check(B[e][n], X[r][:, n].t().contiguous(), A[r], sizes[e], "tn group %d" % e)


def test_w4_weights_past_32_bits():
    E, N, K, group = 5, 250000, 8192, 64                  # 5.1 GB of codes
    Q, S, Z = _codes(15, (E, N), K, group)
    n = _columns(N)
    for sizes in ((1, 0, 2, 0, 3), (30, 0, 0, 40, 50)):
        off, T = plain.offsets_of(sizes), sum(sizes)
        A = _half(16, T, K)
        _say("w4 past 32 bits", sizes)
        C = gf.gemm_w4_f16_grouped_nt(A, Q, S, Z, dev(off), group=group)
        torch.cuda.synchronize()
        for e in range(E):
            r = slice(int(off[e]), int(off[e + 1]))
            if sizes[e]:
                _check(C[r][:, n], A[r], _weights(Q[e][n], S[e][n], Z[e][n], group).t().contiguous(), K,
                       "group %d" % e, rounded=T > 16 * E)


def test_quantize_past_32_bits():
    N, K, group = 550000, 8192, 128                       # 4.5e9 weights
    W = _half(17, N, K, scale=0.1)
    _say("quantize past 32 bits")
    Q, S, Z = gf.w4_quantize_f16(W, group)
    n = torch.cat([_columns(N), torch.tensor([2 ** 31 // K, 2 ** 32 // K, 2 ** 32 // K - 1], device="cuda")])
    q, s, z = plain.quantize(W[n].cpu().numpy(), group, False)
    assert np.array_equal(plain.unpack(Q[n].cpu().numpy()), q)
    assert np.array_equal(S[n].cpu().numpy(), s) and np.array_equal(Z[n].cpu().numpy(), z)
    back = gf.w4_dequantize_f16(Q, S, Z, group, W=W)
    assert np.array_equal(back[n].cpu().numpy(), plain.weights(q, s, z, group).astype(np.float16))


@pytest.mark.parametrize("T,N,K", [(8000, 250000, 64), (8000, 64, 250000)])  # C, then A, of nearly 2^31 elements
def test_rows_of_nearly_2_to_the_31_elements(T, N, K):
    A, W = _half(18, T, K), _half(19, N, K, scale=0.05)
    _say("large rows", T, N, K)
    rows = torch.tensor([0, 1, 31, 32, 4095, T - 2, T - 1], device="cuda")
    n = _columns(N)
    off = dev(np.array([0, 1, T], dtype=np.int32))
    B = torch.stack([W, W])
    C = gf.gemm_f16_grouped_nt(A, B, off)
    torch.cuda.synchronize()
    _check(C[rows][:, n], A[rows], W[n].t().contiguous(), K, "grouped")
    Q, S, Z = gf.w4_quantize_f16(W, 32)
    C = gf.gemm_w4_f16_nt(A, Q, S, Z, group=32)
    torch.cuda.synchronize()
    _check(C[rows][:, n], A[rows], _weights(Q[n], S[n], Z[n], 32).t().contiguous(), K, "w4", rounded=True)
    C = gf.gemm_w4_f16_grouped_nt(A, torch.stack([Q, Q]), torch.stack([S, S]), torch.stack([Z, Z]), off, group=32)
    torch.cuda.synchronize()
    _check(C[rows][:, n], A[rows], _weights(Q[n], S[n], Z[n], 32).t().contiguous(), K, "w4 grouped", rounded=True)


@pytest.mark.parametrize("f32", [False, True])
def test_weight_gradient_of_nearly_2_to_the_31_elements(f32):
    """A's row offsets pass 2^32 bytes within a group; 128 x 128 tiles in 32-row steps, then 256 x 256."""
    T, M, N = 8000, 250000, 64
    A, B = _half(24, T, M), _half(25, T, N)
    n = _columns(M)
    for ends in ((0, 1, T), tuple(range(0, 8001, 250))):
        off = dev(np.array(ends, dtype=np.int32))
        _say("large gradient", len(ends) - 1, f32)
        C = gf.gemm_f16_grouped_tn(A, B, off, out_f32=f32)
        torch.cuda.synchronize()
        for e in (0, 1, len(ends) - 2):
            r = slice(ends[e], ends[e + 1])
            _check(C[e][n], A[r][:, n].t().contiguous(), B[r], ends[e + 1] - ends[e], "group %d" % e,
                   plain.F32 if f32 else plain.F16)
