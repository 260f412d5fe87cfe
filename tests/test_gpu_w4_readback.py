"""4-bit products of many rows are the products of the weights read back.

From 65 rows on (a mean of 17 by expert) each weight may be rounded once to fp16
before it is multiplied.  Against float64 on the unrounded weights, the bound has
to allow for every weight's rounding and could hide a wrong product; against the
weights that w4_dequantize_f16 gives (compared bit for bit elsewhere), what is
left are the roundings of the sum and of the result.  Every tile shape, with K by
windows of 256 and step by step, each group size, single and by expert."""
import sys

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
    return torch.empty(shape, dtype=torch.float16, device="cuda").normal_(0.0, scale, generator=g)


def _codes(seed, lead, K, group, zeros):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = lead + (plain.groups_of(K, group),)
    Q = torch.empty(lead + (K // 8,), dtype=torch.int32, device="cuda").random_(-2 ** 31, 2 ** 31 - 1, generator=g)
    S = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(0.0, 0.05, generator=g)
    Z = torch.empty(shape, dtype=torch.uint8, device="cuda").random_(0, 16, generator=g) if zeros else None
    return Q, S, Z


def _check(got, a, back, what):
    """got against a . back^T in float64: no allowance for the weights."""
    a, b = a.double(), back.double().t().contiguous()
    plain.check(got.cpu().numpy(), (a @ b).cpu().numpy(), (a.abs() @ b.abs()).cpu().numpy(), a.shape[1], plain.F16, what)


# tiles of 256 x 256, 128 x 256, 128 x 128, 64 x 128 and 32 x 128
@pytest.mark.parametrize("M,N", [(2900, 4100), (1500, 4357), (700, 4000), (100, 8204), (100, 4104)])
@pytest.mark.parametrize("K", [512, 1792, 328, 1352])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_tiles(M, N, K, group):
    A, (Q, S, Z) = _half(M, M, K), _codes(K, (N,), K, group, zeros=group != 64)
    _say("read back", M, N, K, group)
    C = gf.gemm_w4_f16_nt(A, Q, S, Z, group=group)
    _check(C, A, gf.w4_dequantize_f16(Q, S, Z, group), "tiles")


# tiles of 32, 64 and 128 rows
@pytest.mark.parametrize("sizes", [(40, 0, 33, 31), (150, 1, 99, 0), (400, 0, 130, 257)])
@pytest.mark.parametrize("K", [512, 1792, 328, 1352])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_grouped_tiles(sizes, K, group):
    E, T, N, off = len(sizes), sum(sizes), 2309, plain.offsets_of(sizes)
    A, (Q, S, Z) = _half(T, T, K), _codes(K, (E, N), K, group, zeros=group != 64)
    _say("read back by expert", sizes, K, group)
    C = gf.gemm_w4_f16_grouped_nt(A, Q, S, Z, dev(off), group=group)
    back = gf.w4_dequantize_f16(Q, S, Z, group)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if sizes[e]:
            _check(C[r], A[r], back[e], "group %d" % e)
