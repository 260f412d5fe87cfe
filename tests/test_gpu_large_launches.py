"""Products within the documented sizes that take more workgroups than one
launch may have (fewer than 2^32 threads).  Whole numbers throughout, so every
output is compared exactly."""
import sys

import pytest

import gemv_fp16_amd as gf

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

CHUNK = 1 << 24


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


def _whole(seed, n):
    """n whole numbers from -4 to 4 as fp16."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-4, 5, (n,), generator=g, device="cuda", dtype=torch.int8).half()


def _filled(*shape):
    return torch.full(shape, 99.0, dtype=torch.float16, device="cuda")


def test_one_token_by_2_to_the_28_rows_of_codes():
    N, K = 2 ** 28 - 1, 8
    g = torch.Generator(device="cuda").manual_seed(1)
    Q = torch.randint(-2 ** 31, 2 ** 31 - 1, (N, 1), generator=g, device="cuda", dtype=torch.int32)
    S = torch.ones((N, 1), dtype=torch.float16, device="cuda")
    x, y = _whole(2, K), _filled(N)
    _say("gemv", N)
    gf.gemv_w4_f16(Q, S, None, x, y, group=32)
    torch.cuda.synchronize()
    shift = torch.arange(0, 32, 4, device="cuda", dtype=torch.int32)
    for at in range(0, N, CHUNK):
        q = ((Q[at:at + CHUNK] >> shift) & 15).float() - 8
        assert torch.equal(y[at:at + CHUNK], (q * x.float()).sum(1).half()), at


def test_2_to_the_27_rows_by_one_row_of_codes():
    M, K = 2 ** 27 + 16, 8
    A = _whole(3, M * K).view(M, K)
    Q = torch.tensor([[0x7b3a9c15]], dtype=torch.int32, device="cuda")
    S, C = torch.ones((1, 1), dtype=torch.float16, device="cuda"), _filled(M, 1)
    _say("gemm", M)
    gf.gemm_w4_f16_nt(A, Q, S, None, C, group=32)
    torch.cuda.synchronize()
    w = torch.tensor([((0x7b3a9c15 >> (4 * i)) & 15) - 8 for i in range(8)], device="cuda").float()
    for at in range(0, M, CHUNK):
        assert torch.equal(C[at:at + CHUNK, 0], (A[at:at + CHUNK].float() * w).sum(1).half()), at


def test_grouped_row_by_2_to_the_30_columns():
    N = 2 ** 30
    B, C = _whole(4, N), _filled(1, N)
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    A = torch.full((1, 1), 3.0, dtype=torch.float16, device="cuda")
    _say("grouped nt", N)
    gf.gemm_f16_grouped_nt(A, B.view(1, N, 1), off, C)
    torch.cuda.synchronize()
    assert torch.equal(C[0], B * 3)


def test_grouped_gradient_of_2_to_the_30_rows():
    """Two groups, the first of them empty: its gradient is zero."""
    M = 2 ** 30
    A, C = _whole(5, M).view(1, M), _filled(2, M, 1)
    off = torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda")
    B = torch.full((1, 1), -5.0, dtype=torch.float16, device="cuda")
    _say("grouped tn", M)
    gf.gemm_f16_grouped_tn(A, B, off, C)
    torch.cuda.synchronize()
    assert not C[0].any()
    assert torch.equal(C[1, :, 0], A[0] * -5)
