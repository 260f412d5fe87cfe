"""Every launch of the calls with adapters, on both sides of each rule that chooses one: bit
for bit on integers, with rows of no adapter among them."""
import sys

import numpy as np
import pytest

import gemv_fp16_amd as gf
from tests.lora_plain import Integers
from tests.util import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

CASES = {
    # vectors: 8, 4 and 2 loads in flight, the products by Down in the kernel or before it,
    # one and several groups of columns to a workgroup; what its LDS does not hold
    "vectors": [(1, 2100, 4096, 16, 4), (1, 2100, 4096, 128, 2), (2, 4100, 2056, 16, 2), (2, 4100, 2056, 64, 2),
                (1, 520, 1024, 64, 1), (2, 520, 1536, 72, 1), (2, 33, 8192, 8, 3), (1, 40, 70000, 16, 2), (2, 40000, 512, 256, 2),
                (1, 520, 1024, 72, 1), (1, 520, 2056, 16, 1), (1, 520, 2056, 128, 1), (2, 520, 1024, 16, 2), (2, 520, 4096, 72, 1)],
    # K in slices: 4 and 8 of them, 3 and 32 rows, one and two blocks of rows, ranks past one wave's
    "slices": [(3, 16, 1544, 8, 3), (16, 520, 4096, 64, 5), (17, 8192, 2048, 72, 2), (32, 264, 4096, 256, 3), (5, 1000, 2056, 16, 1)],
    # streaming with one adapter of up to 16 ranks
    "streaming, one adapter": [(8, 520, 1024, 16, 1), (8, 520, 1024, 8, 1), (32, 520, 1024, 16, 1), (9, 8208, 4096, 16, 1),
                               (16, 16, 264, 16, 1), (20, 8200, 2048, 8, 1)],
    # streaming: each depth, and the smaller ring beside many ranks
    "streaming": [(12, 520, 1024, 24, 3), (9, 8208, 4096, 16, 3), (9, 520, 8192, 16, 3), (30, 8200, 1536, 8, 4), (24, 8208, 4096, 16, 3),
                  (16, 520, 512, 256, 2), (16, 264, 8192, 256, 2), (32, 520, 1024, 256, 2), (32, 8200, 4096, 248, 2), (3, 17, 512, 16, 3),
                  (16, 8208, 4096, 256, 2), (32, 8208, 4096, 256, 2)],
    # the base in parts: 33 to 64 rows, long K, few columns, one and several of them
    "parts": [(33, 520, 512, 16, 3), (64, 8200, 1024, 72, 4), (64, 16400, 1024, 16, 4), (17, 264, 4104, 16, 3), (4, 264, 8200, 256, 2),
              (20, 15, 1024, 16, 2)],
    # tiles of 64 x 64, 128 x 128 with four and two stages, 256 x 128 and 256 x 256
    "tiles": [(65, 520, 264, 8, 3), (300, 130, 1024, 72, 2), (1100, 2064, 264, 24, 5), (1100, 2064, 520, 64, 300),
              (2100, 2200, 264, 16, 3), (2100, 2200, 128, 40, 500), (2100, 4100, 2056, 16, 4), (2100, 4104, 2048, 72, 90),
              (4100, 4100, 1544, 16, 4), (4100, 4100, 1544, 8, 2000)],
    # operands, ranks or K of no such form, with many rows
    "general": [(1, 2100, 4096, 4, 4), (70, 4100, 1030, 12, 3), (2100, 4100, 520, 4, 4), (300, 28700, 64, 4, 3), (520, 66000, 64, 4, 3)],
}


@pytest.mark.parametrize("form,M,N,K,r,L", [(f, *c) for f in CASES for c in CASES[f]])
def test_product(form, M, N, K, r, L):
    p = Integers(M, N, K, r, L, M + N + r)
    A, B, Down, Up, scales, ids = (dev(v) for v in (p.A, p.B, p.Down, p.Up, p.scales, p.ids))
    print("lora forms", form, M, N, K, r, L, flush=True)
    sys.stdout.flush()
    want = torch.from_numpy(p.once()).cuda()
    C = gf.gemm_f16_nt_lora(A, B, ids, Down, Up, scales)
    assert torch.equal(C, want), int((C != want).sum())
    if M > 64 and form == "tiles":
        runs = torch.sort(ids).values                # rows of a request together: one adapter to most blocks
        order = torch.argsort(ids, stable=True)
        C = gf.gemm_f16_nt_lora(A[order].contiguous(), B, runs, Down, Up, scales)
        assert torch.equal(C, want[order])


@pytest.mark.parametrize("M,N,K,r,L", [(1, 33, 512, 16, 1), (20, 264, 4096, 16, 4), (20, 264, 1024, 40, 4), (64, 1000, 512, 72, 3),
                                       (20, 66000, 2560, 8, 2), (300, 4100, 512, 16, 3), (600, 8200, 264, 72, 4),
                                       (520, 4100, 264, 40, 300), (9, 100, 1001, 3, 2)])
def test_onto_a_base_in_fp16_and_fp32(M, N, K, r, L):
    """Sixteen columns to 1, 2 and 4 waves, sixty-four to one, with the products by Down in one and several parts."""
    p = Integers(M, N, K, r, L, M + N + r, far=[(1.0, 1.0)])
    A, Down, Up, scales, ids = (dev(v) for v in (p.A, p.Down, p.Up, p.scales, p.ids))
    print("lora add forms", M, N, K, r, L, flush=True)
    base = np.random.default_rng(M).integers(-2000, 2001, (M, N))
    want = torch.from_numpy(p.once(base.astype(np.float64))).cuda()
    got = gf.lora_add_f16(A, ids, Down, Up, dev(base.astype(np.float16)), scales)
    assert torch.equal(got, want), int((got != want).sum())
    got = gf.lora_add_f16(A, ids, Down, Up, dev(base.astype(np.float32)), scales)
    assert torch.equal(got, want), int((got != want).sum())


def test_more_rows_than_workgroups():
    """2^24 rows and some: the products by Down walk more blocks of 16 rows than there are
    workgroups, most of them without an adapter."""
    M, N, K, r, L = 2 ** 24 + 5003, 8, 8, 8, 3
    g = torch.Generator(device="cuda").manual_seed(3)
    ints = lambda most, *shape: torch.randint(-most, most + 1, shape, generator=g, device="cuda").half()
    A, B, Down, Up, base = ints(7, M, K), ints(9, N, K), ints(9, L, r, K), ints(1, L, N, r), ints(900, M, N)
    ids = torch.randint(0, 60, (M,), generator=g, device="cuda").int()         # a twentieth have one
    scales = torch.tensor([1.0, -1.0, 2.0], device="cuda")
    low = torch.zeros((M, N), device="cuda")
    for e in range(L):
        m = torch.where(ids == e)[0]
        low[m] = scales[e] * ((A[m].float() @ Down[e].float().T) @ Up[e].float().T)
    print("lora", M, N, K, r, flush=True)
    C = gf.gemm_f16_nt_lora(A, B, ids, Down, Up, scales)
    assert torch.equal(C, (A.float() @ B.float().T + low).half())
    want = (base.float() + low).half()
    assert torch.equal(gf.lora_add_f16(A, ids, Down, Up, base.float(), scales), want)
    assert torch.equal(gf.lora_add_f16(A, ids, Down, Up, base, scales), want)


@pytest.mark.parametrize("M,N,K,r,L", [(2, 264, 1024, 16, 3), (20, 264, 2048, 16, 3), (20, 264, 1024, 40, 3), (40, 264, 1024, 16, 3),
                                       (100, 264, 1024, 24, 3), (300, 2100, 512, 16, 3)])
@pytest.mark.parametrize("odd", ["A", "B", "Down", "Up", "C", "base"])
def test_one_operand_off_the_16_byte_grid(M, N, K, r, L, odd):
    p = Integers(M, N, K, r, L, M + K)

    def place(name, v):
        t = dev(v)
        if name != odd:
            return t
        flat = torch.empty(t.numel() + 3, dtype=t.dtype, device="cuda")
        flat[3:].copy_(t.view(-1))
        return flat[3:].view(t.shape)
    A, B, Down, Up, base = (place(n, v) for n, v in (("A", p.A), ("B", p.B), ("Down", p.Down), ("Up", p.Up),
                                                     ("base", p.base.astype(np.float32))))
    scales, ids, want = dev(p.scales), dev(p.ids), torch.from_numpy(p.once()).cuda()
    print("lora off the grid", M, N, K, r, L, odd, flush=True)
    for call in (lambda c: gf.gemm_f16_nt_lora(A, B, ids, Down, Up, scales, C=c),
                 lambda c: gf.lora_add_f16(A, ids, Down, Up, base, scales, out=c)):
        C = place("C", np.full((M, N), 7, dtype=np.float16))
        assert torch.equal(call(C), want), int((C != want).sum())
