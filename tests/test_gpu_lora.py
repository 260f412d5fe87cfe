"""Low-rank adapters beside a shared projection on the GPU against plain 64-bit forms."""
import sys

import numpy as np
import pytest

import gemv_fp16_amd as gf
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
    torch.cuda.synchronize()


def _say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def _shifted(t, elems):
    flat = torch.empty(t.numel() + elems, dtype=t.dtype, device=t.device)
    out = flat[elems:].view(t.shape)
    out.copy_(t)
    return out


def _ids(rng, kind, M, L):
    if kind == "one":
        return np.full(M, L - 1, dtype=np.int32)
    if kind == "none":
        return np.full(M, -1, dtype=np.int32)
    if kind == "runs":                     # requests one after another
        return np.sort(rng.integers(0, L, M)).astype(np.int32)
    ids = rng.integers(0, L, M).astype(np.int32)
    if kind == "stray":                    # a third without an adapter, and ids that are none
        ids[rng.random(M) < 0.3] = -1
        ids[0] = L
        ids[-1] = np.iinfo(np.int32).min
    return ids


class Problem:
    def __init__(self, M, N, K, r, L, kind, seed, scaled=True):
        rng = np.random.default_rng(seed)
        h = lambda s, *shape: (rng.standard_normal(shape) * s).astype(np.float16)
        self.M, self.N, self.K, self.r, self.L = M, N, K, r, L
        self.A, self.B = h(1.0, M, K), h(1.0 / np.sqrt(max(K, 1)), N, K)
        self.Down, self.Up = h(1.0 / np.sqrt(max(K, 1)), L, r, K), h(0.3, L, N, r)
        self.ids = _ids(rng, kind, M, L) if L else np.zeros(M, dtype=np.int32)
        self.scales = (rng.random(L) + 0.5).astype(np.float32) if scaled else None
        self.C0 = h(1.0, M, N)

    def low(self):
        """The adapters' part, the sum of its products' magnitudes, and what
        rounding the product by Down to fp16 can move it by."""
        f = lambda v: v.astype(np.float64)
        out, size, half = (np.zeros((self.M, self.N)) for _ in range(3))
        for a in range(self.L):
            m = np.flatnonzero(self.ids == a)
            if len(m):
                s = float(self.scales[a]) if self.scales is not None else 1.0
                H = s * (f(self.A[m]) @ f(self.Down[a]).T)
                Ha = s * (np.abs(f(self.A[m])) @ np.abs(f(self.Down[a])).T)
                out[m] = H @ f(self.Up[a]).T
                size[m] = Ha @ np.abs(f(self.Up[a])).T
                half[m] = (2.0 ** -11 * np.abs(H) + 2.0 ** -25) @ np.abs(f(self.Up[a])).T
        return out, size, half

    def check(self, C, base, base_size, what):
        """base_size: the sum of the base's products' magnitudes.  Besides the fp32
        sums, one rounding of the result, one of the product by Down and one of the
        base (where it is stored before the adapters are added)."""
        low, size, half = self.low()
        exact = base + low
        err = np.abs(C.cpu().numpy().astype(np.float64) - exact)
        bound = 2.0 ** -11 * (np.abs(exact) * (1 + 2.0 ** -9) + np.abs(base)) + 2.0 ** -24 + half * (1 + 2.0 ** -9) + \
            (self.K + self.r + 16) * 2.0 ** -23 * (base_size + size)
        assert (err <= bound).all(), "%s: worst %.3g times the bound" % (what, float((err / bound).max()))

    def base(self):
        a, b = self.A.astype(np.float64), self.B.astype(np.float64)
        return a @ b.T, np.abs(a) @ np.abs(b).T

    def operands(self, shift=0):
        return [_shifted(dev(v), shift) for v in (self.A, self.B)], dev(self.ids), \
            [_shifted(dev(v), shift) for v in (self.Down, self.Up)], None if self.scales is None else dev(self.scales)


CASES = [(1, 16, 64, 8, 1, "one"), (1, 1, 8, 1, 1, "one"), (1, 520, 1024, 16, 8, "mixed"), (2, 33, 77, 3, 2, "mixed"),
         (4, 1000, 512, 4, 3, "stray"), (16, 264, 2048, 16, 16, "mixed"), (17, 250, 264, 32, 5, "stray"),
         (32, 512, 4096, 64, 24, "mixed"), (33, 72, 1000, 20, 40, "mixed"), (64, 128, 8192, 16, 64, "mixed"),
         (65, 136, 520, 8, 3, "runs"), (100, 300, 128, 256, 2, "mixed"), (130, 256, 512, 16, 6, "runs"),
         (300, 520, 264, 24, 9, "stray"), (520, 264, 1032, 64, 4, "runs"), (700, 384, 256, 16, 500, "mixed"),
         (40, 64, 96, 8, 3, "none"), (8, 48, 0, 8, 2, "mixed"), (1100, 2064, 264, 16, 5, "runs"), (12, 40, 512, 5, 0, "one"),
         (24, 4096, 72, 128, 7, "stray"), (200, 131, 1001, 7, 4, "stray"),
         # 3 to 32 rows, K in slices: ends inside one, ranks past a block, its bounds
         (3, 16, 1544, 8, 2, "mixed"), (16, 1000, 3976, 24, 7, "stray"), (17, 263, 4096, 40, 20, "mixed"),
         (32, 8192, 2048, 16, 1, "one"), (32, 8200, 2056, 16, 3, "runs"), (31, 130, 4104, 16, 4, "mixed"),
         (5, 19, 2048, 256, 4, "none"), (9, 15, 2048, 16, 4, "mixed"), (32, 520, 1536, 16, 32, "mixed"),
         # stored results: 64 columns a wave, and many adapters in 16
         (520, 2100, 520, 72, 4, "runs"), (300, 4096, 264, 40, 300, "mixed"), (32, 66000, 64, 16, 2, "mixed"),
         (1500, 264, 4096, 128, 3, "runs")]


@pytest.mark.parametrize("M,N,K,r,L,kind", CASES)
def test_lora_gemm(M, N, K, r, L, kind):
    p = Problem(M, N, K, r, L, kind, M + N)
    base, size = p.base()
    for shift in (0, 1):
        (A, B), ids, (Down, Up), scales = p.operands(shift)
        _say("lora", M, N, K, r, L, kind, shift)
        C = gf.gemm_f16_nt_lora(A, B, ids, Down, Up, scales)
        p.check(C, base, size, "gemm_f16_nt_lora")


@pytest.mark.parametrize("M,N,K,r,L,kind", CASES)
def test_lora_add(M, N, K, r, L, kind):
    p = Problem(M, N, K, r, L, kind, M + K, scaled=M % 2 == 0)
    for shift in (0, 1):
        (A, B), ids, (Down, Up), scales = p.operands(shift)
        _say("lora add", M, N, K, r, L, kind, shift)
        C = _shifted(dev(p.C0), shift)
        assert gf.lora_add_f16(A, ids, Down, Up, C, scales) is C
        c0 = p.C0.astype(np.float64)
        p.check(C, c0, np.abs(c0), "lora_add_f16")
        dead = (p.ids < 0) | (p.ids >= L)
        assert np.array_equal(C.cpu().view(torch.int16).numpy()[dead], p.C0.view(np.int16)[dead])


def test_lora_add_wide_with_a_long_contraction():
    """Few rows onto many columns, the products by Down in more parts than a tile takes."""
    M, N, K, r, L = 20, 66000, 2560, 8, 2
    p = Problem(M, N, 8, r, L, "mixed", 3)
    q = Problem(M, 16, K, r, L, "mixed", 4)
    p.K, p.A, p.Down = K, q.A, q.Down
    C = dev(p.C0)
    _say("lora add", M, N, K, r, L)
    gf.lora_add_f16(dev(p.A), dev(p.ids), dev(p.Down), dev(p.Up), C, dev(p.scales))
    c0 = p.C0.astype(np.float64)
    p.check(C, c0, np.abs(c0), "lora_add_f16")


def test_rows_without_an_adapter_are_the_plain_product():
    """NaN and infinity in adapters that no row has, and in rows that have none, stay there."""
    for M, K in ((3, 512), (11, 2048), (40, 512), (300, 512)):
        p = Problem(M, 264, K, 16, 4, "stray", M)
        p.ids[p.ids == 2] = -1
        p.Down[2], p.Up[2] = np.nan, np.inf
        row = int(np.flatnonzero((p.ids < 0) | (p.ids >= 4))[0])
        keep = np.arange(M) != row
        p.A[row, 5] = np.nan
        (A, B), ids, (Down, Up), scales = p.operands()
        _say("lora nan", M)
        C = gf.gemm_f16_nt_lora(A, B, ids, Down, Up, scales)
        got = C.cpu().numpy()
        assert np.isnan(got[row]).all() and np.isfinite(got[keep]).all()
        p.A[row], p.Down[2], p.Up[2] = 0, 0, 0
        base, size = p.base()
        C[row] = 0
        p.check(C, base, size, "finite rows")


@pytest.mark.parametrize("M,K", [(2, 1024), (12, 1024), (12, 2048), (30, 1024), (30, 2048), (50, 1024), (100, 1024),
                                 (300, 1024), (600, 1024)])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_an_adapter_that_is_not_finite_stays_in_its_rows(M, K, bad):
    """NaN and infinity in one adapter reach the rows that have it and no others, whichever share a tile with them."""
    for add in (False, True):
        p = Problem(M, 520, K, 16, 4, "mixed", M + 1)
        p.ids[:] = np.random.default_rng(M).choice([0, 2, 3, -1], M)
        p.ids[M // 2] = 1
        p.Up[1, ::3, 5] = bad
        p.Down[1, 7, 9] = bad
        (A, B), ids, (Down, Up), scales = p.operands()
        _say("lora not finite", M, K, bad, add)
        if add:
            C = gf.lora_add_f16(A, ids, Down, Up, dev(p.C0), scales)
            base, size = p.C0.astype(np.float64), np.abs(p.C0.astype(np.float64))
        else:
            C = gf.gemm_f16_nt_lora(A, B, ids, Down, Up, scales)
            base, size = p.base()
        got = C.cpu().numpy()
        assert not np.isfinite(got[M // 2]).any()
        p.Up[1], p.Down[1] = 0, 0
        C[M // 2] = dev(base[M // 2].astype(np.float16))
        p.check(C, base, size, "the other rows")


@pytest.mark.parametrize("M", [1, 24, 100])
def test_beside_4_bit_and_sparse_weights(M):
    p = Problem(M, 256, 512, 16, 5, "mixed", M)
    (A, B), ids, (Down, Up), scales = p.operands()
    Q, S, Z = gf.w4_quantize_f16(B, 64)
    sp, meta = gf.sp24_compress_f16(A)
    for C in (gf.gemm_w4_f16_nt(A, Q, S, Z, group=64), gf.gemm_sp_f16_nt(sp, meta, B)):
        before = C.cpu().numpy().astype(np.float64)
        gf.lora_add_f16(A, ids, Down, Up, C, scales)
        p.check(C, before, np.abs(before), "beside other weights")


def test_adapters_past_2_31_elements():
    """Many adapters, Down past 2^31 elements in all: the last ones are read at their place."""
    L, r, K, N, M = 70000, 8, 4096, 16, 5
    Down = torch.zeros((L, r, K), dtype=torch.float16, device="cuda")
    Up = torch.zeros((L, N, r), dtype=torch.float16, device="cuda")
    p = Problem(M, N, K, r, 3, "mixed", 1)
    for i, a in enumerate((0, L - 1, L // 2 + 40)):
        Down[a], Up[a] = dev(p.Down[i]), dev(p.Up[i])
    ids = dev(np.array([0, L - 1, L // 2 + 40], dtype=np.int32)[p.ids])
    scales = torch.ones(L, device="cuda")
    p.scales = None
    _say("lora", L, r, K)
    C = gf.gemm_f16_nt_lora(dev(p.A), dev(p.B), ids, Down, Up, scales)
    p.check(C, *p.base(), "many adapters")


def test_results_repeat_on_streams_and_in_graphs():
    """Graphs replayed in turn, each with a workspace of its own, a side
    stream and a workspace that held something else: the same bits."""
    graphs, held, problems = [], [], []
    for M, K, kind in ((24, 1024, "mixed"), (20, 2048, "mixed"), (200, 1024, "runs")):
        p = Problem(M, 520, K, 16, 6, kind, M)
        ops = p.operands()
        (A, B), ids, (Down, Up), scales = ops
        want = gf.gemm_f16_nt_lora(A, B, ids, Down, Up, scales)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        need = gf.lora_workspace_bytes(M, 520, K, 16)
        ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        again = gf.gemm_f16_nt_lora(A, B, ids, Down, Up, scales, workspace=ws, stream=side)
        side.synchronize()
        assert torch.equal(want, again) and (ws[need:] == 255).all()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            C = gf.gemm_f16_nt_lora(A, B, ids, Down, Up, scales)
            gf.lora_add_f16(A, ids, Down, Up, C, scales)
        graphs.append(graph)
        held.append(C)
        problems.append(ops)
    for i in range(3):
        for graph, C, ((A, B), ids, (Down, Up), scales) in zip(graphs, held, problems):
            _say("lora graph", i)
            A.copy_(torch.randn(A.shape, device="cuda").half())
            want = gf.gemm_f16_nt_lora(A, B, ids, Down, Up, scales)
            gf.lora_add_f16(A, ids, Down, Up, want, scales)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(C, want)
