"""Infinities in an adapter come out as the formula has them, in every form: an infinity times
a number is one, times zero a NaN, and ranks that are not there add nothing."""
import sys

import numpy as np
import pytest

import gemv_fp16_amd as gf
from tests.lora_plain import Integers
from tests.util import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

# vectors, K in slices, streaming (with and without a launch for the products by Down), parts,
# tiles, ranks that end inside a step of 16 or 32, general forms
CASES = [(2, 264, 1024, 16, 3), (1, 130, 4096, 128, 3), (8, 264, 2048, 16, 3), (20, 130, 4096, 40, 3), (8, 264, 1024, 8, 1),
         (9, 264, 1024, 16, 1), (30, 130, 1024, 24, 3), (8, 130, 1024, 72, 3), (40, 264, 1024, 8, 3), (50, 130, 520, 40, 3),
         (100, 264, 1024, 8, 3), (300, 264, 512, 24, 3), (130, 264, 264, 16, 1), (300, 2100, 264, 8, 1), (520, 4100, 264, 16, 3),
         (40, 130, 264, 4, 3), (7, 100, 1001, 5, 3)]


def _expected(p, Down, Up):
    out = p.base.copy()
    with np.errstate(invalid="ignore", over="ignore"):
        for e in range(p.L):
            m = np.flatnonzero(p.ids == e)
            if not len(m):
                continue
            H = np.zeros((len(m), p.r))
            for j in range(p.r):
                H[:, j] = (p.A[m].astype(np.float64) * Down[e, j].astype(np.float64)).sum(1) * p.scales[e]
            low = np.zeros((len(m), p.N))
            for j in range(p.r):
                low += H[:, j, None] * Up[e, :, j].astype(np.float64)
            out[m] = p.base[m] + low
        return out.astype(np.float16)


@pytest.mark.parametrize("M,N,K,r,L", CASES)
@pytest.mark.parametrize("where", ["Down", "Up", "last ranks", "every Up"])
def test_infinities(M, N, K, r, L, where):
    p = Integers(M, N, K, r, L, M + K + r)
    p.ids[M // 2] = L - 1
    Down, Up, e = p.Down.copy(), p.Up.copy(), L - 1
    if where == "Down":
        Down[e, r // 3, K // 2] = np.inf
        Down[e, r - 1, K - 1] = -np.inf
    elif where == "last ranks":                    # finite products elsewhere, Up without zeros
        Down[e, max(0, r - 8):, K // 3] = np.inf
        Up[e] = np.where(Up[e] == 0, np.float16(1), Up[e])
    elif where == "Up":
        Up[e, ::3, r - 1] = np.inf
        Up[e, 1::3, r // 2] = -np.inf
    else:
        Up[e] = np.inf
    want = _expected(p, Down, Up)
    assert not np.isfinite(want).all()
    A, B, dDown, dUp, scales, ids = (dev(v) for v in (p.A, p.B, Down, Up, p.scales, p.ids))
    print("lora infinities", M, N, K, r, L, where, flush=True)
    sys.stdout.flush()
    outs = [gf.gemm_f16_nt_lora(A, B, ids, dDown, dUp, scales),
            gf.lora_add_f16(A, ids, dDown, dUp, dev(p.base.astype(np.float32)), scales)]
    for got in outs:
        got = got.cpu().numpy()
        bad = ~((got == want) | (np.isnan(got) & np.isnan(want)))
        assert not bad.any(), "%d of %d differ, first at %s: %s, not %s" % (
            bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], want[bad][0])
