"""The scaled products by Down far from 1, and ranks of different sizes, in every form: bit
for bit on integers times powers of two."""
import sys

import numpy as np
import pytest

import gemv_fp16_amd as gf
from tests.lora_plain import Integers
from tests.util import dev

torch = pytest.importorskip("torch")

# vectors, K in slices, streaming (with and without a launch for the products by Down), parts,
# tiles of 64 and 128, ranks past a step of 16 and of 32, general forms
CASES = [(2, 520, 1024, 16, 4), (1, 2100, 4096, 128, 3), (8, 520, 2048, 16, 4), (20, 264, 4096, 40, 6), (8, 520, 1024, 8, 1),
         (30, 264, 1024, 24, 5), (8, 264, 1024, 256, 3), (16, 520, 512, 256, 2), (40, 264, 1024, 16, 4), (50, 130, 520, 72, 4),
         (100, 264, 1024, 8, 4), (300, 520, 512, 24, 5), (300, 2100, 512, 16, 3), (520, 4100, 264, 40, 4), (40, 130, 264, 4, 4)]
# (scale, Up's unit): Down's products past fp16's range, below its steps, and near 1
FAR = [(2.0 ** 20, 2.0 ** -20), (2.0 ** -30, 2.0 ** 15), (2.0 ** -14, 2.0 ** 12), (2.0 ** 24, 2.0 ** -24), (1.0, 1.0)]


def _check(p, shift=0):
    A, B, Down, Up, scales, ids = (dev(v) for v in (p.A, p.B, p.Down, p.Up, p.scales, p.ids))
    base = np.random.default_rng(1).integers(-2000, 2000, (p.M, p.N)).astype(np.float16)
    has = (p.ids >= 0) & (p.ids < p.L)
    for name in ("gemm", "add"):
        if name == "gemm":
            got, want = gf.gemm_f16_nt_lora(A, B, ids, Down, Up, scales), p.once()
        else:
            # onto zeros where there is an adapter: the rest stays as it is
            C = np.where(has[:, None], np.float16(0), base)
            got, want = gf.lora_add_f16(A, ids, Down, Up, dev(C), scales), np.where(has[:, None], p.once(), base)
        got = got.cpu().numpy()
        bad = got != want                        # (+0 and -0 are equal)
        assert not bad.any(), "%s: %d of %d differ, first at %s" % (name, bad.sum(), bad.size, np.argwhere(bad)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r,L", CASES)
def test_adapters_of_any_size(M, N, K, r, L):
    for i in range(len(FAR) if L < len(FAR) else 1):
        print("lora far", M, N, K, r, L, FAR[i], flush=True)
        sys.stdout.flush()
        _check(Integers(M, N, K, r, L, M + r + i, far=FAR[i:] + FAR[:i]))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r,L", CASES)
def test_ranks_of_different_sizes(M, N, K, r, L):
    print("lora spread", M, N, K, r, L, flush=True)
    _check(Integers(M, N, K, r, L, M + r, far=[(2.0 ** -12, 1.0), (1.0, 2.0 ** -4)], spread=12))


@pytest.mark.parametrize("scale,up", FAR[:2] + FAR[3:4])
def test_the_problems_need_more_than_unscaled_pairs(scale, up):
    """On the CPU: two fp16 of the values as they are lose these products."""
    p = Integers(40, 264, 1024, 16, 1, 3, far=[(scale, up)])
    with np.errstate(over="ignore", invalid="ignore"):
        hi = p.H.astype(np.float16)
        lo = (p.H - hi.astype(np.float64)).astype(np.float16)
        pair = hi.astype(np.float64) + np.where(np.isfinite(lo), lo, 0).astype(np.float64)
    has = p.ids == 0
    low = pair[has] @ p.Up[0].astype(np.float64).T
    with np.errstate(invalid="ignore"):
        assert (~(low.astype(np.float16) == p.once()[has])).mean() > 0.5
