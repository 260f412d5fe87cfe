"""The scale of a group of 4-bit codes is fp16((hi - lo) / 15), rounded once.

hi - lo can need more bits than fp32 has.  The cases here lie so near a tie
between two scales that what a difference in fp32 loses decides the rounding.
Expected values come from exact fractions."""
from fractions import Fraction

import numpy as np
import pytest

import gemv_fp16_amd as gf
from tests import w4_plain as plain
from tests.util import dev


def nearest_f16(x):
    """The fp16 nearest to a positive fraction in the normal range, ties to even."""
    e = 0
    while x >= Fraction(2) ** (e + 1):
        e += 1
    while x < Fraction(2) ** e:
        e -= 1
    step = Fraction(2) ** (e - 10)
    m = x / step
    f = m.numerator // m.denominator
    r = m - f
    if r > Fraction(1, 2) or (r == Fraction(1, 2) and f % 2):
        f += 1
    return np.float16(float(f * step))


def near_ties(power):
    """(hi, lo) as fp16 with hi - lo at, above and below 15 times a tie t = m 2^(power - 15)
    (m odd, 12 bits) between two scales: 15 t = hi + n 2^(power - 15) with hi in steps of
    2^(power - 10) and n = 1 or 3, where -lo, next to the second part, reaches past the 24
    bits of the sum."""
    pairs, unit = [], 2.0 ** (power - 15)
    for m in range(2185, 4096, 2):
        n = 15 * m % 32
        if n not in (1, 3):
            continue
        hi, r = np.float16((15 * m - n) * unit), np.float16(n * unit)
        assert float(hi) == (15 * m - n) * unit and float(r) == n * unit
        near = [r]
        for way in (np.float16(0), np.float16(np.inf)):
            v = r
            for _ in range(4):
                v = np.nextafter(v, way)
                near.append(v)
        pairs += [(hi, -v) for v in near] + [(v, -hi) for v in near]
    return pairs


def case(power):
    """W (rows, 32), one group a row, and the scales that the definition gives."""
    pairs = near_ties(power)
    W = np.zeros((len(pairs), 32), dtype=np.float16)
    for i, (hi, lo) in enumerate(pairs):
        W[i, i % 29], W[i, i % 29 + 1 + i % 2] = hi, lo
        W[i, 31] = np.float16(float(hi) * 0.3 + float(lo) * 0.4)
    S = np.array([nearest_f16((Fraction(float(hi)) - Fraction(float(lo))) / 15) for hi, lo in pairs], dtype=np.float16)
    return W, S[:, None]


@pytest.mark.parametrize("power", [0, 7, 14])
def test_the_cases_need_more_than_fp32(power):
    """Some of them differ where hi - lo is rounded to fp32 first."""
    W, S = case(power)
    _, S32, _ = plain.quantize(W, 32, False)
    assert (S32 != S).any() and (S32 == S).any()


@pytest.mark.gpu
@pytest.mark.parametrize("power", [0, 7, 14])
def test_scale_is_rounded_once(power):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    W, S = case(power)
    print("scale", power, len(W), flush=True)
    Q, gS, gZ = gf.w4_quantize_f16(dev(W), 32)
    assert np.array_equal(gS.cpu().numpy().view(np.uint16), S.view(np.uint16))
    s, w = S.astype(np.float64), W.astype(np.float64)
    z = np.minimum(np.rint(-w.min(1, keepdims=True) / s), 15)
    assert np.array_equal(gZ.cpu().numpy(), z.astype(np.uint8))
    assert np.array_equal(plain.unpack(Q.cpu().numpy()), np.clip(np.rint(w / s) + z, 0, 15).astype(np.uint8))
