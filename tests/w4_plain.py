"""Plain 64-bit forms of the 4-bit weight and grouped products, for the tests."""
import numpy as np


def groups_of(K, group):
    return (K + group - 1) // group


def pack(q):
    """(rows, K) codes -> (rows, K/8) int32 words, lowest k in the lowest bits."""
    q = np.asarray(q, dtype=np.uint32)
    w = np.zeros((q.shape[0], q.shape[1] // 8), dtype=np.uint32)
    for i in range(8):
        w |= q[:, i::8] << np.uint32(4 * i)
    return w.view(np.int32)


def unpack(words):
    w = np.ascontiguousarray(words).view(np.uint32)
    q = np.empty((w.shape[0], w.shape[1] * 8), dtype=np.uint8)
    for i in range(8):
        q[:, i::8] = (w >> np.uint32(4 * i)) & np.uint32(15)
    return q


def weights(q, S, Z, group):
    """The float64 weights that codes (rows, K), scales and zero points stand for."""
    K = q.shape[1]
    s = np.repeat(S.astype(np.float64), group, axis=1)[:, :K]
    z = 8.0 if Z is None else np.repeat(Z.astype(np.float64), group, axis=1)[:, :K]
    return (q.astype(np.float64) - z) * s


def quantize(W, group, symmetric):
    """(q, S, Z) of fp16 W by the definition, quotients in float64 (exact at
    every tie: a tie k + 1/2 and a quotient of two 11-bit numbers that is not
    one differ by far more than a float64 rounding)."""
    N, K = W.shape
    G = groups_of(K, group)
    q = np.empty((N, K), dtype=np.uint8)
    S = np.empty((N, G), dtype=np.float16)
    Z = np.empty((N, G), dtype=np.uint8)
    for g in range(G):
        w = W[:, g * group:(g + 1) * group].astype(np.float64)
        bad = ~np.isfinite(w).all(axis=1)
        with np.errstate(all="ignore"):
            w = np.where(bad[:, None], 0.0, w)
            lo, hi = np.minimum(w.min(1), 0.0), np.maximum(w.max(1), 0.0)
            if symmetric:
                s = (np.abs(w).max(1).astype(np.float32) / np.float32(7)).astype(np.float16)     # +0 where all are zero
            else:
                s = ((hi.astype(np.float32) - lo.astype(np.float32)) / np.float32(15)).astype(np.float16)
            s64 = s.astype(np.float64)
            flat = (s64 == 0) | bad
            d = np.where(flat, 1.0, s64)
            z = np.full(N, 8.0) if symmetric else np.where(flat, 0.0, np.minimum(np.rint(-lo / d), 15))
            c = np.clip(np.rint(w / d[:, None]) + z[:, None], 0, 15)
        q[:, g * group:(g + 1) * group] = np.where(flat[:, None], z[:, None], c).astype(np.uint8)
        S[:, g] = np.where(bad, np.float16("nan"), s)
        Z[:, g] = z.astype(np.uint8)
    return q, S, None if symmetric else Z


def bound(exact, absum, depth, eps_half, tiny):
    """How far a result may be: half a step of its type (relative eps_half, or
    half the smallest subnormal), and depth + 8 fp32 roundings of partial sums
    that are at most the sum of the products' magnitudes."""
    return eps_half * np.abs(exact) * (1 + 2.0 ** -10) + tiny + (depth + 8) * 2.0 ** -24 * absum


F16 = dict(eps_half=2.0 ** -11, tiny=2.0 ** -25)
F32 = dict(eps_half=2.0 ** -24, tiny=0.0)


def rounded_weights(absum, a_abs):
    """How far a product may be where each weight is first rounded to fp16: half
    a step of it, relative 2^-11 or absolute 2^-25 below the normal range, times
    the magnitude of its entry of A.  absum: sums of |a w|; a_abs: row sums of |a|."""
    return 2.0 ** -11 * absum + 2.0 ** -25 * a_abs


def check(got, exact, absum, depth, kind, what="", extra=0.0):
    """Compare with the float64 result; infinities and NaN must be the same.
    extra: what the operands themselves may be off (rounded_weights), which the
    result's own rounding then sees too."""
    got = np.asarray(got).astype(np.float64)
    assert got.shape == exact.shape, what
    fin = np.isfinite(exact)
    assert np.array_equal(np.isnan(got), np.isnan(exact)), what + ": NaN differ"
    inf = np.isinf(exact)
    assert np.array_equal(got[inf], exact[inf]), what + ": infinities differ"
    err = np.abs(got[fin] - exact[fin])
    lim = bound(exact[fin], absum[fin], depth, **kind)
    if not np.isscalar(extra):
        lim = lim + extra[fin] * (1 + kind["eps_half"])
    bad = ~(err <= lim)
    assert not bad.any(), "%s: %d of %d entries out of bounds, worst %.3g times the bound" % (
        what, int(bad.sum()), bad.size, float((err / lim).max()))


def offsets_of(sizes, first=0):
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)
