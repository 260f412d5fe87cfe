"""Low-rank adapters on integers: problems whose sums are exact in fp32 whatever their
order, so that a result is right in every bit or wrong."""
import numpy as np


class Integers:
    """A (M, K), B (N, K), Down (L, r, K), Up (L, N, r) of small integers, and their
    products.  The base and the products by Down have more bits than fp16; every sum
    of magnitudes stays below 2^24 units, so that no order of additions rounds.

    far: pairs of powers of two, one for each adapter in turn: its scale, and the unit of
    its Up; the base is 0 then.  spread: ranks are worth 2^-spread to 1 in Down, and the
    inverse in Up."""

    def __init__(self, M, N, K, r, L, seed, far=None, spread=0, stray=True):
        rng = np.random.default_rng(seed)
        ints = lambda most, *shape: rng.integers(-most, most + 1, shape)
        shrink = min(1.0, np.sqrt(512 / max(K, 1)))
        self.M, self.N, self.K, self.r, self.L = M, N, K, r, L
        a, b = ints(7, M, K), ints(max(1, int(127 * shrink)), N, K)
        down, u = ints(max(1, int(63 * shrink)), L, r, K), ints(1, L, N, r)
        u[rng.random(u.shape) < 1 - min(1.0, 8 / r)] = 0           # about 8 ranks to an output
        self.ids = rng.integers(0, max(L, 1), M).astype(np.int32)
        if stray and M > 2:
            self.ids[rng.random(M) < 0.2] = -1
            self.ids[M // 2] = L
        sign = np.where(rng.random(L) < 0.5, -1, 1)
        scale, up = (np.resize([f[i] for f in far or [(1.0, 1.0)]], L) for i in (0, 1))
        if far:
            b[:] = 0
        worth = 2.0 ** -rng.integers(0, spread + 1, (L, r))
        self.scales = (sign * scale).astype(np.float32)
        self.A, self.B = a.astype(np.float16), b.astype(np.float16)
        exact16 = lambda v: (v.astype(np.float16), (v.astype(np.float16) == v).all())
        self.Down, down_ok = exact16(down * worth[:, :, None])
        self.Up, up_ok = exact16(u * (up[:, None] / worth)[:, None, :])
        assert down_ok and up_ok
        self.base = a.astype(np.float64) @ b.T.astype(np.float64)
        size = np.abs(a).astype(np.float64) @ np.abs(b).T.astype(np.float64)
        self.low, self.H = np.zeros((M, N)), np.zeros((M, r))
        for e in range(L):
            m = np.flatnonzero(self.ids == e)
            if len(m):
                h = a[m].astype(np.float64) @ down[e].T.astype(np.float64)
                assert np.abs(h).max(initial=0) < 2 ** 22
                assert (np.abs(a[m]).astype(np.float64) @ np.abs(down[e]).T).max(initial=0) < 2 ** 24
                unit = scale[e] * up[e]
                self.H[m] = sign[e] * scale[e] * worth[e] * h
                self.low[m] = sign[e] * unit * (h @ u[e].T)
                size[m] += unit * (np.abs(h) @ np.abs(u[e]).T)
                assert size[m].max(initial=0) < 2 ** 24 * unit
        assert far or size.max(initial=0) < 2 ** 24
        self.exact = self.base + self.low

    def once(self, base=None):
        """The result: exact sums, rounded once."""
        with np.errstate(over="ignore"):
            return ((self.base if base is None else base) + self.low).astype(np.float16)

    def twice(self):
        with np.errstate(over="ignore"):
            return (self.base.astype(np.float16).astype(np.float64) + self.low).astype(np.float16)
