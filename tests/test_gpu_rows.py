"""Rows to experts and back on the GPU against plain 64-bit forms, and the whole
expert layer, routed by its own router, with its gradients."""
import sys

import numpy as np
import pytest

import gemv_fp16_amd as gf
from tests import route_plain
from tests import w4_plain as plain
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


def _sentinel(*shape):
    return torch.full(shape, SENTINEL, dtype=torch.int16, device="cuda").view(torch.float16)


def _bits(t):
    return t.cpu().view(torch.int16).numpy()


def _shifted(t, elems):
    flat = torch.empty(t.numel() + elems, dtype=t.dtype, device=t.device)
    out = flat[elems:].view(t.shape)
    out.copy_(t)
    return out


def _f16(rng, *shape):
    return rng.standard_normal(shape).astype(np.float16)


def _place(rng, T, k, R, gone):
    """Different rows for all choices, a share of them none: -1, R and far outside."""
    at = rng.permutation(max(R, T * k))[:T * k].reshape(T, k).astype(np.int32)
    at[at >= R] = -1
    dead = rng.random((T, k)) < gone
    at[dead] = rng.choice([-1, R, 2 ** 31 - 1, -2 ** 31], dead.sum())
    return at


CASES = [(1, 1, 1, 1), (1, 8, 8, 4096), (3, 2, 9, 7), (16, 8, 128, 512), (5, 3, 20, 513), (40, 6, 200, 1000),
         (7, 64, 500, 88), (100, 4, 401, 1001), (33, 5, 165, 2056), (2, 10, 20, 8200), (600, 2, 1200, 260), (4, 2, 0, 16)]


@pytest.mark.parametrize("T,k,R,D", CASES)
@pytest.mark.parametrize("gone", [0.0, 0.3])
def test_dispatch(T, k, R, D, gone):
    rng = np.random.default_rng(T * 7 + D)
    X, at = _f16(rng, T, D), _place(rng, T, k, R, gone)
    for shift in (0, 1):
        _say("dispatch", T, k, R, D, gone, shift)
        A = gf.dispatch_f16(_shifted(dev(X), shift), dev(at), A=_shifted(_sentinel(R, D), shift))
        want = np.full((R, D), SENTINEL, dtype=np.int16)
        for t in range(T):
            for j in range(k):
                if 0 <= at[t, j] < R:
                    want[at[t, j]] = X[t].view(np.int16)
        assert np.array_equal(_bits(A), want)


@pytest.mark.parametrize("T,k,R,D", CASES)
@pytest.mark.parametrize("gone", [0.0, 0.3])
@pytest.mark.parametrize("weighted", [False, True])
def test_combine(T, k, R, D, gone, weighted):
    rng = np.random.default_rng(T * 5 + D)
    C, at = _f16(rng, R, D), _place(rng, T, k, R, gone)
    live = (at >= 0) & (at < R)
    w = rng.standard_normal((T, k)).astype(np.float32)
    w[~live] = np.nan                      # a choice of no row adds nothing, whatever its weight
    w1 = np.where(live, w if weighted else 1.0, 0.0).astype(np.float64)
    rows = np.where(live[:, :, None], C[np.where(live, at, 0)] if R else np.zeros((T, k, D)), 0).astype(np.float64)
    exact = (w1[:, :, None] * rows).sum(1)
    absum = np.abs(w1[:, :, None] * rows).sum(1)
    for shift in (0, 1):
        _say("combine", T, k, R, D, gone, weighted, shift)
        Y = gf.combine_f16(_shifted(dev(C), shift), dev(at), dev(w) if weighted else None,
                           Y=_shifted(_sentinel(T, D), shift))
        plain.check(Y.cpu().numpy(), exact, absum, k, plain.F16, "combine")
    dead = ~live.any(1)
    assert (_bits(Y)[dead] == 0).all()


@pytest.mark.parametrize("T,k,R,D", CASES + [(5, 2, 10, 0)])
@pytest.mark.parametrize("gone", [0.0, 0.3])
def test_combine_gradient(T, k, R, D, gone):
    rng = np.random.default_rng(T * 3 + D)
    dY, C, at = _f16(rng, T, D), _f16(rng, R, D), _place(rng, T, k, R, gone)
    live = (at >= 0) & (at < R)
    w = rng.standard_normal((T, k)).astype(np.float32)
    for shift in (0, 1):
        _say("combine gradient", T, k, R, D, gone, shift)
        dC, dw = gf.combine_f16_bwd(_shifted(dev(dY), shift), _shifted(dev(C), shift), dev(at), dev(w),
                                    dC=_shifted(_sentinel(R, D), shift),
                                    dweights=torch.full((T, k), 7.0, device="cuda"))
        got, bits, gw = dC.cpu().numpy(), _bits(dC), dw.cpu().numpy()
        named = np.zeros(R, dtype=bool)
        for t in range(T):
            for j in range(k):
                if not live[t, j]:
                    assert gw[t, j] == 0
                    continue
                r = at[t, j]
                named[r] = True
                exact = float(w[t, j]) * dY[t].astype(np.float64)
                plain.check(got[r], exact, np.abs(exact), 1, plain.F16, "dC")
                prod = dY[t].astype(np.float64) * C[r].astype(np.float64)
                plain.check(gw[t, j:j + 1], np.array([prod.sum()]), np.array([np.abs(prod).sum()]), D, plain.F32, "dw")
        assert (bits[~named] == SENTINEL).all()


def test_results_repeat_on_streams_and_in_graphs():
    rng = np.random.default_rng(3)
    T, k, D = 50, 4, 520
    at = dev(_place(rng, T, k, T * k, 0.1))
    w = dev(rng.standard_normal((T, k)).astype(np.float32))
    X, dY = dev(_f16(rng, T, D)), dev(_f16(rng, T, D))

    def chain(X, dY):
        A = gf.dispatch_f16(X, at, A=torch.zeros((T * k, D), dtype=torch.float16, device="cuda"))
        Y = gf.combine_f16(A, at, w)
        dC, dw = gf.combine_f16_bwd(dY, A, at, w, dC=torch.zeros((T * k, D), dtype=torch.float16, device="cuda"))
        return A, Y, dC, dw, gf.combine_f16(dC, at)

    side = torch.cuda.Stream()
    want = chain(X, dY)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = chain(X, dY)
    side.synchronize()
    for u, v in zip(want, got):
        assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = chain(X, dY)
    for i in range(3):
        _say("rows graph", i)
        X.copy_(dev(_f16(rng, T, D)))
        dY.copy_(dev(_f16(rng, T, D)))
        eager = [t.clone() for t in chain(X.clone(), dY.clone())]
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(held, eager):
            assert torch.equal(u, v)


def test_a_row_that_two_choices_name():
    """Each entry is one or the other's; the other rows, and each choice's dot product, are as ever."""
    rng = np.random.default_rng(5)
    T, k, D, R = 40, 3, 1100, 130
    X, C = dev(_f16(rng, T, D)), dev(_f16(rng, R, D))
    at = np.arange(T * k, dtype=np.int32).reshape(T, k)
    at[7, 2], at[30, 0] = at[30, 1], at[30, 1]             # of two tokens, and twice of one
    place = dev(at)
    w = torch.ones((T, k), device="cuda")
    _say("rows twice")
    A = gf.dispatch_f16(X, place, A=torch.zeros((R, D), dtype=torch.float16, device="cuda"))
    dC, dw = gf.combine_f16_bwd(X, C, place, w, dC=torch.zeros((R, D), dtype=torch.float16, device="cuda"))
    for got in (A, dC):
        row = int(at[30, 1])
        assert ((got[row] == X[7]) | (got[row] == X[30])).all()
        for t in range(T):
            for r in at[t]:
                assert r == row or torch.equal(got[int(r)], X[t])
    want = (X.double().cpu()[:, None, :] * C.double().cpu()[torch.from_numpy(at).long()]).sum(2)
    # each product exact in fp32; 1100 of them summed, in whatever order
    bound = D * 2.0 ** -23 * (X.double().cpu().abs()[:, None, :] * C.double().cpu().abs()[torch.from_numpy(at).long()]).sum(2)
    assert ((dw.double().cpu() - want).abs() <= bound).all()


def test_elements_near_2_31():
    """Rows whose offset passes 2^30 elements (2^31 bytes), at both ends of the operand."""
    D, R = 8192, 262143                    # R * D = 2^31 - 8192 elements
    at = torch.tensor([[0, R - 1], [R // 2, 1], [R - 2, R]], dtype=torch.int32, device="cuda")
    X = torch.arange(3 * D, device="cuda").view(3, D).remainder(2000).half()
    A = torch.zeros((R, D), dtype=torch.float16, device="cuda")
    _say("dispatch", R, D)
    gf.dispatch_f16(X, at, A=A)
    for t, j in ((0, 0), (0, 1), (1, 0), (1, 1), (2, 0)):
        assert torch.equal(A[at[t, j].item()], X[t])
    Y = gf.combine_f16(A, at)
    assert torch.equal(Y[:2], (2 * X[:2].float()).half()) and torch.equal(Y[2], X[2])
    dw = gf.combine_f16_bwd(X, A, at, torch.ones((3, 2), device="cuda"))[1].double()
    want = (X.double() ** 2).sum(1)
    got = torch.stack([dw[0, 0], dw[0, 1], dw[1, 0], dw[1, 1], dw[2, 0]])
    assert ((got - want[[0, 0, 1, 1, 2]]).abs() <= want[[0, 0, 1, 1, 2]] * (D + 8) * 2.0 ** -24).all()
    assert dw[2, 1] == 0


# (tokens, experts, choices, width in, width inside, share of padding tokens)
@pytest.mark.parametrize("T,E,k,D,F,padding", [(1, 16, 4, 128, 64, 0), (37, 8, 2, 136, 264, 0.2), (700, 32, 6, 256, 128, 0.1)])
def test_expert_layer(T, E, k, D, F, padding):
    """Router, dispatch, the experts' product, combine; then the whole way back."""
    rng = np.random.default_rng(T)
    X, W, R = _f16(rng, T, D), _f16(rng, E, F, D) / np.float16(np.sqrt(D)), _f16(rng, E, D)
    W = W.astype(np.float16)
    x = (X.astype(np.float64) @ R.astype(np.float64).T / np.sqrt(D)).astype(np.float32)
    x[rng.random(T) < padding] = -np.inf
    dY = _f16(rng, T, F)
    opt = dict(score="softmax", renorm=False)
    _say("expert layer", T, E, k)
    dX, dW, dx_in, ddY = dev(X), dev(W), dev(x), dev(dY)
    ids, w, off, at = gf.route_topk(dx_in, k, **opt)
    A = gf.dispatch_f16(dX, at)
    C = gf.gemm_f16_grouped_nt(A, dW, off)
    Y = gf.combine_f16(C, at, w)
    gC, gw = gf.combine_f16_bwd(ddY, C, at, w)
    gA = gf.gemm_f16_grouped_nn(gC, dW, off)
    gW = gf.gemm_f16_grouped_tn(gC, A, off, out_f32=True)
    gX = gf.combine_f16(gA, at)
    gx = gf.route_topk_bwd(dx_in, ids, gw, **opt)
    torch.cuda.synchronize()

    X64, W64, dY64 = (v.astype(np.float64) for v in (X, W, dY))
    y, ya = np.zeros((T, F)), np.zeros((T, F))
    gXr, gXa, gWr, gWa = np.zeros((T, D)), np.zeros((T, D)), np.zeros((E, F, D)), np.zeros((E, F, D))
    gxr, gxa = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        chosen = route_plain.choose(x[t], k, None, "softmax")
        assert list(ids[t].tolist()) == chosen
        ws = route_plain.weights(x[t], chosen, "softmax", False, 1.0)
        dw, dwa = np.zeros(k), np.zeros(k)
        for j, e in enumerate(chosen):
            if e < 0:
                continue
            c, ca = W64[e] @ X64[t], np.abs(W64[e]) @ np.abs(X64[t])
            y[t] += ws[j] * c
            ya[t] += ws[j] * ca
            g = ws[j] * dY64[t]
            gXr[t] += W64[e].T @ g
            gXa[t] += np.abs(W64[e]).T @ np.abs(g)
            gWr[e] += np.outer(g, X64[t])
            gWa[e] += np.abs(np.outer(g, X64[t]))
            dw[j], dwa[j] = dY64[t] @ c, np.abs(dY64[t]) @ ca
        gxr[t] = route_plain.grad(x[t], chosen, dw, "softmax", False, 1.0)
        s = route_plain.scores(x[t], "softmax")
        full = np.zeros(E)
        for j, e in enumerate(chosen):
            if e >= 0:
                full[e] += dwa[j]
        gxa[t] = s * (full + (full * s).sum())
    # C, dC and dA are rounded to fp16 between the calls (half a step each), the weights to fp32
    step = 2.0 ** -11
    for got, ref, size, what in ((Y, y, ya, "Y"), (gX, gXr, gXa, "dX"), (gW, gWr, gWa, "dW"), (gx, gxr, gxa, "dx")):
        got = got.double().cpu().numpy()
        bound = 4 * step * size + (D + F + 3 * k + 300) * 2.0 ** -23 * size + 2.0 ** -22 * (1 + np.sqrt(F))
        err = np.abs(got - ref)
        assert (err <= bound).all(), (what, float((err / bound).max()))
