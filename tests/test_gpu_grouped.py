"""Products grouped by expert on the GPU against plain 64-bit forms."""
import sys

import numpy as np
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
    torch.cuda.synchronize()


def _say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def _f16(rng, shape, scale=1.0):
    return (rng.standard_normal(shape) * scale).astype(np.float16)


def _shifted(t, elems):
    flat = torch.empty(t.numel() + elems, dtype=t.dtype, device=t.device)
    out = flat[elems:].view(t.shape)
    out.copy_(t)
    return out


# (sizes of the groups, rows before the first and behind the last)
ROUTES = {
    "one": ([1], 0, 0),
    "token": ([0, 0, 1, 0, 0, 0, 0, 0], 0, 0),
    "few": ([3, 0, 1, 2, 5, 0], 2, 3),
    "mid": ([70, 1, 0, 129, 64], 0, 5),
    "many": ([int(v) for v in np.random.default_rng(1).integers(0, 9, 150)], 1, 1),
    "sixty-four": ([2] * 64, 0, 0),
    "sixty-five": ([1] * 64 + [7], 0, 0),
    "big": ([700, 0, 900, 448], 0, 10),
    "none": ([0, 0, 0], 0, 4),
}
CASES = [("one", 40, 72), ("token", 136, 264), ("few", 200, 520), ("few", 33, 77), ("mid", 264, 136),
         ("mid", 129, 65), ("many", 72, 104), ("sixty-four", 48, 64), ("sixty-five", 16, 24), ("big", 4104, 72),
         ("none", 64, 64), ("few", 64, 0), ("few", 8, 8), ("few", 1, 3), ("few", 16, 2048), ("few", 1000, 3000),
         ("token", 72, 8000), ("many", 40, 4096), ("sixty-four", 24, 8192), ("one", 17, 8), ("few", 100, 9000)]


def _route(name):
    sizes, before, behind = ROUTES[name]
    off = plain.offsets_of(sizes, before)
    return sizes, off, int(off[-1]) + behind


def _rows(off, e):
    return slice(int(off[e]), int(off[e + 1]))


SENTINEL = 0x3A55


def _sentinel(shape):
    return torch.full(shape, SENTINEL, dtype=torch.int16, device="cuda").view(torch.float16)


def _check_rows(C, A, B, off, T, depth, what, transpose, rounded=False):
    """Rows of the groups against float64, the others untouched."""
    bits = C.cpu().view(torch.int16).numpy()
    got = C.cpu().numpy()
    a, seen = A.astype(np.float64), np.zeros(T, dtype=bool)
    for e in range(len(off) - 1):
        r = _rows(off, e)
        seen[r] = True
        b = B[e].astype(np.float64)
        b = b.T if transpose else b
        absum = np.abs(a[r]) @ np.abs(b)
        # 4-bit weights are rounded to fp16 first where the groups have more than 16 rows on average
        extra = plain.rounded_weights(absum, np.abs(a[r]).sum(1, keepdims=True)) if rounded else 0.0
        plain.check(got[r], a[r] @ b, absum, depth, plain.F16, "%s group %d" % (what, e), extra)
    assert (bits[~seen] == SENTINEL).all(), what + ": rows of no group changed"


@pytest.mark.parametrize("route,N,K", CASES)
@pytest.mark.parametrize("form", ["nt", "nn"])
def test_grouped_rows(form, route, N, K):
    sizes, off, T = _route(route)
    E = len(sizes)
    rng = np.random.default_rng(N * 7 + K)
    A = _f16(rng, (T, K))
    B = _f16(rng, (E, N, K) if form == "nt" else (E, K, N))
    _say("grouped", form, route, N, K)
    fn = gf.gemm_f16_grouped_nt if form == "nt" else gf.gemm_f16_grouped_nn
    for shift in ((0, 1) if T < 1000 else (0,)):
        C = fn(_shifted(dev(A), shift), _shifted(dev(B), shift), dev(off), _sentinel((T, N)))
        torch.cuda.synchronize()
        _check_rows(C, A, B, off, T, K, form, form == "nt")


@pytest.mark.parametrize("route,N,K", CASES)
@pytest.mark.parametrize("f32", [False, True])
def test_grouped_tn(f32, route, N, K):
    if K == 0:
        K = 16
    sizes, off, T = _route(route)
    E = len(sizes)
    rng = np.random.default_rng(N * 3 + K)
    A, B = _f16(rng, (T, N)), _f16(rng, (T, K))
    _say("grouped tn", route, N, K, f32)
    for shift in ((0, 1) if T < 1000 else (0,)):
        C = gf.gemm_f16_grouped_tn(_shifted(dev(A), shift), _shifted(dev(B), shift), dev(off), out_f32=f32)
        assert C.dtype == (torch.float32 if f32 else torch.float16)
        got = C.cpu().numpy()
        for e in range(E):
            r = _rows(off, e)
            a, b = A[r].astype(np.float64), B[r].astype(np.float64)
            plain.check(got[e], a.T @ b, np.abs(a).T @ np.abs(b), sizes[e], plain.F32 if f32 else plain.F16,
                        "tn group %d" % e)
            if sizes[e] == 0:
                assert not got[e].any() and not np.signbit(got[e]).any()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("route,N,K", [("one", 40, 72), ("token", 136, 264), ("few", 200, 512), ("few", 33, 136),
                                       ("mid", 136, 256), ("many", 40, 96), ("sixty-five", 16, 32),
                                       ("big", 264, 160), ("big", 3000, 96), ("none", 16, 32), ("few", 200, 1024),
                                       ("few", 33, 4608), ("many", 40, 512), ("token", 100, 8192),
                                       ("mid", 70, 264), ("big", 264, 168), ("sixty-four", 40, 1024)])
def test_w4_grouped(route, N, K, group, zeros):
    sizes, off, T = _route(route)
    E, G = len(sizes), plain.groups_of(K, group)
    rng = np.random.default_rng(N + K + group)
    q = rng.integers(0, 16, (E * N, K)).astype(np.uint8)
    S = (rng.uniform(0.5, 1.5, (E * N, G)) * 2.0 ** rng.integers(-8, 0, (E * N, G))).astype(np.float16)
    Z = rng.integers(0, 16, (E * N, G)).astype(np.uint8) if zeros else None
    A = _f16(rng, (T, K))
    _say("w4 grouped", route, N, K, group, zeros)
    Q3 = dev(plain.pack(q)).view(E, N, K // 8)
    S3, Z3 = dev(S).view(E, N, G), None if Z is None else dev(Z).view(E, N, G)
    W = plain.weights(q, S, Z, group).reshape(E, N, K)
    for shift in (0, 1):
        C = gf.gemm_w4_f16_grouped_nt(_shifted(dev(A), shift), Q3, S3, Z3, dev(off), _sentinel((T, N)), group)
        torch.cuda.synchronize()
        _check_rows(C, A, W, off, T, K, "w4", True, T > 16 * E)


def test_grouped_same_as_one_product():
    """A single group that holds every row is the plain product, bit for bit
    where both run the same products in the same order."""
    rng = np.random.default_rng(3)
    A, B = dev(_f16(rng, (300, 512))), dev(_f16(rng, (1, 264, 512)))
    off = dev(np.array([0, 300], dtype=np.int32))
    assert torch.equal(gf.gemm_f16_grouped_nt(A, B, off), gf.gemm_f16_nt(A, B[0]))


def test_gradients_against_differences():
    """dA and dB of L = sum dC * C against central differences of the 64-bit
    product along random directions.  L is linear in A and in B, so the
    difference is the derivative but for float64 rounding."""
    rng = np.random.default_rng(8)
    sizes, off, T = _route("mid")
    E, N, K = len(sizes), 72, 136
    A, B, dC = _f16(rng, (T, K)), _f16(rng, (E, N, K)), _f16(rng, (T, N))

    def loss(a, b):
        return sum(float((dC[_rows(off, e)].astype(np.float64) * (a[_rows(off, e)] @ b[e].T)).sum())
                   for e in range(E))

    dA = gf.gemm_f16_grouped_nn(dev(dC), dev(B), dev(off), _sentinel((T, K))).cpu().numpy().astype(np.float64)
    dB = gf.gemm_f16_grouped_tn(dev(dC), dev(A), dev(off), out_f32=True).cpu().numpy().astype(np.float64)
    a, b, h = A.astype(np.float64), B.astype(np.float64), 1e-3
    inside = np.zeros((T, 1))
    inside[off[0]:off[-1]] = 1
    for _ in range(3):
        u, v = rng.standard_normal(A.shape) * inside, rng.standard_normal(B.shape)
        num_a = (loss(a + h * u, b) - loss(a - h * u, b)) / (2 * h)
        num_b = (loss(a, b + h * v) - loss(a, b - h * v)) / (2 * h)
        # each entry is off by at most half a step of its type plus its sum's roundings
        lim_a = lim_b = 1e-6 * (abs(num_a) + abs(num_b) + 1)
        for e in range(E):
            r, d, w = _rows(off, e), np.abs(dC[_rows(off, e)].astype(np.float64)), np.abs(b[e])
            lim_a += (np.abs(u[r]) * plain.bound(dA[r], d @ w, N, **plain.F16)).sum()
            lim_b += (np.abs(v[e]) * plain.bound(dB[e], d.T @ np.abs(a[r]), sizes[e], **plain.F32)).sum()
        assert abs((dA * u * inside).sum() - num_a) <= lim_a
        assert abs((dB * v).sum() - num_b) <= lim_b


def test_expert_layer_run_together():
    """Forward, both gradients, then the same experts quantized: the grouped
    4-bit product, and the grouped product of the weights read back."""
    rng = np.random.default_rng(9)
    sizes, off, T = _route("mid")
    E, N, K = len(sizes), 256, 384
    X, W, dC = _f16(rng, (T, K)), _f16(rng, (E, N, K), 0.05), _f16(rng, (T, N))
    o, x, w, d = dev(off), dev(X), dev(W), dev(dC)
    y = gf.gemm_f16_grouped_nt(x, w, o, _sentinel((T, N)))
    dx = gf.gemm_f16_grouped_nn(d, w, o, _sentinel((T, K)))
    dw = gf.gemm_f16_grouped_tn(d, x, o, out_f32=True)
    Q, S, Z = gf.w4_quantize_f16(w, 64)
    y4 = gf.gemm_w4_f16_grouped_nt(x, Q, S, Z, o, _sentinel((T, N)), 64)
    back = gf.w4_dequantize_f16(Q, S, Z, 64)
    yb = gf.gemm_f16_grouped_nt(x, back, o, _sentinel((T, N)))
    torch.cuda.synchronize()
    _check_rows(y, X, W, off, T, K, "y", True)
    _check_rows(dx, dC, W, off, T, N, "dx", False)
    for e in range(E):
        a, b = dC[_rows(off, e)].astype(np.float64), X[_rows(off, e)].astype(np.float64)
        plain.check(dw[e].cpu().numpy(), a.T @ b, np.abs(a).T @ np.abs(b), sizes[e], plain.F32, "dw")
    q = plain.unpack(Q.view(E * N, -1).cpu().numpy())
    W4 = plain.weights(q, S.view(E * N, -1).cpu().numpy(), Z.view(E * N, -1).cpu().numpy(), 64).reshape(E, N, K)
    _check_rows(y4, X, W4, off, T, K, "y4", True, T > 16 * E)
    _check_rows(yb, X, back.cpu().numpy(), off, T, K, "yb", True)


def test_offsets_against_the_contract_stay_inside():
    """Decreasing, negative and too large offsets: the operands' neighbours in
    memory keep their contents."""
    rng = np.random.default_rng(4)
    T, E, N, K = 100, 4, 72, 64
    A, B = dev(_f16(rng, (T, K))), dev(_f16(rng, (E, N, K)))
    Q, S, Z = gf.w4_quantize_f16(B, 32)
    D = dev(_f16(rng, (T, N)))
    for off in ([50, 20, 90, 10, 60], [-5, 30, 30, 400, 2 ** 31 - 1], [-2 ** 31, -1, 200, -7, 100], [0, 0, 0, 0, 10 ** 6]):
        o = dev(np.array(off, dtype=np.int32))
        _say("offsets", off)
        whole = _sentinel((3 * T, N))
        gf.gemm_f16_grouped_nt(A, B, o, whole[T:2 * T])
        gf.gemm_w4_f16_grouped_nt(A, Q, S, Z, o, whole[T:2 * T], 32)
        back = _sentinel((3 * T, K))
        gf.gemm_f16_grouped_nn(D, B, o, back[T:2 * T])
        dw = torch.full((3 * E, N, K), 7.0, dtype=torch.float32, device="cuda")
        gf.gemm_f16_grouped_tn(D, A, o, dw[E:2 * E])
        torch.cuda.synchronize()
        for t in (whole, back):
            v = t.view(torch.int16)
            assert (v[:T] == SENTINEL).all() and (v[2 * T:] == SENTINEL).all()
        assert (dw[:E] == 7).all() and (dw[2 * E:] == 7).all()


def _serving_calls(b, out):
    gf.gemm_f16_grouped_nt(b["x"], b["w"], b["o"], out["y"])
    gf.gemm_f16_grouped_nn(b["d"], b["w"], b["o"], out["dx"])
    gf.gemm_f16_grouped_tn(b["d"], b["x"], b["o"], out["dw"])
    gf.w4_quantize_f16(b["w"], 64, Q=out["Q"], S=out["S"], Z=out["Z"])
    gf.w4_dequantize_f16(out["Q"], out["S"], out["Z"], 64, W=out["back"])
    gf.gemm_w4_f16_grouped_nt(b["x"], out["Q"], out["S"], out["Z"], b["o"], out["y4"], 64)
    gf.gemm_w4_f16_nt(b["x"], out["Q"][0], out["S"][0], out["Z"][0], out["c4"], 64)
    gf.gemv_w4_f16(out["Q"][1], out["S"][1], out["Z"][1], b["x"][0], out["g4"], 64)


def _buffers(T, E, N, K):
    e = lambda s, dt=torch.float16: torch.zeros(s, dtype=dt, device="cuda")
    b = dict(x=e((T, K)), w=e((E, N, K)), d=e((T, N)), o=e((E + 1,), torch.int32))
    outs = [dict(y=e((T, N)), dx=e((T, K)), dw=e((E, N, K), torch.float32), Q=e((E, N, K // 8), torch.int32),
                 S=e((E, N, K // 64)), Z=e((E, N, K // 64), torch.uint8), back=e((E, N, K)), y4=e((T, N)),
                 c4=e((T, N)), g4=e((N,))) for _ in range(2)]
    return b, outs


def _fill(b, seed, T, E):
    rng = np.random.default_rng(seed)
    for k in ("x", "w", "d"):
        b[k].copy_(dev(_f16(rng, tuple(b[k].shape), 0.5)))
    cuts = np.sort(rng.integers(0, T + 1, E - 1))
    b["o"].copy_(dev(np.concatenate([[0], cuts, [T]]).astype(np.int32)))


def test_graph_replays_with_new_routes():
    """One captured graph serves every route: the offsets are read on the
    device at each replay."""
    T, E, N, K = 150, 5, 136, 192
    b, outs = _buffers(T, E, N, K)
    _fill(b, 0, T, E)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _serving_calls(b, outs[0])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    _say("capturing")
    with torch.cuda.graph(g):
        _serving_calls(b, outs[0])
    for rep in range(4):
        _fill(b, 10 + rep, T, E)
        for t in outs[0].values():
            t.fill_(3)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        _serving_calls(b, outs[1])
        torch.cuda.synchronize()
        for k in outs[0]:
            assert torch.equal(outs[0][k], outs[1][k]), "replay %d: %s" % (rep, k)


def test_two_streams_and_an_explicit_one():
    T, E, N, K = 150, 5, 136, 192
    b, outs = _buffers(T, E, N, K)
    _fill(b, 1, T, E)
    want = outs[0]
    _serving_calls(b, want)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    sets = [_buffers(T, E, N, K)[1][0] for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o in ((s1, sets[0]), (s2, sets[1])):
            with torch.cuda.stream(s):
                _serving_calls(b, o)
    made = gf.gemm_f16_grouped_nt(b["x"], b["w"], b["o"], stream=s1)
    torch.cuda.synchronize()
    for o in sets:
        for k in want:
            assert torch.equal(o[k], want[k]), k
    assert torch.equal(made, want["y"])
