"""Routing to experts, the sort by expert and the router's gradient on the GPU
against plain 64-bit forms."""
import sys

import numpy as np
import pytest

import gemv_fp16_amd as gf
from tests import route_plain as plain
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


def _logits(rng, T, E, f32, kind="normal"):
    x = rng.standard_normal((T, E)) * 1.5
    if kind == "ties":                     # few values: most choices are ties
        x = np.round(x)
    elif kind == "masked":                 # some experts out, one row with nothing, one with a single expert
        x[rng.random((T, E)) < 0.4] = -np.inf
        x[T // 2] = -np.inf
        x[T // 3] = -np.inf
        x[T // 3, E // 2] = 0.25
    elif kind == "lowest":                 # the type's lowest value as a mask
        x[rng.random((T, E)) < 0.5] = np.finfo(np.float32 if f32 else np.float16).min
        x[T // 2] = np.finfo(np.float32 if f32 else np.float16).min
    elif kind == "far":                    # scores over the whole range, most of them underflow
        x = x * 40 - 60
    return x.astype(np.float32 if f32 else np.float16)


def _check_rows(ids, offsets, place, E):
    off, at = plain.rows(ids, E)
    assert np.array_equal(offsets.cpu().numpy(), off)
    assert np.array_equal(place.cpu().numpy(), at)


def _check(x, k, bias, opt, out):
    ids, w, offsets, place = out
    got, gw = ids.cpu().numpy(), w.cpu().numpy().astype(np.float64)
    choice = {n: opt[n] for n in ("groups", "top_groups", "group_best") if n in opt}
    for t in range(len(x)):
        ref = plain.choose(x[t], k, bias, opt["score"], **choice)
        assert list(got[t]) == ref, (t, got[t], ref)
        rw = plain.weights(x[t], ref, opt["score"], opt["renorm"], opt.get("scale", 1.0))
        err = np.abs(gw[t] - rw)
        assert (err <= plain.weight_bound(x[t], rw)).all(), (t, gw[t], rw)
    _check_rows(got, offsets, place, x.shape[1])


SIZES = [(1, 1, 1), (1, 8, 2), (3, 64, 8), (16, 60, 6), (64, 65, 3), (65, 128, 8), (200, 130, 1), (7, 256, 64),
         (130, 257, 10), (33, 512, 8), (90, 1000, 12), (70, 1024, 5), (300, 16, 16), (5000, 24, 2)]


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_choices_and_weights(T, E, k, score, with_bias):
    rng = np.random.default_rng(T * 31 + E)
    for f32 in ((False, True) if T < 1000 else (True,)):
        for kind in ("normal", "ties", "masked", "lowest", "far"):
            if T >= 1000 and kind != "normal":
                continue
            x = _logits(rng, T, E, f32, kind)
            bias = (rng.standard_normal(E) * 0.1).astype(np.float32) if with_bias else None
            opt = dict(score=score, renorm=kind != "lowest", scale=2.5 if kind == "ties" else 1.0)
            _say("route", T, E, k, score, f32, kind, opt)
            out = gf.route_topk(dev(x), k, bias=None if bias is None else dev(bias), **opt)
            _check(x, k, bias, opt, out)


@pytest.mark.parametrize("T,E,k,groups,top_groups", [
    (5, 64, 8, 8, 4), (70, 256, 8, 8, 4), (20, 160, 6, 8, 3), (20, 60, 4, 5, 2), (9, 1024, 10, 64, 7),
    (9, 64, 3, 64, 3), (3, 33, 5, 3, 3), (66, 512, 32, 2, 1), (5, 24, 7, 6, 2), (1, 2, 1, 2, 1)])
@pytest.mark.parametrize("group_best", [1, 2])
@pytest.mark.parametrize("with_bias", [False, True])
def test_groups(T, E, k, groups, top_groups, group_best, with_bias):
    rng = np.random.default_rng(E + groups)
    for kind in ("normal", "ties", "masked"):
        for score in ("softmax", "sigmoid"):
            x = _logits(rng, T, E, score == "sigmoid", kind)
            bias = (rng.standard_normal(E) * 0.2).astype(np.float32) if with_bias else None
            opt = dict(score=score, renorm=score == "sigmoid", groups=groups, top_groups=top_groups,
                       group_best=group_best)
            _say("route groups", T, E, k, kind, opt, with_bias)
            out = gf.route_topk(dev(x), k, bias=None if bias is None else dev(bias), **opt)
            _check(x, k, bias, opt, out)


def test_bias_of_minus_infinity_closes_an_expert():
    rng = np.random.default_rng(5)
    x = _logits(rng, 20, 32, True)
    bias = np.zeros(32, dtype=np.float32)
    bias[[0, 3, 31]] = -np.inf
    for E_open, k in ((29, 29), (29, 32)):
        opt = dict(score="softmax", renorm=False)
        out = gf.route_topk(dev(x), k, bias=dev(bias), **opt)
        got = out[0].cpu().numpy()
        assert not np.isin(got, [0, 3, 31]).any()
        assert ((got >= 0).sum(1) == E_open).all()
        _check_rows(got, out[2], out[3], 32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_nan_and_infinity(score, renorm):
    """A NaN ranks above every number and shows in the weights; other rows are untouched by it."""
    rng = np.random.default_rng(6)
    x = _logits(rng, 6, 40, True)
    x[1, 7] = np.nan
    x[3, 9] = np.inf
    x[4, :] = np.nan
    ids, w, offsets, place = gf.route_topk(dev(x), 3, score=score, renorm=renorm)
    got, gw = ids.cpu().numpy(), w.cpu().numpy()
    assert got[1, 0] == 7 and got[3, 0] == 9 and list(got[4]) == [0, 1, 2]
    assert np.isnan(gw[1, 0]) and np.isnan(gw[4]).all()
    assert np.isnan(gw[3, 0]) if score == "softmax" else gw[3, 0] > 0
    for t in (0, 2, 5):
        assert list(got[t]) == plain.choose(x[t], 3, None, score)
        assert np.isfinite(gw[t]).all()
    _check_rows(got, offsets, place, 40)


def test_without_rows_and_with_the_callers_outputs():
    rng = np.random.default_rng(7)
    for T in (5, 300):
        x = dev(_logits(rng, T, 96, False))
        a = gf.route_topk(x, 4)
        b = gf.route_topk(x, 4, rows=False)
        assert b[2] is None and b[3] is None
        ids = torch.full((T, 4), -7, dtype=torch.int32, device="cuda")
        w = torch.full((T, 4), 7.0, device="cuda")
        off = torch.full((97,), -7, dtype=torch.int32, device="cuda")
        at = torch.full((T, 4), -7, dtype=torch.int32, device="cuda")
        ws = torch.full((gf.route_workspace_bytes(T, 96, 4) + 64,), 255, dtype=torch.uint8, device="cuda")
        c = gf.route_topk(x, 4, ids=ids, weights=w, offsets=off, place=at, workspace=ws)
        assert c[0] is ids and c[1] is w and c[2] is off and c[3] is at
        for u, v in ((a, b[:2]), (a, c)):
            for p, q in zip(u, v):
                assert torch.equal(p, q)
        assert (ws[-64:] == 255).all()


def test_unaligned_logits():
    rng = np.random.default_rng(8)
    for f32 in (False, True):
        x = dev(_logits(rng, 70, 256, f32))
        flat = torch.empty(x.numel() + 1, dtype=x.dtype, device="cuda")
        y = flat[1:].view(x.shape)
        y.copy_(x)
        for u, v in zip(gf.route_topk(x, 8), gf.route_topk(y, 8)):
            assert torch.equal(u, v)


def test_no_tokens():
    x = torch.empty((0, 16), device="cuda")
    ids, w, offsets, place = gf.route_topk(x, 2)
    assert ids.shape == (0, 2) and (offsets == 0).all()
    offsets, place = gf.route_rows(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 16,
                                   offsets=torch.full((17,), 9, dtype=torch.int32, device="cuda"))
    assert (offsets == 0).all()


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (4096, 1, 8), (4097, 1, 8), (512, 8, 256), (513, 8, 256), (3000, 7, 1024),
                                   (700, 6, 33), (40000, 4, 64), (9, 500, 3), (150000, 2, 1000)])
@pytest.mark.parametrize("kind", ["even", "one", "none", "stray"])
def test_sort_of_given_ids(T, k, E, kind):
    rng = np.random.default_rng(T + E)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    if kind == "one":
        ids[:] = E - 1
    elif kind == "none":
        ids[:] = -1
    elif kind == "stray":                  # ids that are no expert's
        ids[rng.random((T, k)) < 0.3] = -1
        ids[0, 0], ids[-1, -1] = E, np.iinfo(np.int32).min
    _say("sort", T, k, E, kind)
    offsets, place = gf.route_rows(dev(ids), E)
    _check_rows(ids, offsets, place, E)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 64, 8), (70, 160, 6), (9, 1000, 64), (300, 33, 4), (2, 512, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("f32", [False, True])
def test_gradient(T, E, k, score, renorm, f32):
    rng = np.random.default_rng(T + E + k)
    for kind in ("normal", "masked", "lowest", "far"):
        x = _logits(rng, T, E, f32, kind)
        ids = np.array([plain.choose(x[t], k, None, score) for t in range(T)], dtype=np.int32)
        if kind == "normal" and k > 2:     # stray ids, and one expert twice
            ids[0, 1], ids[-1, 0], ids[T // 2, 2] = -1, E + 5, ids[T // 2, 1]
        dw = rng.standard_normal((T, k)).astype(np.float32)
        _say("route gradient", T, E, k, score, renorm, f32, kind)
        dx = gf.route_topk_bwd(dev(x), dev(ids), dev(dw), score=score, renorm=renorm, scale=1.5).cpu().numpy()
        for t in range(T):
            ref = plain.grad(x[t], ids[t], dw[t], score, renorm, 1.5)
            bound = plain.grad_bound(x[t], ids[t], dw[t], ref, score, renorm, 1.5, plain.F32 if f32 else plain.F16)
            err = np.abs(dx[t].astype(np.float64) - ref)
            assert (err <= bound).all(), (t, err.max(), bound[err.argmax()])


def test_results_repeat_on_streams_and_in_graphs():
    """A side stream, and a graph of all three calls replayed over new inputs
    with eager calls between, give the eager results bit for bit."""
    rng = np.random.default_rng(11)
    for T, E, k in ((40, 64, 8), (700, 256, 8)):
        xs = [_logits(rng, T, E, True) for _ in range(4)]
        dws = [rng.standard_normal((T, k)).astype(np.float32) for _ in range(4)]
        opt = dict(score="sigmoid", renorm=True)
        bias = dev((rng.standard_normal(E) * 0.1).astype(np.float32))
        x, dw = dev(xs[0]), dev(dws[0])

        def chain(x, dw):
            out = gf.route_topk(x, k, bias=bias, groups=8, top_groups=4, group_best=2, **opt)
            off, at = gf.route_rows(out[0], E)
            return (*out, off, at, gf.route_topk_bwd(x, out[0], dw, **opt))

        side = torch.cuda.Stream()
        want = chain(x, dw)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            got = chain(x, dw)
        explicit = gf.route_topk(x, k, bias=bias, groups=8, top_groups=4, group_best=2, stream=side, **opt)
        side.synchronize()
        for u, v in zip(want, got):
            assert torch.equal(u, v)
        for u, v in zip(want, explicit):
            assert torch.equal(u, v)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = chain(x, dw)
        for i in range(1, 4):
            _say("route graph", T, i)
            x.copy_(dev(xs[i]))
            dw.copy_(dev(dws[i]))
            eager = [t.clone() for t in chain(x.clone(), dw.clone())]
            graph.replay()
            torch.cuda.synchronize()
            for u, v in zip(held, eager):
                assert torch.equal(u, v)
