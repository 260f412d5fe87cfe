"""Routing in every launch: four tokens a wave up to 256 experts, one a wave, in one
workgroup, in small ones and in those of 16 waves, with each type, mask and kind of tie."""
import numpy as np
import pytest

import gemv_fp16_amd as gf
from tests import route_plain as plain
from tests.test_gpu_route import _check_rows, _logits, _say
from tests.util import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SIZES = [(4097, 200, 8), (4097, 256, 16), (4099, 129, 3), (4095, 256, 8), (4100, 257, 4), (1025, 300, 5), (1024, 300, 5),
         (1100, 1000, 2), (4096, 128, 17), (2000, 64, 6), (1500, 12, 3), (1500, 30, 4), (1500, 100, 8), (1500, 40, 20),
         (10, 20, 3), (100, 20, 3), (100, 60, 4), (100, 128, 20), (10, 100, 20), (10, 400, 5)]


def _check_some(x, k, bias, opt, out):
    """Choices and weights of 100 tokens, the first, last and masked ones among them; all places."""
    T = len(x)
    got, gw = out[0].cpu().numpy(), out[1].cpu().numpy().astype(np.float64)
    choice = {n: opt[n] for n in ("groups", "top_groups", "group_best") if n in opt}
    for t in {0, 1, T // 3, T // 2, T - 2, T - 1, *np.random.default_rng(T).integers(0, T, 94)}:
        ref = plain.choose(x[t], k, bias, opt["score"], **choice)
        assert list(got[t]) == ref, (t, got[t], ref)
        rw = plain.weights(x[t], ref, opt["score"], opt["renorm"], opt["scale"])
        assert (np.abs(gw[t] - rw) <= plain.weight_bound(x[t], rw)).all(), (t, gw[t], rw)
    _check_rows(got, out[2], out[3], x.shape[1])


@pytest.mark.parametrize("T,E,k", SIZES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked", "lowest", "far"])
def test_choices_and_weights(T, E, k, f32, kind):
    rng = np.random.default_rng(T + E + k)
    x = _logits(rng, T, E, f32, kind)
    opt = dict(score="sigmoid" if kind in ("ties", "far") else "softmax", renorm=kind in ("normal", "ties"), scale=1.0)
    _say("route forms", T, E, k, f32, kind)
    out = gf.route_topk(dev(x), k, **opt)
    key = x.astype(np.float64)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    ids[np.take_along_axis(key, ids, 1) == -np.inf] = -1
    assert np.array_equal(out[0].cpu().numpy(), ids)
    _check_some(x, k, None, opt, out)


@pytest.mark.parametrize("T,E,k,groups", [(1025, 300, 5, 1), (1500, 256, 8, 8), (1100, 60, 6, 3), (1030, 1000, 12, 1), (1100, 100, 5, 1), (10, 100, 4, 1), (10, 400, 4, 1)])
@pytest.mark.parametrize("kind", ["normal", "ties", "masked"])
def test_with_a_bias(T, E, k, groups, kind):
    rng = np.random.default_rng(T + E)
    for f32 in (False, True):
        x = _logits(rng, T, E, f32, kind)
        bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
        opt = dict(score="sigmoid" if groups > 1 else "softmax", renorm=True, scale=2.5, groups=groups,
                   top_groups=(groups + 1) // 2, group_best=2 if groups > 1 else 1)
        _say("route forms, bias", T, E, k, f32, kind)
        _check_some(x, k, bias, opt, gf.route_topk(dev(x), k, bias=dev(bias), **opt))


def test_nan_and_infinity():
    for T, E, k in ((4100, 200, 4), (1100, 300, 4)):
        x = _logits(np.random.default_rng(T), T, E, True)
        x[5, 7], x[9, E - 1], x[T - 1, :] = np.nan, np.inf, np.nan
        _say("route forms, nan", T, E, k)
        ids, w, offsets, place = gf.route_topk(dev(x), k, score="sigmoid")
        got, gw = ids.cpu().numpy(), w.cpu().numpy()
        assert got[5, 0] == 7 and got[9, 0] == E - 1 and list(got[T - 1]) == [0, 1, 2, 3]
        assert np.isnan(gw[5, 0]) and gw[9, 0] > 0 and np.isnan(gw[T - 1]).all()
        for t in (4, 6, 8, 10, T - 2):
            assert list(got[t]) == plain.choose(x[t], k, None, "sigmoid") and np.isfinite(gw[t]).all()
        _check_rows(got, offsets, place, E)
