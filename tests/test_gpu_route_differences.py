"""route_topk_bwd against differences of route_topk's own weights."""
import numpy as np
import pytest

import gemv_fp16_amd as gf
from tests import route_plain as plain
from tests.util import dev

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,k", [(1, 1), (5, 2), (24, 6), (64, 64), (200, 8), (300, 20)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_against_differences(E, k, score, renorm):
    """The chosen logits lie a step and more above the others, so that all points of a
    difference choose the same experts.  A central difference of step h is off by at most h^2 /
    6 of the third derivative, at most 1 for each weight, and by the weights' own bounds over h."""
    rng = np.random.default_rng(E * 3 + k)
    h, scale = 2.0 ** -6, 1.5
    x = rng.uniform(-2.0, -1.0, E)
    x[rng.permutation(E)[:k]] += 2.5
    x = x.astype(np.float32)
    dw = rng.standard_normal(k).astype(np.float32)
    opt = dict(score=score, renorm=renorm, scale=scale)
    ids = gf.route_topk(dev(x[None]), k, **opt)[0]
    order = ids.cpu().numpy()[0]
    print("route differences", E, k, opt, flush=True)
    dx = gf.route_topk_bwd(dev(x[None]), ids, dev(dw[None]), **opt).cpu().numpy()[0].astype(np.float64)
    moved = np.repeat(x[None].astype(np.float64), 2 * E, 0)
    moved[np.arange(E), np.arange(E)] += h
    moved[E + np.arange(E), np.arange(E)] -= h
    moved = moved.astype(np.float32)
    step = (moved[np.arange(E), np.arange(E)].astype(np.float64) - moved[E + np.arange(E), np.arange(E)])
    got, w = (t.cpu().numpy() for t in gf.route_topk(dev(moved), k, **opt)[:2])
    of = np.full(E, -1)
    of[order] = np.arange(k)
    assert (np.sort(got, 1) == np.sort(order)).all()
    loss, err = np.zeros(2 * E), np.zeros(2 * E)
    for t in range(2 * E):
        g = dw[of[got[t]]].astype(np.float64)
        loss[t] = (g * w[t].astype(np.float64)).sum()
        ref = plain.weights(moved[t], list(got[t]), score, renorm, scale)
        err[t] = (np.abs(g) * plain.weight_bound(moved[t], ref)).sum()
    diff = (loss[:E] - loss[E:]) / step
    size = scale * np.abs(dw).sum()
    bound = (err[:E] + err[E:]) / step + h * h / 6 * size + plain.F32 * 200 * size
    assert (np.abs(diff - dx) <= bound).all(), float((np.abs(diff - dx) / bound).max())
