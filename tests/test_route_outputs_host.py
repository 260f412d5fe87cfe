"""The routing calls' outputs are tensors of their own: each can be kept, saved or changed in
place by itself.  On the CPU, with the launch taken out."""
import os

import pytest

import gemv_fp16_amd as gf

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True)
def _host(monkeypatch):
    if not os.path.exists(gf.LIB_PATH):
        from gemv_fp16_amd import build
        build.build()
    monkeypatch.setattr(gf, "_ptr", lambda t, dtype, name: t.data_ptr())
    monkeypatch.setattr(gf, "_launch", lambda name, tensors, stream, *args: None)


@pytest.mark.parametrize("T", [1, 16, 100])
def test_outputs_share_nothing(T):
    out = gf.route_topk(torch.zeros((T, 8)), 2)
    assert [tuple(t.shape) for t in out] == [(T, 2), (T, 2), (9,), (T, 2)]
    assert [t.dtype for t in out] == [torch.int32, torch.float32, torch.int32, torch.int32]
    assert len({t.untyped_storage().data_ptr() for t in out}) == 4
    for t in out:
        assert t.untyped_storage().nbytes() == 4 * t.numel() and t._base is None
    before = [t._version for t in out]
    out[0].zero_()
    assert [t._version for t in out] == [before[0] + 1] + before[1:]


def test_ids_changed_after_the_weights_were_used_under_autograd():
    for change in (0, 2, 3):
        out = gf.route_topk(torch.zeros((20, 8)), 2)
        x = torch.ones((20, 2), requires_grad=True)
        y = (x * out[1]).sum()
        out[change].fill_(-1)
        y.backward()
        assert torch.equal(x.grad, out[1])


def test_weights_scaled_after_the_ids_were_saved_for_a_backward():
    class Routed(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, ids):
            ctx.save_for_backward(ids)
            return x.clone()

        @staticmethod
        def backward(ctx, g):
            return g + 0 * ctx.saved_tensors[0], None

    ids, weights = gf.route_topk(torch.zeros((20, 8)), 2)[:2]
    ids.zero_()
    x = torch.ones((20, 2), requires_grad=True)
    y = Routed.apply(x, ids).sum()
    weights.mul_(0.5)
    y.backward()
    assert (x.grad == 1).all()


def test_rows_of_given_ids():
    offsets, place = gf.route_rows(torch.zeros((5000, 2), dtype=torch.int32), 8)
    assert offsets.untyped_storage().data_ptr() != place.untyped_storage().data_ptr()
    assert offsets.untyped_storage().nbytes() == 36 and place.untyped_storage().nbytes() == 40000
