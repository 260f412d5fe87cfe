"""Adapters beside a projection are rounded once, in every form: bit for bit on integers."""
import sys

import numpy as np
import pytest

import gemv_fp16_amd as gf
from tests.lora_plain import Integers
from tests.util import dev

torch = pytest.importorskip("torch")


def _say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def _shifted(t, elems):
    flat = torch.empty(t.numel() + elems, dtype=t.dtype, device=t.device)
    out = flat[elems:].view(t.shape)
    out.copy_(t)
    return out


def _same(got, want, what):
    got, want = got.cpu().view(torch.int16).numpy(), want.view(np.int16)
    bad = got != want
    assert not bad.any(), "%s: %d of %d differ, first at %s" % (what, bad.sum(), bad.size, np.argwhere(bad)[0])


# (M, N, K, r, adapters): vectors; K in slices; streaming, with and without a launch for
# the products by Down; 33 to 64 rows and long K; tiles; ranks, K and sizes of no form;
# more rows than one round of the general form takes; no adapters at all
CASES = [(1, 2100, 4096, 16, 8), (2, 4100, 2056, 32, 2), (1, 130, 512, 256, 3), (3, 16, 1544, 8, 2), (16, 1000, 4096, 24, 3),
         (32, 520, 2048, 16, 8), (8, 520, 1024, 16, 1), (12, 520, 1024, 16, 4), (30, 264, 512, 40, 7), (9, 520, 8200, 16, 3),
         (20, 520, 8192, 16, 4), (33, 72, 1000, 24, 5), (40, 130, 264, 8, 9), (64, 4096, 4096, 16, 24), (5, 9, 640, 16, 2),
         (65, 136, 520, 8, 3), (300, 520, 264, 24, 9), (700, 384, 256, 16, 50), (2100, 264, 512, 64, 3),
         (1, 33, 77, 3, 2), (7, 100, 1001, 4, 3), (48, 264, 512, 4, 6), (200, 131, 1001, 7, 4), (300, 264, 512, 12, 2),
         (200, 66000, 64, 4, 3), (40, 66000, 64, 12, 2), (17, 40, 512, 5, 0), (70, 64, 0, 8, 2), (4, 20, 0, 8, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r,L", CASES)
def test_product_with_adapters(M, N, K, r, L):
    p = Integers(M, N, K, r, L, M + N + K)
    for shift in (0, 1):
        A, B, Down, Up = (_shifted(dev(v), shift) for v in (p.A, p.B, p.Down, p.Up))
        _say("lora integers", M, N, K, r, L, shift)
        need = gf.lora_workspace_bytes(M, N, K, r)
        ws = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
        C = gf.gemm_f16_nt_lora(A, B, dev(p.ids), Down, Up, dev(p.scales), workspace=ws,
                                C=_shifted(torch.full((M, N), 7.0, dtype=torch.float16, device="cuda"), shift))
        _same(C, p.once(), "gemm_f16_nt_lora")
        assert (ws[need:] == 255).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r,L", CASES)
def test_onto_a_base_in_fp32(M, N, K, r, L):
    p = Integers(M, N, K, r, L, M + N + K + 1)
    for shift in (0, 1):
        A, Down, Up = (_shifted(dev(v), shift) for v in (p.A, p.Down, p.Up))
        base = _shifted(dev(p.base.astype(np.float32)), shift)
        before = base.clone()
        _say("lora integers, base", M, N, K, r, L, shift)
        out = _shifted(torch.full((M, N), 7.0, dtype=torch.float16, device="cuda"), shift)
        assert gf.lora_add_f16(A, dev(p.ids), Down, Up, base, dev(p.scales), out=out) is out
        _same(out, p.once(), "lora_add_f16 of a base in fp32")
        assert torch.equal(base, before)
    made = gf.lora_add_f16(dev(p.A), dev(p.ids), dev(p.Down), dev(p.Up), base, dev(p.scales))
    assert made.dtype == torch.float16 and torch.equal(made.view(torch.int16), out.view(torch.int16))


@pytest.mark.gpu
def test_after_a_split_k_product():
    p = Integers(48, 264, 1024, 16, 4, 3)
    base = gf.gemm_f16_nt_splitk_ex(dev(p.A), dev(p.B), split_k=4)
    _same(gf.lora_add_f16(dev(p.A), dev(p.ids), dev(p.Down), dev(p.Up), base, dev(p.scales)), p.once(), "after split-K")


@pytest.mark.gpu
def test_replayed_in_a_graph_and_on_a_side_stream():
    """33 rows and more, and the general form: parts, products by Down and sums of one call
    in a graph that is replayed over new inputs with eager calls between."""
    for M, N, K, r, L in ((48, 264, 1024, 16, 4), (40, 264, 1024, 4, 4), (20, 264, 8192, 16, 4)):
        problems = [Integers(M, N, K, r, L, s) for s in range(3)]
        p = problems[0]
        A, B, Down, Up, scales, ids = (dev(v) for v in (p.A, p.B, p.Down, p.Up, p.scales, p.ids))
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        _same(gf.gemm_f16_nt_lora(A, B, ids, Down, Up, scales, stream=side), p.once(), "side stream")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            C = gf.gemm_f16_nt_lora(A, B, ids, Down, Up, scales)
        for q in problems[1:] + problems[:1]:
            _say("lora integers, graph", M, N, K, r)
            for t, v in ((A, q.A), (B, q.B), (Down, q.Down), (Up, q.Up), (scales, q.scales), (ids, q.ids)):
                t.copy_(dev(v))
            _same(gf.gemm_f16_nt_lora(A, B, ids, Down, Up, scales), q.once(), "eager")
            graph.replay()
            torch.cuda.synchronize()
            _same(C, q.once(), "replayed")


def test_the_problems_show_a_second_rounding():
    """On the CPU: rounding the base before the adapters are added changes these results."""
    for M, N, K, r, L in ((48, 264, 1024, 16, 4), (20, 520, 8192, 16, 4), (48, 264, 512, 4, 6)):
        p = Integers(M, N, K, r, L, M + N + K)
        has = (p.ids >= 0) & (p.ids < L)
        assert (p.once() != p.twice())[has].mean() > 0.02
        assert (p.once() == p.twice())[~has].all()


# ---- refusals, on the CPU ---------------------------------------------------

def test_refusals():
    import ctypes
    import os
    if not os.path.exists(gf.LIB_PATH):
        from gemv_fp16_amd import build
        build.build()
    L = gf.lib()
    P, ODD, TWO, NULL = (ctypes.c_void_p(v) for v in (0x10000, 0x10001, 0x10002, 0))      # never dereferenced
    need = L.lora_workspace_bytes(4, 16, 64, 8)

    def f(A=P, ids=P, Dn=P, Up=P, s=NULL, base=P, C=P, M=4, N=16, K=64, r=8, n=2, ws=P, b=1 << 30):
        return L.lora_add_f32(A, ids, Dn, Up, s, base, C, M, N, K, r, n, ws, b, NULL)
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(r=0), dict(r=257), dict(n=-1), dict(M=65536, N=65536),
                dict(base=NULL), dict(base=ODD), dict(base=TWO), dict(C=NULL), dict(C=ODD), dict(A=NULL), dict(ids=NULL),
                dict(Dn=NULL), dict(Up=NULL), dict(ws=NULL), dict(b=need - 1), dict(n=0, base=NULL)):
        assert f(**bad) == gf.GF_ERR_INVALID_ARG, bad
    assert f(M=0, base=NULL, ws=NULL, b=0) == gf.GF_OK
    # a round of rows, its base in fp32 and the products by Down are what a long call needs
    one = L.lora_workspace_bytes(4096, 4096, 4096, 16)
    assert 4096 * 4096 * 4 <= one <= 4096 * 4096 * 4 + 2 * 4096 * 16 * 4
    assert L.lora_workspace_bytes(2 ** 17, 4096, 64, 16) <= 8192 * 4096 * 4 + 2 ** 17 * 16 * 4
    assert L.lora_workspace_bytes(10000, 4096, 64, 16) <= 5120 * 4096 * 4 + 10000 * 16 * 4
    assert L.lora_workspace_bytes(2, 2 ** 29, 2, 16) <= 2 * 2 ** 29 * 4 + 64 * 16 * 4
    assert L.lora_workspace_bytes(0, 8, 8, 8) == 0 and L.lora_workspace_bytes(8, 0, 8, 8) == 0


def test_binding_refusals():
    h = lambda *s: torch.zeros(s, dtype=torch.float16)
    f, i = lambda *s: torch.zeros(s), lambda *s: torch.zeros(s, dtype=torch.int32)
    for call in (lambda: gf.lora_add_f16(h(2, 8), i(2), h(2, 4, 8), h(2, 4, 4), f(2, 5)),
                 lambda: gf.lora_add_f16(h(2, 8), i(2), h(2, 4, 8), h(2, 4, 4), f(2, 4), out=h(3, 4)),
                 lambda: gf.lora_add_f16(h(2, 8), i(2), h(2, 4, 8), h(2, 4, 4), h(2, 4), out=h(2, 4))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):             # host tensors
        gf.lora_add_f16(h(2, 8), i(2), h(2, 4, 8), h(2, 4, 4), f(2, 4))
