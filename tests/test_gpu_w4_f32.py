"""4-bit products that leave their sums in fp32, and adapters added to them with one rounding."""
import ctypes
import os
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


def _weights(N, K, group, zeros, seed):
    """Words of codes, scales 1, 2 and 4, zero points, and the integers they stand for."""
    rng = np.random.default_rng(seed)
    G = (K + group - 1) // group
    q = rng.integers(0, 16, (N, K // 8, 8)).astype(np.uint32)
    Q = (q << np.arange(0, 32, 4, dtype=np.uint32)).sum(2, dtype=np.uint32).view(np.int32)
    S = (2.0 ** rng.integers(0, 3, (N, G))).astype(np.float16)
    Z = rng.integers(0, 16, (N, G)).astype(np.uint8) if zeros else None
    up = lambda v: np.repeat(v, group, axis=1)[:, :K].astype(np.float64)
    W = (q.reshape(N, K).astype(np.float64) - (up(Z) if zeros else 8.0)) * up(S)
    return Q, S, Z, W


# (M, N, K): A in LDS, in passes of 16 and of 32 rows, long K; general forms; few blocks past
# 64 rows; each tile; no K
SIZES = [(1, 520, 4096), (9, 2048, 2048), (24, 4096, 4096), (24, 11008, 1024), (64, 264, 8192), (3, 100, 8632), (40, 130, 264),
         (100, 500, 4096), (65, 40, 96), (300, 520, 512), (300, 4096, 520), (700, 4096, 512), (1024, 8192, 256),
         (2048, 8192, 256), (2100, 8200, 264), (5, 33, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_sums_in_fp32(M, N, K, group):
    """Integers: the fp32 sums are exact.  Random values: rounded, they are the fp16 result."""
    rng = np.random.default_rng(M + K)
    Q, S, Z, W = _weights(N, K, group, M % 2 == 0, N + K)
    A = rng.integers(-7, 8, (M, K)).astype(np.float16)
    exact = A.astype(np.float64) @ W.T
    assert (np.abs(A).astype(np.float64).sum(1) * 60).max(initial=0) < 2 ** 24
    Q, S, Z = dev(Q), dev(S), None if Z is None else dev(Z)
    for shift in (0, 1):
        _say("w4 fp32", M, N, K, group, shift)
        held = torch.full((M * N + 64,), 7.0, device="cuda")
        C = held[shift:shift + M * N].view(M, N)
        assert gf.gemm_w4_f16_nt(_shifted(dev(A), shift), Q, S, Z, C=C, group=group) is C
        assert np.array_equal(C.cpu().numpy(), exact.astype(np.float32))
        assert (held[:shift] == 7).all() and (held[shift + M * N:] == 7).all()
        X = _shifted(dev(rng.standard_normal((M, K)).astype(np.float16)), shift)
        both = [gf.gemm_w4_f16_nt(X, Q, S, Z, group=group, out_f32=f) for f in (True, False)]
        assert both[0].dtype == torch.float32
        assert torch.equal(both[0].half().view(torch.int16), both[1].view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,r,L", [(1, 520, 4096, 16, 3), (24, 11008, 4096, 16, 16), (24, 130, 1000, 4, 5), (64, 264, 8192, 24, 4),
                                       (100, 500, 4096, 16, 4), (300, 520, 1024, 16, 6)])
def test_adapters_beside_4_bit_weights_are_rounded_once(M, N, K, r, L):
    p = Integers(M, 8, K, r, L, M + K)
    rng = np.random.default_rng(N)
    Q, S, Z, W = _weights(N, K, 64, True, N + K)
    u = rng.integers(-1, 2, (L, N, r)) * (rng.random((L, N, r)) < 8 / r)
    low = np.zeros((M, N))
    for e in range(L):
        m = p.ids == e
        low[m] = p.H[m] @ u[e].T.astype(np.float64)
    base = p.A.astype(np.float64) @ W.T
    with np.errstate(over="ignore"):
        once = (base + low).astype(np.float16)
        assert (once != (base.astype(np.float16).astype(np.float64) + low).astype(np.float16)).any()
    A, Q, S, Z = dev(p.A), dev(Q), dev(S), dev(Z)
    _say("w4 lora", M, N, K, r, L)
    C = gf.gemm_w4_f16_nt(A, Q, S, Z, group=64, out_f32=True)
    got = gf.lora_add_f16(A, dev(p.ids), dev(p.Down), dev(u.astype(np.float16)), C, dev(p.scales))
    assert np.array_equal(got.cpu().view(torch.int16).numpy(), once.view(np.int16))


@pytest.mark.gpu
def test_pair_in_a_graph():
    M, N, K, r, L = 24, 1024, 4096, 16, 4
    Q, S, Z, W = _weights(N, K, 64, True, 1)
    problems = [Integers(M, N, K, r, L, s) for s in range(3)]
    p = problems[0]
    Q, S, Z = dev(Q), dev(S), dev(Z)
    A, Down, Up, scales, ids = (dev(v) for v in (p.A, p.Down, p.Up, p.scales, p.ids))

    def chain():
        return gf.lora_add_f16(A, ids, Down, Up, gf.gemm_w4_f16_nt(A, Q, S, Z, group=64, out_f32=True), scales)
    chain()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        C = chain()
    for q in problems[1:] + problems[:1]:
        _say("w4 lora graph")
        for t, v in ((A, q.A), (Down, q.Down), (Up, q.Up), (scales, q.scales), (ids, q.ids)):
            t.copy_(dev(v))
        want = q.once(q.A.astype(np.float64) @ W.T)
        assert np.array_equal(chain().cpu().view(torch.int16).numpy(), want.view(np.int16))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(C.cpu().view(torch.int16).numpy(), want.view(np.int16))


def test_refusals():
    if not os.path.exists(gf.LIB_PATH):
        from gemv_fp16_amd import build
        build.build()
    P, ODD, TWO, NULL = (ctypes.c_void_p(v) for v in (0x10000, 0x10001, 0x10002, 0))      # never dereferenced

    def f(A=P, Q=P, S=P, Z=NULL, C=P, M=4, N=16, K=64, group=64):
        return gf.lib().gemm_w4_f16_nt_f32(A, Q, S, Z, C, M, N, K, group, NULL)
    for bad in (dict(M=-1), dict(N=-1), dict(K=-8), dict(K=60), dict(group=16), dict(C=TWO), dict(C=ODD), dict(C=NULL),
                dict(A=NULL), dict(A=ODD), dict(Q=TWO), dict(S=ODD), dict(M=65536, N=65536), dict(M=2 ** 30 + 1)):
        assert f(**bad) == gf.GF_ERR_INVALID_ARG, bad
    assert f(M=0, C=NULL) == gf.GF_OK and f(N=0, C=NULL) == gf.GF_OK
    with pytest.raises(ValueError):
        gf.gemm_w4_f16_nt(torch.zeros((2, 8), dtype=torch.float16), torch.zeros((3, 1), dtype=torch.int32),
                          torch.zeros((3, 1), dtype=torch.float16), C=torch.zeros((2, 4)), group=64)
