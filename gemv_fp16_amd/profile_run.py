"""Launch one operation a fixed number of times, for an external profiler.

    rocprofv3 --kernel-trace --stats -- python3 -m gemv_fp16_amd.profile_run gemm
    rocprofv3 --pmc FETCH_SIZE -- python3 -m gemv_fp16_amd.profile_run gemv

Ops (inputs are the seeded uniform[-1,1] fp16 workloads):
  gemm    C = A . B^T at M = N = K = 8192 (default tile config); --layout nn / tn
          stores B as K x N (and A as K x M) and runs gemm_f16 on them
  gemv    y = W . x at N = K = 8192, rotating 5 W copies (640 MiB)
  splitk  M = N = 1024, K = 16384, split --split (default 8): fp32 atomic, fp32 two-pass, fp16
          two-pass, operands rotated over 4 copies (256 MiB)
  skinny  C = A . B^T with M = 4 and M = 16 rows of A against an 8192 x 8192 B (5 B copies
          rotated, 640 MiB); the library's default form for each M
  sparse  2:4 sparse C = decompress(A_sparse, E) . B^T at M = N = K = 8192 (A compressed
          once on the GPU from a dense uniform A; default tile config)
  compress  2:4 compression of an 8192 x 8192 A, rotating 3 copies (384 MiB)
  w4      4-bit weights with zero points in groups of 128: quantize and back (8192 x 8192, 3
          copies), one token against 1024 x 1024 (64 copies) and 8192 x 8192 (16), 24 rows against
          11008 x 4096 (24; the same without zero points in groups of 64) and 2048 rows against
          8192 x 4096
  grouped products by expert over uneven groups: a decode batch of 48 rows over 16 experts of
          4096 x 2048, 8191 rows over 8 of 4096 x 4096, both gradients of 4096 rows over 8 of
          4096 x 2048 and of 2999 over 32 of 1024 x 2048 (the one of the weights in fp32 and in
          fp16), and with 4-bit weights 24 rows over 16
          of 4096 x 4096 and 1111 over 8 of 2048 x 4096 (weights of the small ones: 3 copies)
  copy    torch copy of a 512 MiB buffer: a plain copy kernel of known size,
          the calibration for the HBM byte counters
"""
from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def half(torch, seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.float16, device="cuda").uniform_(-1, 1, generator=g)


def offsets(torch, rows, experts):
    """Uneven groups: expert i of n gets a share of the rows in proportion to 1 + i % 5."""
    share = [1 + i % 5 for i in range(experts)]
    ends = [rows * sum(share[:i]) // sum(share) for i in range(experts + 1)]
    return torch.tensor(ends, dtype=torch.int32, device="cuda")


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("op", choices=["gemm", "gemv", "splitk", "skinny", "sparse", "compress", "w4", "grouped", "copy"])
    ap.add_argument("--iters", type=int, default=10)
    ap.add_argument("--m", type=int, default=8192)
    ap.add_argument("--n", type=int, default=8192)
    ap.add_argument("--k", type=int, default=8192)
    ap.add_argument("--layout", choices=["nt", "nn", "tn"], default="nt")
    ap.add_argument("--split", type=int, default=8, help="split-K slices (op splitk)")
    ap.add_argument("--cfg", default="",
                    help="gemm tile config block_m,block_n,block_k,stages,threads,raster[,schedule] "
                         "(default: the library's choice)")
    a = ap.parse_args(argv)

    import torch
    import gemv_fp16_amd as gf
    import inputs

    torch.cuda.set_device(0)
    if a.op == "gemm":
        A = torch.from_numpy(inputs.uniform_f16((a.m, a.k), 0, 0)).cuda()
        B = torch.from_numpy(inputs.uniform_f16((a.n, a.k), 0, 1)).cuda()
        C = torch.empty((a.m, a.n), dtype=torch.float16, device="cuda")
        cfg = None
        if a.cfg:
            v = [int(t) for t in a.cfg.split(",")]
            cfg = dict(zip(("block_m", "block_n", "block_k", "stages", "threads", "raster",
                            "schedule"), v + [0] * (7 - len(v))))
        if a.layout == "nt":
            call = gf.prepare_gemm_f16_nt(A, B, C, cfg=cfg)
        else:
            a_km = a.layout == "tn"
            As = A.t().contiguous() if a_km else A
            Bs = B.t().contiguous()
            del A, B
            def call():
                gf.gemm_f16(As, Bs, C, a_km, True, cfg=cfg)
        for _ in range(a.iters):
            call()
    elif a.op == "gemv":
        Ws = [torch.from_numpy(inputs.uniform_f16((a.n, a.k), i, 0)).cuda() for i in range(5)]
        x = torch.from_numpy(inputs.uniform_f16((a.k,), 0, 1)).cuda()
        y = torch.empty((a.n,), dtype=torch.float16, device="cuda")
        calls = [gf.prepare_gemv_f16(w, x, y) for w in Ws]
        for i in range(a.iters):
            calls[i % len(calls)]()
    elif a.op == "splitk":
        A = torch.from_numpy(inputs.uniform_f16((1024, 16384), 0, 0)).cuda()
        B = torch.from_numpy(inputs.uniform_f16((1024, 16384), 0, 1)).cuda()
        As, Bs = [A] + [A.clone() for _ in range(3)], [B] + [B.clone() for _ in range(3)]
        C = torch.empty((1024, 1024), dtype=torch.float32, device="cuda")
        C16 = torch.empty((1024, 1024), dtype=torch.float16, device="cuda")
        ws = torch.empty(a.split * 1024 * 1024, dtype=torch.float32, device="cuda")
        for i in range(a.iters):
            j = i % 4
            gf.gemm_f16_nt_splitk_ex(As[j], Bs[j], C, a.split, gf.GF_SPLITK_ATOMIC, ws)
            gf.gemm_f16_nt_splitk_ex(As[j], Bs[j], C, a.split, gf.GF_SPLITK_TWOPASS, ws)
            gf.gemm_f16_nt_splitk_f16(As[j], Bs[j], C16, a.split, ws)
    elif a.op == "skinny":
        Bs = [torch.from_numpy(inputs.uniform_f16((a.n, a.k), i, 1)).cuda() for i in range(5)]
        for m in (4, 16):
            A = torch.from_numpy(inputs.uniform_f16((m, a.k), 0, 0)).cuda()
            C = torch.empty((m, a.n), dtype=torch.float16, device="cuda")
            for i in range(a.iters):
                gf.gemm_f16_nt(A, Bs[i % len(Bs)], C)
    elif a.op == "sparse":
        A = torch.from_numpy(inputs.uniform_f16((a.m, a.k), 0, 0)).cuda()
        B = torch.from_numpy(inputs.uniform_f16((a.n, a.k), 0, 1)).cuda()
        Asp, E = gf.sp24_compress_f16(A)
        del A
        C = torch.empty((a.m, a.n), dtype=torch.float16, device="cuda")
        call = gf.prepare_gemm_sp_f16_nt(Asp, E, B, C)
        for _ in range(a.iters):
            call()
    elif a.op == "compress":
        As = [torch.from_numpy(inputs.uniform_f16((a.m, a.k), i, 0)).cuda() for i in range(3)]
        outs = [(torch.empty((a.m, a.k // 2), dtype=torch.float16, device="cuda"),
                 torch.empty((a.m, a.k // 16), dtype=torch.int16, device="cuda")) for _ in range(3)]
        for i in range(a.iters):
            gf.sp24_compress_f16(As[i % 3], *outs[i % 3])
    elif a.op == "w4":
        Ws = [half(torch, i, 8192, 8192) for i in range(3)]
        outs = [gf.w4_quantize_f16(w) for w in Ws]
        for i in range(a.iters):
            Q, S, Z = outs[i % 3]
            gf.w4_quantize_f16(Ws[i % 3], Q=Q, S=S, Z=Z)
            gf.w4_dequantize_f16(Q, S, Z, W=Ws[i % 3])
        del Ws, outs
        for m, n, k, group, copies in ((1, 1024, 1024, 128, 64), (1, 8192, 8192, 128, 16), (24, 11008, 4096, 128, 24),
                                       (24, 11008, 4096, 64, 24), (2048, 8192, 4096, 128, 1)):
            w = [gf.w4_quantize_f16(half(torch, i, n, k), group, symmetric=group == 64) for i in range(copies)]
            A, C = half(torch, 99, m, k), torch.empty((m, n), dtype=torch.float16, device="cuda")
            for i in range(a.iters):
                gf.gemm_w4_f16_nt(A, *w[i % copies], C=C, group=group)
    elif a.op == "grouped":
        for rows, e, n, k, copies in ((48, 16, 4096, 2048, 3), (8191, 8, 4096, 4096, 1)):
            off, A = offsets(torch, rows, e), half(torch, 98, rows, k)
            Bs = [half(torch, i, e, n, k) for i in range(copies)]
            C = torch.empty((rows, n), dtype=torch.float16, device="cuda")
            for i in range(a.iters):
                gf.gemm_f16_grouped_nt(A, Bs[i % copies], off, C)
        for rows, e, n, k in ((4096, 8, 4096, 2048), (2999, 32, 1024, 2048)):
            off, A, B, D = offsets(torch, rows, e), half(torch, 97, rows, k), half(torch, 0, e, n, k), half(torch, 96, rows, n)
            dA = torch.empty_like(A)
            dBs = [torch.empty((e, n, k), dtype=t, device="cuda") for t in (torch.float32, torch.float16)]
            for _ in range(a.iters):
                gf.gemm_f16_grouped_nn(D, B, off, dA)
                for dB in dBs:
                    gf.gemm_f16_grouped_tn(D, A, off, dB)
        for rows, e, n, k, copies in ((24, 16, 4096, 4096, 3), (1111, 8, 2048, 4096, 3)):
            off, A = offsets(torch, rows, e), half(torch, 95, rows, k)
            w = [gf.w4_quantize_f16(half(torch, i, e, n, k)) for i in range(copies)]
            C = torch.empty((rows, n), dtype=torch.float16, device="cuda")
            for i in range(a.iters):
                gf.gemm_w4_f16_grouped_nt(A, *w[i % copies], off, C)
    else:
        src = torch.ones(128 << 20, dtype=torch.float32, device="cuda")   # 512 MiB
        dst = torch.empty_like(src)
        for _ in range(a.iters):
            dst.copy_(src)
    torch.cuda.synchronize()
    print("profile_run %s: %d iterations done" % (a.op, a.iters), flush=True)


if __name__ == "__main__":
    main()
