"""Measured cases of the 4-bit weight and grouped (per expert) products.

Five operators, each in a plain form (elementary torch operations in fp32,
rounded once) and through the library's calls (``own``):

* quantize   W (N, K) fp16 -> 4-bit codes, a scale and a zero point per group of
             consecutive k, and back: S, Z and the weights the codes stand for.
* w4         C = A . dequantize(Q, S, Z)^T, M rows of A from one token to a prompt.
* grouped    C[r] = A[r] . B[e]^T for the rows r of group e, rows sorted by group.
* backward   the gradients of that product: dA[r] = dC[r] . B[e] and
             dB[e] = sum over the rows of group e of dC[r]^T A[r] (fp32).
* w4_grouped the grouped product with 4-bit weights.

Codes: word j of a row of Q holds k = 8 j .. 8 j + 7, four bits each, lowest
first.  Group g of row n is k = g * group .. and stands for (q - z) * s with
s = S[n][g] and z = Z[n][g], or z = 8 where there is no Z.
"""
from __future__ import annotations

import math
import random

import torch

own = False

_DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token through a small projection: the latency of a call
        dict(name="w4-token-1024", kind="w4", M=1, N=1024, K=1024, group=128, zeros=True),
        # one token through a large projection: the weights' bytes
        dict(name="w4-token-8192", kind="w4", M=1, N=8192, K=8192, group=128, zeros=True),
        # a decode batch, symmetric codes in shorter groups
        dict(name="w4-batch-24", kind="w4", M=24, N=11008, K=4096, group=64, zeros=False),
        # a prompt against the same kind of weights
        dict(name="w4-prompt-2048", kind="w4", M=2048, N=8192, K=4096, group=128, zeros=True),
        # a checkpoint's large matrix quantized at load, and its check against the original
        dict(name="quantize-8192", kind="quantize", N=8192, K=8192, group=128, zeros=True),
        # an odd small one: a last group that is cut short, rows off the 16-byte grid
        dict(name="quantize-1001x2056", kind="quantize", N=1001, K=2056, group=32, zeros=False),
        # a decode batch routed to 16 experts, two of them without a row
        dict(name="grouped-decode-48", kind="grouped", E=16, T=48, N=4096, K=2048, empty=2),
        # a long prompt over 8 experts, uneven
        dict(name="grouped-prompt-8191", kind="grouped", E=8, T=8191, N=4096, K=4096, empty=0),
        # the gradients of a training step's expert layer
        dict(name="backward-4096", kind="backward", E=8, T=4096, N=4096, K=2048, empty=0),
        # many small experts, short ragged groups, three empty
        dict(name="backward-2999x32", kind="backward", E=32, T=2999, N=1024, K=2048, empty=3),
        # 4-bit experts: a decode batch
        dict(name="w4-grouped-decode-24", kind="w4_grouped", E=16, T=24, N=4096, K=4096, group=128, zeros=True,
             empty=3),
        # 4-bit experts: a short prompt
        dict(name="w4-grouped-prompt-1111", kind="w4_grouped", E=8, T=1111, N=2048, K=4096, group=64, zeros=False,
             empty=1),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng: random.Random):
    kind = rng.choice(["w4", "w4", "quantize", "grouped", "backward", "w4_grouped"])
    limit = max(_cost(c) for c in listed() if c["kind"] == kind)
    while True:
        case = dict(kind=kind)
        if kind in ("w4", "quantize"):
            case.update(N=_log(rng, 256, 16384), K=_log(rng, 256, 16384, 8))
            if kind == "w4":
                case["M"] = _log(rng, 1, 2048)
        else:
            case.update(E=_log(rng, 2, 64), T=_log(rng, 2, 8192), N=_log(rng, 256, 8192, 8),
                        K=_log(rng, 256, 8192, 8))
            case["empty"] = rng.randrange(0, max(1, case["E"] // 4))
            if case["E"] * case["N"] * case["K"] > 1 << 29:
                continue
            case["empty"] = max(case["empty"], case["E"] - case["T"])
        if kind in ("w4", "quantize", "w4_grouped"):
            case.update(group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5)
            if rng.random() < 0.75:                  # most rows lie on the 16-byte grid
                case["K"] = max(256, case["K"] // 32 * 32)
        if _cost(case) <= limit:
            return case


def _groups(case):
    return (case["K"] + case["group"] - 1) // case["group"]


def work(case):
    kind, N, K = case["kind"], case["N"], case["K"]
    if kind in ("w4", "quantize", "w4_grouped"):
        packed = N * K // 2 + N * _groups(case) * (3 if case["zeros"] else 2)
    if kind == "w4":
        M = case["M"]
        return {"bytes": packed + 2 * M * K + 2 * M * N, "flops": 2 * M * N * K}
    if kind == "quantize":
        return {"bytes": 4 * N * K + packed, "flops": 6 * N * K}
    T, used = case["T"], case["E"] - case["empty"]
    if kind == "grouped":
        return {"bytes": 2 * T * K + 2 * T * N + 2 * used * N * K, "flops": 2 * T * N * K}
    if kind == "backward":
        return {"bytes": 4 * T * K + 2 * T * N + 2 * used * N * K + 4 * case["E"] * N * K, "flops": 4 * T * N * K}
    return {"bytes": 2 * T * K + 2 * T * N + used * packed, "flops": 2 * T * N * K}


def _cost(case):
    w = work(case)
    return w["flops"] / 1e15 + w["bytes"] / 5e12


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=_DEV).manual_seed(seed)


def _randn(g, shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=_DEV) * scale).half()


def _sizes(case, seed):
    """Rows of each group: uneven, `empty` of them without any, T in all."""
    rng = random.Random(seed * 1000003 + 17)
    E, T, empty = case["E"], case["T"], case["empty"]
    used = rng.sample(range(E), E - empty)
    share = [rng.expovariate(1.0) + 0.1 for _ in used]
    total, sizes = sum(share), [0] * E
    for e, s in zip(used, share):
        sizes[e] = 1 + int((T - len(used)) * s / total)
    rest = T - sum(sizes)
    for i in range(rest):
        sizes[used[i % len(used)]] += 1
    return sizes


def _codes(g, rows, K, group, zeros):
    """Bell-shaped 4-bit codes, scales of a few hundredths, zero points about 8."""
    G = (K + group - 1) // group
    q = (torch.randn((rows, K), generator=g, device=_DEV) * 2.7 + 8.0).round_().clamp_(0, 15).to(torch.int32)
    shift = torch.arange(0, 32, 4, device=_DEV, dtype=torch.int32)
    words = torch.zeros((rows, K // 8), dtype=torch.int32, device=_DEV)
    q = q.view(rows, K // 8, 8)
    for i in range(8):
        words |= q[:, :, i] << shift[i]
    S = (torch.rand((rows, G), generator=g, device=_DEV) * 0.01 + 0.005).half()
    Z = None
    if zeros:
        Z = torch.randint(5, 12, (rows, G), generator=g, device=_DEV).to(torch.uint8)
    return words, S, Z


def _inputs(case, seed):
    g, kind, N, K = _gen(seed), case["kind"], case["N"], case["K"]
    if kind == "quantize":
        # weights of a layer: rows of different spread
        spread = torch.rand((N, 1), generator=g, device=_DEV) * 0.03 + 0.01
        return dict(W=(torch.randn((N, K), generator=g, device=_DEV) * spread).half())
    if kind == "w4":
        Q, S, Z = _codes(g, N, K, case["group"], case["zeros"])
        return dict(A=_randn(g, (case["M"], K)), Q=Q, S=S, Z=Z)
    sizes = _sizes(case, seed)
    ends = [0]
    for n in sizes:
        ends.append(ends[-1] + n)
    d = dict(sizes=sizes, offsets=torch.tensor(ends, dtype=torch.int32, device=_DEV), A=_randn(g, (case["T"], K)))
    E = case["E"]
    if kind == "w4_grouped":
        Q, S, Z = _codes(g, E * N, K, case["group"], case["zeros"])
        d.update(Q=Q.view(E, N, -1), S=S.view(E, N, -1), Z=None if Z is None else Z.view(E, N, -1))
    else:
        d["B"] = _randn(g, (E, N, K), 1.0 / math.sqrt(K))
    if kind == "backward":
        d["dC"] = _randn(g, (case["T"], N))
    return d


def prepare(case, seed):
    return dict(_inputs(case, seed), case=case)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return _own(state) if own else _plain(state)


def _own(state):
    import gemv_fp16_amd as gf
    case = state["case"]
    kind = case["kind"]
    if kind == "w4":
        if case["M"] == 1:
            return gf.gemv_w4_f16(state["Q"], state["S"], state["Z"], state["A"].view(-1),
                                  group=case["group"]).view(1, -1)
        return gf.gemm_w4_f16_nt(state["A"], state["Q"], state["S"], state["Z"], group=case["group"])
    if kind == "quantize":
        Q, S, Z = gf.w4_quantize_f16(state["W"], group=case["group"], symmetric=not case["zeros"])
        W = gf.w4_dequantize_f16(Q, S, Z, group=case["group"])
        return [S, W] if Z is None else [S, W, Z]
    if kind == "grouped":
        return gf.gemm_f16_grouped_nt(state["A"], state["B"], state["offsets"])
    if kind == "backward":
        return [gf.gemm_f16_grouped_nn(state["dC"], state["B"], state["offsets"]),
                gf.gemm_f16_grouped_tn(state["dC"], state["A"], state["offsets"], out_f32=True)]
    return gf.gemm_w4_f16_grouped_nt(state["A"], state["Q"], state["S"], state["Z"], state["offsets"],
                                     group=case["group"])


def _spread(t, group, K):
    """One entry per group -> one per k."""
    return t.repeat_interleave(group, dim=-1)[..., :K]


def _weights(Q, S, Z, group, K):
    """The fp32 weights that codes, scales and zero points stand for."""
    shift = torch.arange(0, 32, 4, device=Q.device, dtype=torch.int32)
    q = ((Q.unsqueeze(-1) >> shift) & 15).flatten(-2).float()
    z = 8.0 if Z is None else _spread(Z.float(), group, K)
    return (q - z) * _spread(S.float(), group, K)


def _plain(state):
    case = state["case"]
    kind, K = case["kind"], case["K"]
    if kind == "w4":
        return (state["A"].float() @ _weights(state["Q"], state["S"], state["Z"], case["group"], K).t()).half()
    if kind == "quantize":
        return _plain_quantize(state["W"], case["group"], case["zeros"])
    bounds, at = [], 0
    for e, n in enumerate(state["sizes"]):
        if n:
            bounds.append((e, at, at + n))
        at += n
    A = state["A"].float()
    if kind == "backward":
        dC = state["dC"].float()
        dA = torch.empty_like(A)
        dB = torch.zeros(state["B"].shape, dtype=torch.float32, device=A.device)
        for e, lo, hi in bounds:
            torch.matmul(dC[lo:hi], state["B"][e].float(), out=dA[lo:hi])
            torch.matmul(dC[lo:hi].t(), A[lo:hi], out=dB[e])
        return [dA.half(), dB]
    C = torch.empty((case["T"], case["N"]), dtype=torch.float32, device=A.device)
    for e, lo, hi in bounds:
        if kind == "grouped":
            B = state["B"][e].float()
        else:
            Z = state["Z"]
            B = _weights(state["Q"][e], state["S"][e], None if Z is None else Z[e], case["group"], K)
        torch.matmul(A[lo:hi], B.t(), out=C[lo:hi])
    return C.half()


def _plain_quantize(W, group, zeros):
    N, K = W.shape
    G = (K + group - 1) // group
    w = torch.nn.functional.pad(W.float(), (0, G * group - K)).view(N, G, group)
    # Quotients in 64 bits: a code changes at a tie, where an inexact one would decide it.
    if zeros:
        lo, hi = w.amin(2).clamp(max=0.0), w.amax(2).clamp(min=0.0)
        S = ((hi - lo).double() / 15.0).float().half()
    else:
        S = (w.abs().amax(2).double() / 7.0).float().half()
    s = S.double().unsqueeze(2)
    live = s > 0
    safe = torch.where(live, s, torch.ones_like(s))
    if zeros:
        z = torch.where(live, (-lo.double().unsqueeze(2) / safe).round().clamp(0, 15), torch.zeros_like(s))
    else:
        z = torch.full_like(s, 8.0)
    q = ((w.double() / safe).round() + z).clamp(0, 15)
    q = torch.where(live, q, z)
    back = ((q - z).float() * S.float().unsqueeze(2)).half().view(N, G * group)[:, :K].contiguous()
    return [S, back, z.squeeze(2).to(torch.uint8)] if zeros else [S, back]


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain form
# ---------------------------------------------------------------------------

def exact(case, seed):
    d, kind, K = _inputs(case, seed), case["kind"], case["K"]
    if kind == "quantize":
        return _exact_quantize(d["W"].double(), case["group"], case["zeros"])

    def weights(Q, S, Z):
        w = torch.empty((Q.shape[0], K), dtype=torch.float64, device=Q.device)
        for i in range(8):                            # code i of every word
            w[:, i::8] = ((Q >> (4 * i)) & 15).double()
        for g in range(S.shape[1]):
            part = w[:, g * case["group"]:(g + 1) * case["group"]]
            part -= 8.0 if Z is None else Z[:, g:g + 1].double()
            part *= S[:, g:g + 1].double()
        return w

    if kind == "w4":
        return d["A"].double() @ weights(d["Q"], d["S"], d["Z"]).t()
    off = d["offsets"].tolist()
    A = d["A"].double()
    if kind == "backward":
        dC = d["dC"].double()
        dA = torch.cat([dC[off[e]:off[e + 1]] @ d["B"][e].double() for e in range(case["E"])])
        dB = torch.stack([dC[off[e]:off[e + 1]].t() @ A[off[e]:off[e + 1]] for e in range(case["E"])])
        return [dA, dB]
    rows = []
    for e in range(case["E"]):
        if off[e] == off[e + 1]:
            continue
        B = d["B"][e].double() if kind == "grouped" else weights(
            d["Q"][e], d["S"][e], None if d["Z"] is None else d["Z"][e])
        rows.append(A[off[e]:off[e + 1]] @ B.t())
    return torch.cat(rows)


def _exact_quantize(W, group, zeros):
    N, K = W.shape
    scales, codes, points = [], torch.empty_like(W), []
    for k0 in range(0, K, group):
        w = W[:, k0:k0 + group]
        top, low = w.max(1).values, w.min(1).values
        if zeros:
            top, low = torch.maximum(top, torch.zeros_like(top)), torch.minimum(low, torch.zeros_like(low))
            s64 = (top - low) / 15.0
        else:
            s64 = torch.maximum(top, -low) / 7.0
        s = s64.float().half().double()               # the scale that is stored
        some = s != 0
        s1 = s + (~some).double()
        z = torch.round(-low / s1) if zeros else torch.full_like(s, 8.0)
        z = torch.where(some, z, torch.zeros_like(z) if zeros else z)
        q = torch.clamp(torch.round(w / s1[:, None]) + z[:, None], 0, 15)
        q = torch.where(some[:, None], q, z[:, None].expand_as(q))
        codes[:, k0:k0 + group] = (q - z[:, None]) * s[:, None]
        scales.append(s64)
        points.append(z)
    out = [torch.stack(scales, 1), codes]
    return out + [torch.stack(points, 1).to(torch.uint8)] if zeros else out
