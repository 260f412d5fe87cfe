"""Measured cases of expert routing, of moving rows to experts and back, and of low-rank adapters.

Three operators, each in a plain form (elementary torch operations in fp32,
rounded once; scores in fp64, where a choice hangs on their last bits) and
through the library's calls (``own``):

* route  logits (T, E) -> the k experts of each token, their weights, the
         offsets of the experts' row groups and each (token, choice)'s row in
         the sorted order.  With `grad`: the weights' gradient to the logits'.
* rows   A[place[t][j]] = X[t], and Y[t] = sum_j w[t][j] C[place[t][j]].  With
         `grad`: the gradients of both, dX from dA, and dC and dw from dY.
* lora   C[m] = A[m] B^T + scale[a] (A[m] Down[a]^T) Up[a]^T with the adapter
         a = ids[m] of each row (none where it is -1); B in fp16, or in 4 bits
         (codes of 8 consecutive k in a word, lowest first, standing for
         (q - z) * s in groups of consecutive k).

Scores are softmax or sigmoid; the choice is by score + bias, in groups by the
sum of each group's best; an expert whose logit is -inf is never chosen, and
where fewer than k are left the id is -1 and the weight 0.
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
        # one token of one request: the latency of a call
        dict(name="route-token", kind="route", grad=False, T=1, E=64, k=8, f32=False, score="softmax", bias=False,
             groups=1, top_groups=1, group_best=1, renorm=True, scale=1.0, masked=0.0),
        # a decode batch, balanced by a bias, experts limited to the best groups
        dict(name="route-batch-96", kind="route", grad=False, T=96, E=256, k=8, f32=True, score="sigmoid", bias=True,
             groups=8, top_groups=4, group_best=2, renorm=True, scale=2.5, masked=0.0),
        # a long prompt, weights as the softmax gives them
        dict(name="route-prompt-8192", kind="route", grad=False, T=8192, E=128, k=8, f32=True, score="softmax",
             bias=False, groups=1, top_groups=1, group_best=1, renorm=False, scale=1.0, masked=0.0),
        # a training step's router gradient; an odd number of tokens, some experts masked out
        dict(name="route-grad-8191", kind="route", grad=True, T=8191, E=160, k=6, f32=False, score="softmax",
             bias=True, groups=8, top_groups=3, group_best=1, renorm=False, scale=1.0, masked=0.1),
        # a decode batch's rows to 8 experts each and back
        dict(name="rows-decode-16", kind="rows", grad=False, T=16, k=8, E=64, D=4096, masked=0.0),
        # a prompt's
        dict(name="rows-prompt-4096", kind="rows", grad=False, T=4096, k=8, E=64, D=2048, masked=0.0),
        # a training step's gradients, two experts a token
        dict(name="rows-grad-8191", kind="rows", grad=True, T=8191, k=2, E=8, D=4096, masked=0.0),
        # an odd small one: rows off the 16-byte grid, padding tokens that go nowhere
        dict(name="rows-grad-601", kind="rows", grad=True, T=601, k=5, E=33, D=1001, masked=0.1),
        # one token with its adapter: the latency of a decode step's projection
        dict(name="lora-token", kind="lora", M=1, N=4096, K=4096, r=16, L=8, none=0.0, bits=16),
        # a decode batch of many requests, a few without an adapter
        dict(name="lora-batch-32", kind="lora", M=32, N=8192, K=4096, r=32, L=24, none=0.1, bits=16),
        # prompts of a few requests together
        dict(name="lora-prompt-2048", kind="lora", M=2048, N=4096, K=4096, r=16, L=8, none=0.0, bits=16),
        # a decode batch beside 4-bit weights
        dict(name="lora-w4-batch-24", kind="lora", M=24, N=11008, K=4096, r=16, L=16, none=0.0, bits=4, group=64),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng: random.Random):
    kind = rng.choice(["route", "route", "rows", "lora", "lora"])
    limit = max(_cost(c) for c in listed() if c["kind"] == kind)
    while True:
        if kind == "route":
            groups = rng.choice([1, 1, 1, 2, 4, 8])
            E = groups * _log(rng, max(2, 8 // groups), 512 // groups)
            top = rng.randint(max(1, groups // 4), groups)
            k = rng.randint(1, min(12, E // groups * top))
            case = dict(kind=kind, grad=rng.random() < 0.3, T=_log(rng, 1, 8192), E=E, k=k, f32=rng.random() < 0.5,
                        score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                        top_groups=top, group_best=rng.choice([1, 2]), renorm=rng.random() < 0.6,
                        scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.0, 0.1, 0.9]))
            if case["T"] < 16:
                case["masked"] = 0.0
            if case["grad"] and case["renorm"]:      # a single renormalised weight has no gradient
                case.update(k=max(2, k), masked=min(case["masked"], 0.1))
        elif kind == "rows":
            case = dict(kind=kind, grad=rng.random() < 0.5, T=_log(rng, 1, 8192), k=rng.randint(1, 10),
                        E=_log(rng, 2, 256), D=_log(rng, 64, 8192), masked=rng.choice([0.0, 0.0, 0.1]))
            if rng.random() < 0.75:                  # most rows lie on the 16-byte grid
                case["D"] = max(64, case["D"] // 8 * 8)
        else:
            case = dict(kind=kind, M=_log(rng, 1, 2048), N=_log(rng, 256, 11008), K=_log(rng, 256, 8192, 8),
                        r=rng.choice([4, 8, 16, 16, 32, 64]), L=_log(rng, 1, 32), none=rng.choice([0.0, 0.1]),
                        bits=rng.choice([16, 16, 4]))
            if case["bits"] == 4:
                case["group"] = rng.choice([32, 64, 128])
        if _cost(case) <= limit:
            return case


def work(case):
    kind = case["kind"]
    if kind == "route":
        T, E, k, size = case["T"], case["E"], case["k"], 4 if case["f32"] else 2
        if case["grad"]:
            return {"bytes": 2 * T * E * size + 8 * T * k, "flops": 6 * T * E}
        return {"bytes": T * E * size + 12 * T * k + 4 * (E + 1) + (4 * E if case["bias"] else 0), "flops": 4 * T * E}
    if kind == "rows":
        T, k, D = case["T"], case["k"], case["D"]
        n = T * k - int(case["masked"] * T) * k
        if case["grad"]:
            return {"bytes": 2 * D * (2 * T + 3 * n) + 16 * T * k, "flops": 4 * n * D}
        return {"bytes": 2 * D * (2 * T + 2 * n) + 12 * T * k, "flops": 2 * n * D}
    M, N, K, r = case["M"], case["N"], case["K"], case["r"]
    live = M - int(case["none"] * M)
    base = 2 * N * K if case["bits"] == 16 else N * K // 2 + N * _groups(case) * 3
    return {"bytes": base + 2 * M * (K + N) + 2 * min(live, case["L"]) * r * (N + K) + 4 * M,
            "flops": 2 * M * N * K + 2 * live * r * (N + K)}


def _groups(case):
    return (case["K"] + case["group"] - 1) // case["group"]


def _cost(case):
    w = work(case)
    return w["flops"] / 1e15 + w["bytes"] / 5e12


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _inputs(case, seed):
    g = torch.Generator(device=_DEV).manual_seed(seed)

    def randn(*shape, scale=1.0, dtype=torch.float16):
        return (torch.randn(shape, generator=g, device=_DEV) * scale).to(dtype)

    def rand(*shape):
        return torch.rand(shape, generator=g, device=_DEV)

    if case["kind"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        dtype = torch.float32 if case["f32"] else torch.float16
        # some experts are wanted more than others
        x = (randn(T, E, scale=1.3, dtype=torch.float32) + randn(1, E, scale=0.5, dtype=torch.float32)).to(dtype)
        if case["masked"]:
            x = x.masked_fill(rand(T, E) < case["masked"], -math.inf)
            x[T // 2] = -math.inf                    # a padding token
        d = dict(x=x, bias=randn(E, scale=0.05, dtype=torch.float32) if case["bias"] else None)
        if case["grad"]:
            d["ids"] = _plain_choice(d["x"], d["bias"], case)[0].int()
            d["dw"] = randn(T, k, scale=0.1, dtype=torch.float32)
        return d
    if case["kind"] == "rows":
        T, k, E, D = case["T"], case["k"], case["E"], case["D"]
        if k <= E:                                   # k different experts a token, as a router gives them
            ids = rand(T, E).argsort(1)[:, :k].int()
        else:
            ids = (rand(T, k) * E).int()
        gone = rand(T).argsort()[: int(case["masked"] * T)]
        ids[gone] = -1
        place = _plain_rows(ids, E)[1]
        d = dict(place=place, w=rand(T, k) / k)
        n = T * k
        if case["grad"]:
            d.update(dA=randn(n, D), dY=randn(T, D), C=randn(n, D), dC=torch.zeros((n, D), dtype=torch.float16, device=_DEV))
        else:
            d.update(X=randn(T, D), C=randn(n, D), A=torch.zeros((n, D), dtype=torch.float16, device=_DEV))
        return d
    M, N, K, r, L = (case[n] for n in ("M", "N", "K", "r", "L"))
    # rows of a request lie together; a decode batch has one row of each
    runs = min(M, L)
    ids = torch.div(torch.arange(M, device=_DEV) * runs, M, rounding_mode="floor")
    ids = rand(L).argsort()[:runs][ids].int()
    if M <= 64:
        ids = ids[rand(M).argsort()]
    ids[rand(M).argsort()[: int(case["none"] * M)]] = -1
    d = dict(A=randn(M, K), ids=ids, Down=randn(L, r, K, scale=1.0 / math.sqrt(K)), Up=randn(L, N, r, scale=0.25),
             scales=rand(L) + 0.5)
    if case["bits"] == 16:
        d["B"] = randn(N, K, scale=1.0 / math.sqrt(K))
    else:
        # bell-shaped codes, zero points about 8
        q = (torch.randn((N, K // 8, 8), generator=g, device=_DEV) * 2.7 + 8.0).round_().clamp_(0, 15).to(torch.int32)
        d["Q"] = (q << torch.arange(0, 32, 4, device=_DEV, dtype=torch.int32)).sum(2, dtype=torch.int32)
        d["S"] = ((rand(N, _groups(case)) + 0.5) / (2.7 * math.sqrt(K))).half()
        d["Z"] = torch.randint(5, 12, (N, _groups(case)), generator=g, device=_DEV).to(torch.uint8)
    return d


def prepare(case, seed):
    return dict(_inputs(case, seed), case=case)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import gemv_fp16_amd as gf
    case = s["case"]
    if case["kind"] == "route":
        if case["grad"]:
            return gf.route_topk_bwd(s["x"], s["ids"], s["dw"], score=case["score"], renorm=case["renorm"],
                                     scale=case["scale"])
        ids, w, offsets, place = gf.route_topk(
            s["x"], case["k"], bias=s["bias"], score=case["score"], groups=case["groups"],
            top_groups=case["top_groups"], group_best=case["group_best"], renorm=case["renorm"], scale=case["scale"])
        return [ids, w, offsets, place]
    if case["kind"] == "rows":
        if case["grad"]:
            dC, dw = gf.combine_f16_bwd(s["dY"], s["C"], s["place"], s["w"], dC=s["dC"])
            return [gf.combine_f16(s["dA"], s["place"]), dC, dw]
        return [gf.dispatch_f16(s["X"], s["place"], A=s["A"]), gf.combine_f16(s["C"], s["place"], s["w"])]
    if case["bits"] == 16:
        return gf.gemm_f16_nt_lora(s["A"], s["B"], s["ids"], s["Down"], s["Up"], s["scales"])
    C = gf.gemm_w4_f16_nt(s["A"], s["Q"], s["S"], s["Z"], group=case["group"], out_f32=True)   # rounded once, below
    return gf.lora_add_f16(s["A"], s["ids"], s["Down"], s["Up"], C, s["scales"])


def _plain_choice(x, bias, case):
    """The chosen experts (-1: none), and all scores, in fp64."""
    x = x.double()
    out = x == -math.inf
    if case["score"] == "softmax":
        top = x.amax(1, keepdim=True).clamp(min=-1e300)
        e = torch.exp(x - top)
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    by = x if bias is None and not (case["groups"] > 1 and case["group_best"] == 2) else s
    if bias is not None:
        by = s + bias.double()
    by = by.masked_fill(out, -math.inf)
    T, E = x.shape
    if case["groups"] > 1:
        per = by.view(T, case["groups"], -1)
        best = per.sort(dim=2, descending=True).values[:, :, : case["group_best"]]
        if case["group_best"] == 2:                  # a group with one expert left counts it alone
            best = torch.cat([best[:, :, :1], best[:, :, 1:].masked_fill(best[:, :, 1:] == -math.inf, 0.0)], 2)
        order = best.sum(2).sort(dim=1, descending=True, stable=True).indices[:, : case["top_groups"]]
        stay = torch.zeros((T, case["groups"]), dtype=torch.bool, device=x.device).scatter_(1, order, True)
        by = per.masked_fill(~stay.unsqueeze(2), -math.inf).view(T, E)
    val, ids = by.sort(dim=1, descending=True, stable=True)
    val, ids = val[:, : case["k"]], ids[:, : case["k"]]
    return ids.masked_fill(val == -math.inf, -1), s


def _plain_rows(ids, E):
    """Offsets of the experts' groups, and each entry's place in the order sorted by expert."""
    flat = ids.reshape(-1).long()
    count = torch.bincount(flat + 1, minlength=E + 1)
    offsets = count.cumsum(0) - count[0]
    order = flat.sort(stable=True).indices
    place = torch.empty_like(flat)
    place[order] = torch.arange(flat.numel(), device=flat.device) - count[0]
    return offsets.int(), place.clamp(min=-1).masked_fill(flat < 0, -1).int().view(ids.shape)


def _plain(s):
    case = s["case"]
    if case["kind"] == "route":
        if case["grad"]:
            return _plain_route_grad(s, case)
        ids, score = _plain_choice(s["x"], s["bias"], case)
        w = score.gather(1, ids.clamp(min=0)).masked_fill(ids < 0, 0.0)
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        return [ids.int(), (w * case["scale"]).float(), *_plain_rows(ids, case["E"])]
    if case["kind"] == "rows":
        place = s["place"].long()
        live = (place >= 0).unsqueeze(2)
        at = place.clamp(min=0)
        if case["grad"]:
            zero = torch.zeros((), device=_DEV)
            dX = torch.where(live, s["dA"].float()[at], zero).sum(1).half()
            dY = s["dY"].float().unsqueeze(1)
            dw = (torch.where(live, s["C"].float()[at], zero) * dY).sum(2)
            dC = s["dC"]
            keep = place >= 0
            dC[place[keep]] = (s["w"].unsqueeze(2) * dY).half()[keep]
            return [dX, dC, dw]
        A = s["A"]
        t, j = torch.where(place >= 0)
        A[place[t, j]] = s["X"][t]
        w = s["w"].masked_fill(place < 0, 0.0).unsqueeze(2)
        return [A, (s["C"].float()[at] * w).sum(1).half()]
    # adapters: all of them side by side, each row's own kept
    L, r, K = s["Down"].shape
    A = s["A"].float()
    mine = (s["ids"].unsqueeze(1) == torch.arange(L, device=_DEV)).float() * s["scales"]
    H = (A @ s["Down"].float().view(L * r, K).t()).view(-1, L, r) * mine.unsqueeze(2)
    low = H.view(-1, L * r) @ s["Up"].float().transpose(1, 2).reshape(L * r, -1)
    if case["bits"] == 16:
        B = s["B"].float()
    else:
        shift = torch.arange(0, 32, 4, device=_DEV, dtype=torch.int32)
        B = ((s["Q"].unsqueeze(2) >> shift) & 15).flatten(1).float()
        B = (B - s["Z"].float().repeat_interleave(case["group"], 1)[:, :K]) * \
            s["S"].float().repeat_interleave(case["group"], 1)[:, :K]
    return (A @ B.t() + low).half()


def _plain_route_grad(s, case):
    x, ids, dw = s["x"].float(), s["ids"].long(), s["dw"] * case["scale"]
    live, at = ids >= 0, ids.clamp(min=0)
    dw = dw.masked_fill(~live, 0.0)
    xs = x.gather(1, at).masked_fill(~live, -math.inf)
    zero = torch.zeros_like(x)
    if case["score"] == "softmax":
        if not case["renorm"]:
            e = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e30))
            p = e / e.sum(1, keepdim=True).clamp(min=1e-30)
            g = zero.scatter_add(1, at, dw)
            dx = p * (g - (g * p).sum(1, keepdim=True))
            return dx.to(s["x"].dtype)
        e = torch.exp(xs - xs.amax(1, keepdim=True).clamp(min=-1e30))
        share = e / e.sum(1, keepdim=True).clamp(min=1e-30)
        d = share * (dw - (share * dw).sum(1, keepdim=True))
    else:
        sig = 1.0 / (1.0 + torch.exp(-xs))
        if case["renorm"]:
            share = sig / sig.sum(1, keepdim=True).clamp(min=1e-30)
            d = share * (1.0 - sig) * (dw - (share * dw).sum(1, keepdim=True))
        else:
            d = sig * (1.0 - sig) * dw
    return zero.scatter_add(1, at, d.masked_fill(~live, 0.0)).to(s["x"].dtype)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the plain form
# ---------------------------------------------------------------------------

def exact(case, seed):
    d = _inputs(case, seed)
    if case["kind"] == "route":
        return _exact_route_grad(d, case) if case["grad"] else _exact_route(d, case)
    if case["kind"] == "rows":
        place, w = d["place"].long(), d["w"].double()
        T, k = place.shape
        n, D = d["C"].shape
        token = torch.full((n + 1,), T, device=_DEV)             # of each sorted row; T: none
        slot = torch.zeros((n + 1,), dtype=torch.long, device=_DEV)
        flat = torch.where(place < 0, n, place).view(-1)
        token[flat] = torch.arange(T, device=_DEV).repeat_interleave(k)
        slot[flat] = torch.arange(k, device=_DEV).repeat(T)
        token, slot = token[:n], slot[:n]
        held = token < T

        def rows(X):                                             # one row of X for each sorted row
            return torch.cat([X, X.new_zeros((1, D))])[token]

        def back(R):                                             # sorted rows summed by token
            return torch.zeros((T + 1, D), dtype=torch.float64, device=_DEV).index_add_(0, token, R)[:T]

        share = torch.where(held, w[token.clamp(max=T - 1), slot], 0.0)[:, None]
        if not case["grad"]:
            return [rows(d["X"].double()), back(d["C"].double() * share)]
        dY = rows(d["dY"].double())
        dw = torch.zeros((T + 1, k), dtype=torch.float64, device=_DEV)
        dw[token, slot] = (dY * d["C"].double()).sum(1)
        return [back(d["dA"].double()), dY * share, dw[:T]]
    A, ids = d["A"].double(), d["ids"]
    K = A.shape[1]
    if case["bits"] == 16:
        B = d["B"].double()
    else:
        B = torch.empty((case["N"], K), dtype=torch.float64, device=_DEV)
        for i in range(8):                                       # code i of every word
            B[:, i::8] = ((d["Q"] >> (4 * i)) & 15).double()
        for g in range(d["S"].shape[1]):
            part = B[:, g * case["group"]:(g + 1) * case["group"]]
            part -= d["Z"][:, g:g + 1].double()
            part *= d["S"][:, g:g + 1].double()
    C = A @ B.t()
    for a in range(case["L"]):
        m = torch.where(ids == a)[0]
        if len(m):
            C[m] += d["scales"][a].double() * ((A[m] @ d["Down"][a].double().t()) @ d["Up"][a].double().t())
    return C


def _exact_scores(x, case):
    if case["score"] == "sigmoid":
        return torch.special.expit(x)
    return torch.nan_to_num(torch.softmax(x, 1))                 # a row with nothing left: zeros


def _exact_route(d, case):
    x = d["x"].double()
    T, E = x.shape
    s = _exact_scores(x, case)
    rank = s if d["bias"] is None else s + d["bias"].double()
    open_ = x > -math.inf
    if case["groups"] > 1:
        G = case["groups"]
        part = torch.where(open_, rank, -math.inf).view(T, G, E // G)
        some = open_.view(T, G, E // G).sum(2)
        first = part.max(2)
        total = first.values.clone()
        if case["group_best"] == 2:
            second = part.scatter(2, first.indices.unsqueeze(2), -math.inf).max(2).values
            total = torch.where(some > 1, total + second, total)
        for _ in range(G - case["top_groups"]):                  # close the worst group, the last of equal ones
            closed = torch.isnan(total)
            low = torch.where(closed, math.inf, total).min(1, keepdim=True).values
            at = G - 1 - (torch.where(closed, math.inf, total) == low).flip(1).int().argmax(1)
            total[torch.arange(T, device=_DEV), at] = math.nan
        open_ = open_ & (~torch.isnan(total)).repeat_interleave(E // G, 1)
    if d["bias"] is None and not (case["groups"] > 1 and case["group_best"] == 2):
        rank = x
    ids = torch.full((T, case["k"]), -1, dtype=torch.int64, device=_DEV)
    w = torch.zeros((T, case["k"]), dtype=torch.float64, device=_DEV)
    left = torch.where(open_, rank, -math.inf)
    row = torch.arange(T, device=_DEV)
    for j in range(case["k"]):
        best = left.max(1, keepdim=True).values
        at = (left == best).int().argmax(1)                      # the first of equal ones
        some = best[:, 0] > -math.inf
        ids[:, j] = torch.where(some, at, ids[:, j])
        w[:, j] = torch.where(some, s[row, at], w[:, j])
        left[row, at] = -math.inf
    if case["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True))
    hit = torch.nn.functional.one_hot(ids.view(-1) + 1, E + 1)[:, 1:]
    count = hit.sum(0)
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    earlier = ((hit.cumsum(0) - hit) * hit).sum(1).view(ids.shape)
    place = torch.where(ids < 0, -1, offsets[ids.clamp(min=0)] + earlier)
    return [ids.int(), w * case["scale"], offsets.int(), place.int()]


def _exact_route_grad(d, case):
    """Through the weights' own definition, differentiated by autograd in 64 bits."""
    x = d["x"].double()
    shut = x == -math.inf
    leaf = x.masked_fill(shut, 0.0).requires_grad_()
    ids = d["ids"].long()
    live = ids >= 0
    if case["score"] == "sigmoid":
        s = torch.special.expit(leaf)
    else:
        e = torch.exp(leaf - leaf.detach().amax(1, keepdim=True)) * (~shut)
        s = e / (e.sum(1, keepdim=True) + shut.all(1, keepdim=True))
    w = s.gather(1, ids.clamp(min=0)) * live
    if case["renorm"]:
        w = w / (w.sum(1, keepdim=True) + ~live.any(1, keepdim=True))
    (w * case["scale"] * d["dw"].double()).sum().backward()
    return leaf.grad
