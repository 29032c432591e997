"""Cases of the MoE layer's operators: the router and its gradient, the gradients of
dispatch and combine, and the experts' products with 4-bit weights.

``run`` computes an operator in its plain form (elementary torch operations), or,
where ``own`` is set, through the framework's entry points.  ``exact`` computes the
same outputs from the definitions in 64 bits.

Notation: T tokens, H hidden size, E experts, K slots per token, R receive rows;
``dst_row`` [T, K] is the receive row of each slot, -1 where it has none.
"""
from __future__ import annotations

import math

import torch

own = False

FLT_MAX = 3.4028234663852886e38


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------

def listed():
    return [
        # One decode batch through a router with sigmoid scores, a load-balancing bias
        # and 4 of 8 expert groups: the smallest call, where latency counts.
        dict(name="route decode", op="route", T=128, E=256, K=8, dtype="fp32", score="sigmoid",
             groups=8, topk_groups=4, bias=True, normalize=True, scale=2.5, masked=0.0),
        # A prefill batch of the same router, a few tokens of it padding.
        dict(name="route prefill", op="route", T=4096, E=256, K=8, dtype="fp32",
             score="sigmoid", groups=8, topk_groups=4, bias=True, normalize=True, scale=2.5,
             masked=0.03),
        # A training batch of a softmax router with bf16 logits and an odd expert count.
        dict(name="route softmax bf16", op="route", T=16383, E=160, K=6, dtype="bf16",
             score="softmax", groups=1, topk_groups=1, bias=False, normalize=False, scale=1.0,
             masked=0.0),
        # The gradient of a softmax router that does not renormalise: dense over the experts.
        dict(name="route backward dense", op="route_backward", T=4096, E=256, K=8, dtype="fp32",
             score="softmax", normalize=False, scale=1.0, masked=0.03),
        # The gradient of a renormalising top-2 router over few experts, many tokens.
        dict(name="route backward top2", op="route_backward", T=32768, E=8, K=2, dtype="bf16",
             score="softmax", normalize=True, scale=1.0, masked=0.0),
        # Training step, 4096 tokens of a wide top-8 layer: the largest case.
        dict(name="combine backward top8", op="combine_backward", T=4096, H=7168, E=256, K=8,
             masked=0.0),
        # Odd token count and width, padded tokens and dropped slots.
        dict(name="combine backward ragged", op="combine_backward", T=1003, H=1032, E=40, K=6,
             masked=0.1),
        # Training step of the wide top-8 layer, back through dispatch.
        dict(name="dispatch backward top8", op="dispatch_backward", T=4096, H=7168, E=256, K=8,
             masked=0.0),
        # Coarse experts: many tokens, top-2, some slots dropped.
        dict(name="dispatch backward top2", op="dispatch_backward", T=32767, H=2048, E=8, K=2,
             masked=0.05),
        # One token in decode: its 8 experts among this GPU's 32, down projection, bf16 rows.
        dict(name="w4 one token down", op="w4", E=32, C=4, rows=8, I=2048, N=7168, G=128,
             x="bf16", zeros=False, act=False, offsets=False),
        # 128 rows over this GPU's 32 experts, FP8 rows as the decode dispatch writes them,
        # gate and up projection with the activation behind them.
        dict(name="w4 decode gate up", op="w4", E=32, C=32, rows=128, I=7168, N=2048, G=128,
             x="fp8", zeros=False, act=True, offsets=False),
        # A prefill chunk over contiguous expert runs: uneven runs, small groups, zero points.
        dict(name="w4 ragged zeros", op="w4", E=12, C=160, rows=500, I=1440, N=1000, G=32,
             x="bf16", zeros=True, act=False, offsets=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "combine_backward", "dispatch_backward", "w4",
                     "w4"])
    masked = rng.choice([0.0, 0.02, 0.2])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _log(rng, 2, 256 // groups) if groups > 1 else _log(rng, 4, 512)
        tg = 1 if groups == 1 else rng.randint(1, groups)
        K = rng.randint(1, min(10, E // groups * tg))
        T = min(_log(rng, 1, 32768), (1 << 23) // E)
        case = dict(op=op, T=T, E=E, K=K, dtype=rng.choice(["fp32", "bf16"]),
                    score=rng.choice(["sigmoid", "softmax"]), normalize=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), masked=masked)
        if op == "route":
            case.update(groups=groups, topk_groups=tg, bias=rng.random() < 0.5)
        return case
    if op in ("combine_backward", "dispatch_backward"):
        K = rng.choice([1, 2, 3, 4, 6, 8, 10])
        H = 8 * _log(rng, 16, 1024)
        T = min(_log(rng, 1, 32768), 200_000_000 // (K * H))
        return dict(op=op, T=T, H=H, E=_log(rng, max(K, 4), 256), K=K, masked=masked)
    fp8 = rng.random() < 0.5
    G = rng.choice([32, 64, 128])
    step = 128 if fp8 else G
    I = step * _log(rng, max(1, 256 // step), 7168 // step)
    N = 8 * _log(rng, 16, 896)
    act = rng.random() < 0.5
    E = max(1, min(_log(rng, 1, 64), 900_000_000 // (I * N * (2 if act else 1))))
    rows = _log(rng, 1, 256)
    return dict(op="w4", E=E, C=min(rows, 8 + 4 * (rows // E)), rows=rows, I=I, N=N, G=G,
                x="fp8" if fp8 else "bf16", zeros=rng.random() < 0.5, act=act,
                offsets=rng.random() < 0.5)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 11)
    return g


def _logits(case, g):
    """Router logits; a masked share of the tokens is padding (every logit -inf), and as
    large a share of the rest has one expert that must not be taken."""
    T, E = case["T"], case["E"]
    l = torch.randn((T, E), device="cuda", generator=g) * 1.5
    if case["masked"]:
        u = torch.rand(T, device="cuda", generator=g)
        l[u < case["masked"]] = -math.inf
        one = torch.randint(0, E, (T,), device="cuda", generator=g)
        hit = (torch.rand(T, device="cuda", generator=g) < case["masked"]).nonzero()[:, 0]
        l[hit, one[hit]] = -math.inf
    return l.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)


def _routing(case, g):
    """dst_row [T, K] as dispatch numbers the rows (by expert, then token and slot) and the
    gate weights; a masked share of the slots, and of the tokens, has no row."""
    T, E, K = case["T"], case["E"], case["K"]
    idx = torch.rand((T, E), device="cuda", generator=g).argsort(dim=1)[:, :K].contiguous()
    w = torch.softmax(torch.randn((T, K), device="cuda", generator=g), dim=1)
    if case["masked"]:
        idx[torch.rand((T, K), device="cuda", generator=g) < case["masked"]] = E
        idx[torch.rand(T, device="cuda", generator=g) < case["masked"]] = E
    order = idx.view(-1).argsort(stable=True)
    dst = torch.empty(T * K, dtype=torch.int32, device="cuda")
    dst[order] = torch.arange(T * K, dtype=torch.int32, device="cuda")
    dst[idx.view(-1) == E] = -1
    return dst.view(T, K), w


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    dev = "cuda"
    if op == "route":
        s["logits"] = _logits(case, g)
        s["expert_bias"] = (torch.randn(case["E"], device=dev, generator=g) * 0.1
                            if case["bias"] else None)
    elif op == "route_backward":
        s["logits"] = _logits(case, g)
        l = s["logits"].double()
        val, idx = l.sort(dim=1, descending=True, stable=True)
        s["topk_idx"] = torch.where(val > -math.inf, idx, -1)[:, :case["K"]].contiguous()
        s["grad_weights"] = torch.randn((case["T"], case["K"]), device=dev, generator=g) * 0.01
    elif op == "combine_backward":
        T, H, K = case["T"], case["H"], case["K"]
        s["dst_row"], s["weights"] = _routing(case, g)
        s["grad_out"] = (torch.randn((T, H), device=dev, generator=g) * 0.01).bfloat16()
        s["y"] = torch.randn((T * K, H), device=dev, generator=g).bfloat16()
        # rows that no slot names are left as they are: the buffers start as zeros
        s["grad_y"] = torch.zeros((T * K, H), dtype=torch.bfloat16, device=dev)
        s["grad_weights"] = torch.zeros((T, K), device=dev)
    elif op == "dispatch_backward":
        T, H, K = case["T"], case["H"], case["K"]
        s["dst_row"], _ = _routing(case, g)
        s["grad_recv_x"] = (torch.randn((T * K, H), device=dev, generator=g) * 0.01).bfloat16()
    else:
        E, C, I, N, G = (case[k] for k in ("E", "C", "I", "N", "G"))
        WN = 2 * N if case["act"] else N
        # uneven rows per expert, at most C each, as a router fills them
        p = torch.rand(E, device=dev, generator=g) + 0.3
        p = p / p.sum()
        if case["rows"] < E:       # fewer rows than experts: one row each for some of them
            cnt = torch.zeros(E, dtype=torch.int64, device=dev)
            cnt[torch.rand(E, device=dev, generator=g).argsort()[:case["rows"]]] = 1
        else:
            cnt = (p * case["rows"]).round().long().clamp(max=C)
        s["counts"] = cnt.to(torch.int32)
        off = torch.zeros(E + 1, dtype=torch.int32, device=dev)
        off[1:] = cnt.cumsum(0).to(torch.int32)
        s["expert_offsets"] = off if case["offsets"] else None
        R = E * C
        x = torch.randn((R, I), device=dev, generator=g)
        if case["x"] == "fp8":
            a = x.view(R, I // 128, 128).abs().amax(dim=2).clamp(min=1e-4)
            s["x_scales"] = a / 448.0
            q = (x.view(R, I // 128, 128) * (448.0 / a)[:, :, None]).to(torch.float8_e4m3fn)
            s["x"] = q.view(torch.uint8).view(R, I)
        else:
            s["x_scales"] = None
            s["x"] = x.bfloat16()
        s["weight"] = torch.randint(0, 256, (E, WN, I // 2), dtype=torch.uint8, device=dev,
                                    generator=g)
        s["scales"] = ((torch.rand((E, I // G, WN), device=dev, generator=g) + 0.5)
                       * (0.2 / math.sqrt(I))).bfloat16()
        s["zeros"] = (torch.randint(4, 13, (E, I // G, WN), dtype=torch.uint8, device=dev,
                                    generator=g) if case["zeros"] else None)
        s["y"] = torch.zeros((R, N), dtype=torch.bfloat16, device=dev)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"route": _route, "route_backward": _route_backward,
            "combine_backward": _combine_backward, "dispatch_backward": _dispatch_backward,
            "w4": _w4}[s["op"]](s)


def _run_own(s):
    from combine_ep_get_dispatch_amd import binding as ep
    op = s["op"]
    if op == "route":
        return ep.route(s["logits"], s["K"], expert_bias=s["expert_bias"], score=s["score"],
                        num_groups=s["groups"], topk_groups=s["topk_groups"],
                        normalize=s["normalize"], scale=s["scale"])
    if op == "route_backward":
        return ep.route_backward(s["logits"], s["topk_idx"], s["grad_weights"],
                                 score=s["score"], normalize=s["normalize"], scale=s["scale"])
    if op == "combine_backward":
        return ep.combine_backward(s["grad_out"], s["y"], s["dst_row"], s["weights"],
                                   out=(s["grad_y"], s["grad_weights"]))
    if op == "dispatch_backward":
        return ep.dispatch_backward(s["grad_recv_x"], s["dst_row"])
    return ep.expert_linear_w4(s["x"], s["weight"], s["scales"], s["counts"],
                               expert_offsets=s["expert_offsets"],
                               capacity=0 if s["offsets"] else s["C"], x_scales=s["x_scales"],
                               zeros=s["zeros"], swiglu=s["act"], out=s["y"])


def _scores(l, score):
    """Scores in 64 bits (an expert's place is decided by them); an expert whose logit is
    -inf or NaN is not available and scores 0."""
    avail = l > -math.inf
    l = torch.where(avail, l.clamp(max=FLT_MAX), -math.inf)
    if score == "sigmoid":
        return avail, l, torch.where(avail, 1.0 / (1.0 + torch.exp(-l)), 0.0)
    m = l.amax(dim=1, keepdim=True).clamp(min=-FLT_MAX)
    e = torch.exp(l - m)
    return avail, l, e / e.sum(dim=1, keepdim=True).clamp(min=1e-300)


def _over_selected(l, sc, ok, idx, score):
    """Shares of the selected experts: their scores over the scores' sum (0 if that is 0)."""
    if score == "softmax":
        ls = torch.where(ok, l.gather(1, idx), -math.inf)
        m = ls.amax(dim=1, keepdim=True).clamp(min=-FLT_MAX)
        v = torch.exp(ls - m)
    else:
        v = torch.where(ok, sc.gather(1, idx), 0.0)
    tot = v.sum(dim=1, keepdim=True)
    return torch.where(tot > 0, v / torch.where(tot > 0, tot, 1.0), 0.0), tot


def _route(s):
    T, E, K, NG = s["T"], s["E"], s["K"], s["groups"]
    avail, l, sc = _scores(s["logits"].double(), s["score"])
    choice = sc if s["expert_bias"] is None else sc + s["expert_bias"].double()
    choice = torch.where(avail, choice, -math.inf)
    rank_by = l if s["expert_bias"] is None else choice
    if NG > 1:
        best = choice.view(T, NG, E // NG).sort(dim=2, descending=True).values[:, :, :2]
        gs = torch.where(best > -math.inf, best, 0.0).sum(dim=2)
        gs = torch.where(best[:, :, 0] > -math.inf, gs, -math.inf)
        keep = gs.sort(dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        allowed = torch.zeros((T, NG), dtype=torch.bool, device=l.device).scatter(1, keep, True)
        rank_by = torch.where(allowed.repeat_interleave(E // NG, dim=1), rank_by, -math.inf)
    val, idx = rank_by.sort(dim=1, descending=True, stable=True)
    val, idx = val[:, :K], idx[:, :K]
    ok = val > -math.inf
    if s["normalize"]:
        w, _ = _over_selected(l, sc, ok, idx, s["score"])
    else:
        w = torch.where(ok, sc.gather(1, idx), 0.0)
    return torch.where(ok, idx, -1), (w * s["scale"]).float()


def _route_backward(s):
    avail, l, sc = _scores(s["logits"].double(), s["score"])
    ok = s["topk_idx"] >= 0
    idx = s["topk_idx"].clamp(min=0)
    c = torch.where(ok, s["grad_weights"].double() * s["scale"], 0.0)
    grad = torch.zeros_like(l)
    if s["normalize"]:
        q, tot = _over_selected(l, sc, ok, idx, s["score"])
        d = q * (c - (c * q).sum(dim=1, keepdim=True))
        if s["score"] == "sigmoid":
            d = d * (1.0 - sc.gather(1, idx))
        grad.scatter_add_(1, idx, d)
    elif s["score"] == "sigmoid":
        v = sc.gather(1, idx)
        grad.scatter_add_(1, idx, c * v * (1.0 - v))
    else:
        dense = torch.zeros_like(l).scatter_add_(1, idx, c)
        grad = sc * (dense - (dense * sc).sum(dim=1, keepdim=True))
    return grad.to(s["logits"].dtype)


def _combine_backward(s):
    ok = s["dst_row"] >= 0
    r = s["dst_row"].clamp(min=0).long()
    g = s["grad_out"].float()[:, None, :]
    dw = (g * s["y"][r].float()).sum(dim=2)
    s["grad_weights"].copy_(torch.where(ok, dw, 0.0))
    s["grad_y"][r[ok]] = (g * s["weights"][:, :, None])[ok].to(torch.bfloat16)
    return s["grad_y"], s["grad_weights"]


def _dispatch_backward(s):
    ok = s["dst_row"] >= 0
    rows = s["grad_recv_x"][s["dst_row"].clamp(min=0).long()].float()
    return torch.where(ok[:, :, None], rows, 0.0).sum(dim=1).to(torch.bfloat16)


def _rows_of(s):
    """[E, C] receive row of each place, and whether it holds a token."""
    E, C = s["E"], s["C"]
    j = torch.arange(C, device="cuda")
    begin = (s["expert_offsets"][:E].long() if s["offsets"]
             else torch.arange(E, device="cuda") * C)
    held = j[None, :] < s["counts"][:, None]
    return torch.where(held, begin[:, None] + j[None, :], 0), held


def _w4(s):
    rows, held = _rows_of(s)
    E, I, G = s["E"], s["I"], s["G"]
    x = s["x"]
    if s["x_scales"] is not None:
        R = x.shape[0]
        x = (x.view(torch.float8_e4m3fn).float().view(R, I // 128, 128)
             * s["x_scales"][:, :, None]).view(R, I)
    xe = x[rows].float()
    p = s["weight"]
    q = torch.stack((p & 15, p >> 4), dim=3).view(E, -1, I // G, G).float()
    z = 8.0 if s["zeros"] is None else s["zeros"].float().transpose(1, 2)[..., None]
    w = (q - z) * s["scales"].float().transpose(1, 2)[..., None]
    y = torch.bmm(xe, w.view(E, -1, I).transpose(1, 2))
    if s["act"]:
        gate, up = y[..., :s["N"]], y[..., s["N"]:]
        y = gate / (1.0 + torch.exp(-gate)) * up
    s["y"][rows[held]] = y[held].to(torch.bfloat16)
    return s["y"]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("route", "route_backward"):
        T, E, K = case["T"], case["E"], case["K"]
        b = 2 if case["dtype"] == "bf16" else 4
        if op == "route":
            return {"bytes": T * E * b + T * K * 12, "flops": T * E * 10}
        dense = case["score"] == "softmax" and not case["normalize"]
        return {"bytes": T * E * b + T * K * 12 + (T * E if dense else T * K) * b,
                "flops": T * (E * 8 if dense else K * 10)}
    if op in ("combine_backward", "dispatch_backward"):
        T, H, K = case["T"], case["H"], case["K"]
        n = T * K * (1 - case["masked"]) ** 2
        if op == "combine_backward":
            return {"bytes": T * H * 2 + 2 * n * H * 2 + T * K * 12, "flops": 3 * n * H}
        return {"bytes": T * H * 2 + n * H * 2 + T * K * 4, "flops": n * H}
    E, I, N, rows = case["E"], case["I"], case["N"], case["rows"]
    WN = 2 * N if case["act"] else N
    active = min(E, rows)
    per = WN * I // 2 + (I // case["G"]) * WN * (3 if case["zeros"] else 2)
    xb = I + I // 128 * 4 if case["x"] == "fp8" else 2 * I
    return {"bytes": active * per + rows * (xb + 2 * N), "flops": 2 * rows * WN * I}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return None, _exact_route(s)
    if op == "route_backward":
        return _exact_route_backward(s)
    if op == "combine_backward":
        T, H, K = case["T"], case["H"], case["K"]
        g = s["grad_out"].double()
        gy = torch.zeros((T * K, H), dtype=torch.float64, device="cuda")
        gw = torch.zeros((T, K), dtype=torch.float64, device="cuda")
        for k in range(K):
            t = (s["dst_row"][:, k] >= 0).nonzero()[:, 0]
            r = s["dst_row"][t, k].long()
            gy[r] = s["weights"][t, k, None].double() * g[t]
            gw[t, k] = (g[t] * s["y"][r].double()).sum(1)
        return gy, gw
    if op == "dispatch_backward":
        out = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
        for k in range(case["K"]):
            t = (s["dst_row"][:, k] >= 0).nonzero()[:, 0]
            out[t] += s["grad_recv_x"][s["dst_row"][t, k].long()].double()
        return out
    return _exact_w4(s)


def _exact_shares(l, idx, ok, score, normalize):
    """What the weights are before the scale, with the selected experts given."""
    if score == "sigmoid":
        v = torch.sigmoid(l.gather(1, idx))
    else:
        v = torch.softmax(l, dim=1).gather(1, idx)
    v = torch.where(ok, v, 0.0)
    if normalize:
        v = v / v.sum(dim=1, keepdim=True)
    return torch.nan_to_num(v)


def _exact_route(s):
    """Weights alone: the experts are picked one after the other from the highest down."""
    l = s["logits"].double()
    T, E = l.shape
    sc = torch.sigmoid(l) if s["score"] == "sigmoid" else torch.nan_to_num(torch.softmax(l, 1))
    dead = l == -math.inf
    ch = sc + (s["expert_bias"].double() if s["expert_bias"] is not None else 0.0)
    ch = ch.masked_fill(dead, -math.inf)
    NG = s["groups"]
    if NG > 1:
        grp = ch.view(T, NG, E // NG)
        a, at = grp.max(dim=2)
        b = (grp.scatter(2, at[..., None], -math.inf).amax(dim=2) if E // NG > 1
             else torch.full_like(a, -math.inf))
        gs = torch.where(b > -math.inf, a + b, a)
        kept = torch.zeros((T, NG), dtype=torch.bool, device="cuda")
        for _ in range(s["topk_groups"]):
            best = gs.masked_fill(kept, -math.inf).argmax(dim=1)
            kept[torch.arange(T, device="cuda"), best] = True
        ch = ch.masked_fill(~kept.repeat_interleave(E // NG, 1), -math.inf)
    idx, ok = [], []
    left = ch.clone()
    for _ in range(s["K"]):
        v, i = left.max(dim=1)
        idx.append(i)
        ok.append(v > -math.inf)
        left[torch.arange(T, device="cuda"), i] = -math.inf
    idx, ok = torch.stack(idx, 1), torch.stack(ok, 1)
    return _exact_shares(l, idx, ok, s["score"], s["normalize"]) * s["scale"]


def _exact_route_backward(s):
    """The gradient by automatic differentiation in 64 bits."""
    l = torch.nan_to_num(s["logits"].double(), neginf=-1e9).requires_grad_(True)
    ok = s["topk_idx"] >= 0
    idx = s["topk_idx"].clamp(min=0)
    v = (torch.sigmoid(l) if s["score"] == "sigmoid" else torch.softmax(l, dim=1)).gather(1, idx)
    v = torch.where(ok, v, 0.0)
    if s["normalize"]:
        v = v / v.sum(dim=1, keepdim=True).clamp(min=1e-300)
    (v * s["grad_weights"].double() * s["scale"]).sum().backward()
    return l.grad * (s["logits"] > -math.inf)


def _exact_w4(s):
    if s["rows"] * s["I"] * s["N"] > 1e11:
        return None
    out = torch.zeros((s["E"] * s["C"], s["N"]), dtype=torch.float64, device="cuda")
    for e, n in enumerate(s["counts"].tolist()):
        if n == 0:
            continue
        b = int(s["expert_offsets"][e]) if s["offsets"] else e * s["C"]
        x = s["x"][b:b + n]
        if s["x_scales"] is not None:
            x = (x.view(torch.float8_e4m3fn).double()
                 * s["x_scales"][b:b + n].double().repeat_interleave(128, 1))
        x = x.double()
        w = torch.empty((s["weight"].shape[1], s["I"]), dtype=torch.float64, device="cuda")
        w[:, 0::2] = (s["weight"][e] % 16).double()
        w[:, 1::2] = (s["weight"][e] // 16).double()
        if s["zeros"] is None:
            w -= 8
        else:
            w -= s["zeros"][e].t().double().repeat_interleave(s["G"], 1)
        w *= s["scales"][e].t().double().repeat_interleave(s["G"], 1)
        y = x @ w.t().contiguous()
        if s["act"]:
            y = torch.nn.functional.silu(y[:, :s["N"]]) * y[:, s["N"]:]
        out[b:b + n] = y
    return out
