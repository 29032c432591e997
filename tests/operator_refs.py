"""Plain 64-bit references (torch on the CPU) of the router, the gradients of
dispatch and combine, and the experts' 4-bit products, written from their
definitions, with the error bounds that the tests hold the kernels to.

A rounding to nearest is off by at most half a step relative to the value:
U32 = 2^-24 for fp32, UBF = 2^-8 for bf16.  TINY covers results below the
smallest normal bf16 / fp32 value.
"""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24
UBF = 2.0 ** -8
TINY = 2.0 ** -126
FLT_MAX = 3.4028234663852886e38


def clean(logits):
    """Logits in 64 bits: +inf as fp32's largest value, -inf and NaN as -inf."""
    l = logits.double()
    return torch.where(l > -math.inf, l.clamp(max=FLT_MAX), -math.inf)


def scores(logits, score):
    l = clean(logits)
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    m = l.amax(dim=1, keepdim=True).clamp(min=-FLT_MAX)
    e = torch.exp(l - m)
    return e / e.sum(dim=1, keepdim=True).clamp(min=1e-300)


def route(logits, K, bias=None, score="softmax", num_groups=1, topk_groups=1, normalize=False,
          scale=1.0):
    """(topk_idx, weights in 64 bits), token by token."""
    T, E = logits.shape
    l = clean(logits)
    s = scores(logits, score)
    idx = torch.full((T, K), -1, dtype=torch.int64)
    w = torch.zeros((T, K), dtype=torch.float64)
    gsz = E // num_groups
    for t in range(T):
        choice = []
        for e in range(E):
            c = float(s[t, e]) + (0.0 if bias is None else float(bias[e]))
            ok = float(l[t, e]) > -math.inf and c > -math.inf
            choice.append(c if ok else -math.inf)
        open_ = [c > -math.inf for c in choice]
        if num_groups > 1:
            gs = []
            for g in range(num_groups):
                best = sorted((c for c in choice[g * gsz:(g + 1) * gsz] if c > -math.inf),
                              reverse=True)[:2]
                gs.append(sum(best) if best else -math.inf)
            kept = sorted(range(num_groups), key=lambda g: (-gs[g], g))[:topk_groups]
            open_ = [o and e // gsz in kept for e, o in enumerate(open_)]
        by = choice if bias is not None else [float(v) for v in l[t]]
        chosen = sorted((e for e in range(E) if open_[e]), key=lambda e: (-by[e], e))[:K]
        if not chosen:
            continue
        idx[t, :len(chosen)] = torch.tensor(chosen)
        if normalize and score == "softmax":
            v = torch.softmax(l[t, chosen], dim=0)
        else:
            v = s[t, chosen]
            if normalize:
                v = v / v.sum() if float(v.sum()) > 0 else torch.zeros_like(v)
        w[t, :len(chosen)] = v * scale
    return idx, w


def route_weight_tol(w, E):
    """fp32 softmax sum: each term's exponent is off by the rounding of l - m
    (at most ln E half steps on average over the weights of the terms) and by
    4 half steps of expf; a term passes at most 16 + 6 additions; one rounding
    to fp32 at the end."""
    return (math.log(E) + 4 + 22 + 2) * U32 * w.abs() + TINY


def route_backward(logits, topk_idx, gw, score, normalize, scale):
    """(gradient in 64 bits, size of the terms it is the difference of)."""
    T, E = logits.shape
    l = clean(logits)
    s = scores(logits, score)
    ok = (topk_idx >= 0) & (topk_idx < E)
    idx = torch.where(ok, topk_idx, 0)
    c = torch.where(ok, gw.double() * scale, 0.0)
    if score == "softmax" and not normalize:
        dense = torch.zeros_like(s).scatter_add_(1, idx, c)
        size = torch.zeros_like(s).scatter_add_(1, idx, c.abs())
        pk = torch.where(ok, s.gather(1, idx), 0.0)
        mean = (c * pk).sum(1, keepdim=True)
        return s * (dense - mean), s * (size + (c * pk).abs().sum(1, keepdim=True))
    sk = torch.where(ok, s.gather(1, idx), 0.0)
    if score == "softmax":
        lk = torch.where(ok, l.gather(1, idx), -math.inf)
        m = lk.amax(1, keepdim=True).clamp(min=-FLT_MAX)
        v = torch.exp(lk - m)
    else:
        v = sk
    if normalize:
        tot = v.sum(1, keepdim=True)
        q = torch.where(tot > 0, v / tot.clamp(min=1e-300), 0.0)
        d = q * (c - (c * q).sum(1, keepdim=True))
        size = q * (c.abs() + (c * q).abs().sum(1, keepdim=True))
    else:
        d, size = c * sk, (c * sk).abs()
    if score == "sigmoid":
        # 1 - s as sigmoid(-l): it does not cancel for large logits
        one = torch.where(ok, torch.sigmoid(-l.gather(1, idx)), 0.0)
        d, size = d * one, size * one
    grad = torch.zeros_like(s).scatter_add_(1, idx, d)
    return grad, torch.zeros_like(s).scatter_add_(1, idx, size)


def route_backward_tol(grad, size, E, dtype):
    """The shares as in route_weight_tol, their inverse sum, two products, the
    difference and the additions of a repeated expert: 8 roundings more; then
    the rounding to the result's type."""
    out = UBF if dtype == torch.bfloat16 else U32
    return (math.log(E) + 4 + 22 + 2 + 8) * U32 * size + out * grad.abs() + TINY


def combine_backward(grad_out, y, dst_row, w):
    """(grad_y, grad_weights, sum of |g * y|) in 64 bits; grad_y 0 where no slot writes."""
    T, K = dst_row.shape
    R, H = y.shape
    gy = torch.zeros((R, H), dtype=torch.float64)
    gw = torch.zeros((T, K), dtype=torch.float64)
    size = torch.zeros((T, K), dtype=torch.float64)
    g, yd, d = grad_out.double(), y.double(), dst_row.tolist()
    for t in range(T):
        for k in range(K):
            r = d[t][k]
            if 0 <= r < R:
                gy[r] = float(w[t, k]) * g[t]
                gw[t, k] = (g[t] * yd[r]).sum()
                size[t, k] = (g[t] * yd[r]).abs().sum()
    return gy, gw, size


def dispatch_backward(grad_recv, dst_row):
    """(grad_x, sum of |terms|) in 64 bits."""
    T, K = dst_row.shape
    R, H = grad_recv.shape
    out = torch.zeros((T, H), dtype=torch.float64)
    size = torch.zeros((T, H), dtype=torch.float64)
    g = grad_recv.double()
    for k in range(K):
        ok = (dst_row[:, k] >= 0) & (dst_row[:, k] < R)
        rows = g[dst_row[:, k].clamp(0, max(R - 1, 0)).long()] if R else out * 0
        out += torch.where(ok[:, None], rows, 0.0)
        size += torch.where(ok[:, None], rows.abs(), 0.0)
    return out, size


def e4m3_values():
    """The 256 values of OCP E4M3, from the format: 4 exponent bits of bias 7,
    3 fraction bits, subnormals at exponent 0."""
    v = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        a = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if code & 0x7f == 0x7f:
            a = math.nan
        v.append(-a if code & 0x80 else a)
    return torch.tensor(v, dtype=torch.float64)


def expert_linear(x, x_scales, weight, scales, zeros, ranges, N, swiglu):
    """(y, bound on |kernel - y| before the last rounding) in 64 bits; NaN in
    rows outside ``ranges`` (a list of (first row, rows) per expert).

    The bound: a group's sum is formed from |x| (q + 128) <= 143 |x| or from
    |x| q <= 15 |x| and its zero point's part, in fp32; G products are added
    in at most G roundings, counted at a full step 2^-23 each since a matrix
    instruction may cut instead of rounding; where a block's zero points are
    taken off after its four groups, the four scaled sums and the four
    corrections are added at that size, 8 roundings more; the groups' results,
    scaled, are added with at most I/G + 64 roundings more."""
    R, I = x.shape
    E, W, _ = weight.shape
    NG = scales.shape[1]
    G = I // NG
    y = torch.full((R, N), math.nan, dtype=torch.float64)
    tol = torch.zeros((R, N), dtype=torch.float64)
    if x_scales is not None:
        xd = e4m3_values()[x.long()] * x_scales.double().repeat_interleave(128, 1)
    else:
        xd = x.double()
    for e, (b, n) in enumerate(ranges):
        if n <= 0:
            continue
        q = torch.empty((W, I), dtype=torch.float64)
        q[:, 0::2] = (weight[e] & 15).double()
        q[:, 1::2] = (weight[e] >> 4).double()
        z = torch.full((W, I), 8.0, dtype=torch.float64) if zeros is None else \
            (zeros[e].t() & 15).double().repeat_interleave(G, 1)
        s = scales[e].t().double().repeat_interleave(G, 1)
        rows = xd[b:b + n]
        a = rows @ ((q - z) * s).t()
        big = rows.abs() @ (143.0 * s.abs()).t()
        each = rows.abs() @ ((q - z).abs() * s.abs()).t()
        err = (G + 8) * 2 * U32 * big + (NG + 64) * U32 * each
        if swiglu:
            g, u, eg, eu = a[:, :N], a[:, N:], err[:, :N], err[:, N:]
            sg = g * torch.sigmoid(g)
            y[b:b + n] = sg * u
            # |silu'| <= 1.1; expf, the division and two products: 8 half steps
            tol[b:b + n] = 1.1 * eg * (u.abs() + eu) + sg.abs() * eu + 8 * U32 * (sg * u).abs()
        else:
            y[b:b + n], tol[b:b + n] = a, err
    return y, tol
