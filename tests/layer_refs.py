"""Plain 64-bit references (torch on the CPU) of the experts' products and their
gradients, the gated activation and the root-mean-square norm, with the error
bounds that the tests hold the kernels to.

A rounding to nearest is off by at most half a step relative to the value:
U32 = 2^-24 for fp32, UBF = 2^-8 for bf16, U8 = 2^-4 for E4M3.  Sums of matrix
instructions may cut instead of rounding: a full step, 2 U32, each.
"""
from __future__ import annotations

import torch

from operator_refs import TINY, U32, UBF, e4m3_values

U8 = 2.0 ** -4


def ranges(counts, offsets, capacity, R):
    """(first row, rows) of each expert, inside [0, R)."""
    out = []
    for e, n in enumerate(counts):
        b = offsets[e] if offsets is not None else e * capacity
        end = b + (n if offsets is not None else min(n, capacity))
        b, end = max(b, 0), min(end, R)
        out.append((b, max(end - b, 0)))
    return out


def fp8_values(codes, scales, channels_per_block=None):
    """Values of E4M3 rows (a scale per 128 channels)."""
    return e4m3_values()[codes.long()] * scales.double().repeat_interleave(128, -1)


def weight_values(codes, scales, N):
    """[E, W, I] values of E4M3 weights with a scale per 128 x 128 block of each
    half of N channels."""
    E, W, I = codes.shape
    NB = (N + 127) // 128
    ch = torch.arange(W)
    block = ch // N * NB + ch % N // 128
    return e4m3_values()[codes.long()] * scales.double()[:, block].repeat_interleave(128, 2)


# The sigmoid's result is 0 below v = -87.3, where the reciprocal of 1 + exp(-v) would
# be subnormal: |silu(v)| is at most 87.4 * e^-87.3 < 2^-119 there.
LOST = 2.0 ** -119


def silu_steps(v):
    """Half steps of fp32 that silu(v) * u is off by.  v * log2(e) is rounded once,
    the constant once at 0.22 half steps: exp makes 1.25 |v| half steps of that.
    exp itself 2, the sum 1, the reciprocal 2, two products 2."""
    return 1.25 * v.abs() + 8


def silu(v):
    return v * torch.sigmoid(v)


def linear(x, w, runs, N, swiglu, cut=0.0):
    """(y, bound ahead of the last rounding) in 64 bits, NaN in rows of no
    expert.  I products of fp32 are added: I + 8 steps of 2 U32 of the sum of
    their sizes; E4M3 products (cut = 2^-13) lose up to that much of the largest
    of eight neighbours, which all eight together are at least as large as."""
    R, I = x.shape
    y = torch.full((R, N), float("nan"), dtype=torch.float64)
    tol = torch.zeros((R, N), dtype=torch.float64)
    for e, (b, n) in enumerate(runs):
        if n == 0:
            continue
        a = x[b:b + n] @ w[e].t()
        err = ((I + 8) * 2 * U32 + 8 * cut) * (x[b:b + n].abs() @ w[e].abs().t())
        if swiglu:
            g, u, eg, eu = a[:, :N], a[:, N:], err[:, :N], err[:, N:]
            sg = silu(g)
            y[b:b + n] = sg * u
            # |silu'| <= 1.1
            tol[b:b + n] = (1.1 * eg * (u.abs() + eu) + sg.abs() * eu
                            + silu_steps(g) * U32 * (sg * u).abs() + LOST * u.abs())
        else:
            y[b:b + n], tol[b:b + n] = a, err
    return y, tol


def gate(a, N):
    """(y, bound ahead of its rounding)."""
    a = a.double()
    g = a[:, :N]
    y = silu(g) * a[:, N:]
    return y, silu_steps(g) * U32 * y.abs() + LOST * a[:, N:].abs() + TINY


def gate_backward(gy, a, N):
    """(gradient, bound ahead of its rounding).  s as in silu_steps; 1 - s: U32
    against s <= 1 and s's own error carried over; the rest 6 products and
    additions of terms whose sizes add up to `size`."""
    a, gy = a.double(), gy.double()
    g, u = a[:, :N], a[:, N:]
    s = torch.sigmoid(g)
    dg = gy * u * (s + g * s * (1 - s))
    size = (gy * u).abs() * (s + (g * s).abs())
    du = gy * g * s
    steps = silu_steps(g)
    return (torch.cat((dg, du), 1),
            torch.cat((2 * steps * U32 * size + LOST * (gy * u).abs(),
                       steps * U32 * du.abs() + LOST * gy.abs()), 1) + TINY)


def to_e4m3(y, tol):
    """(scales, their bound, values, their bound) of dispatch's rule on values
    known within tol.  The largest of a group is off by at most the group's
    largest bound; a code is off by half a step of E4M3 (2^-10 of the smallest
    normal, 2^-6, below that) more than its value, counted in the scale's unit."""
    R, H = y.shape
    v, t = y.view(R, H // 128, 128), tol.view(R, H // 128, 128)
    top = v.abs().amax(2).clamp(min=1e-4)
    scales = top / 448
    stol = t.amax(2) / 448 + 4 * U32 * scales
    vt = t + (U8 + 4 * U32) * (v.abs() + t) + 2.0 ** -10 * (scales + stol)[..., None]
    return scales, stol, y, vt.view(R, H)


def norm(h, weight, eps):
    """(y, its bound, inv, its bound).  A thread's sum passes up to 64 additions
    and the workgroup's 22 more, squares of one sign; mean, eps, root and
    reciprocal 4 more; half of it for the root.  y: two products more."""
    h = h.double()
    inv = (h.square().mean(1) + eps).rsqrt()
    itol = (0.5 * 90 + 4) * U32 * inv
    y = h * inv[:, None] * weight.double()
    return y, (0.5 * 90 + 6) * U32 * y.abs() + TINY, inv, itol


def norm_backward(gy, h, weight, inv, gres):
    """(grad_x, bound ahead of its rounding, grad_weight, its bound), inv as
    given.  The row's sum: 90 roundings of the sizes' mean; six more for the
    rest.  grad_weight: T terms of 2 roundings added in at most T steps."""
    gy, h, w, inv = gy.double(), h.double(), weight.double(), inv.double()[:, None]
    n, gn = h * inv, gy * w
    mean = (gn * n).mean(1, keepdim=True)
    size = (gn * n).abs().mean(1, keepdim=True)
    gx = inv * (gn - n * mean)
    tol = inv * (8 * U32 * gn.abs() + n.abs() * (96 * U32 * size + 8 * U32 * mean.abs()))
    if gres is not None:
        gx = gx + gres.double()
        tol = tol + U32 * gx.abs()
    T = gy.shape[0]
    return gx, tol + TINY, (gy * n).sum(0), (T + 4) * U32 * (gy * n).abs().sum(0) + TINY


def bf16_tol(y, tol):
    return tol * (1 + UBF) + UBF * y.abs() + TINY
