"""The gated activation over all gates: to half a step of bf16 but for 17 * 2^-24, and far
below zero, by itself, behind the products, and its gradient."""
import math

import pytest
import torch

import layer_refs as ref
from combine_ep_get_dispatch_amd import binding as ep
from operator_refs import TINY, U32, UBF
from parity import announce
from test_gpu_expert_linear import device, gen, within

pytestmark = pytest.mark.gpu

# Half steps of fp32 that silu(g) * u is off by: exp(g / 2) 3 (v_exp_f32 2, what its
# argument lost 1), its square 6, one sum, one reciprocal (2), four products.  The
# gate is taken as 17.5 where it is more: 1 - 2^-25 at most.
STEPS = 14
# The activation by itself, where eight neighbours are at least -8: silu(g) * u from exp(-g),
# whose argument is off by 1.22 |g| half steps (a rounding, 1, and its constant, 0.22), exp
# itself 2, one sum, one reciprocal (2), two products: 7 + 1.22 * 8.
ALONE = 17


def all_gates():
    """Every bf16 value from -170 to 200 of at least 2^-20, and zero."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.uint16)
    v = bits.view(torch.bfloat16)
    d = v.double()
    # (neighbouring gates are alike: groups of eight above and below -8)
    v = v[(d >= -170) & (d <= 200) & ((d.abs() >= 2.0 ** -20) | (d == 0))]
    return v[: v.numel() // 128 * 128]


def inputs(top=20):
    """[R, 2N]: all gates beside ups of sizes of 2^-top to 2^top, and far gates beside
    ups that bring the product back."""
    g = all_gates()
    N = 128
    gates = g.repeat(4).view(-1, N)
    size = 2.0 ** (torch.rand(gates.shape, generator=gen(1)) * 2 * top - top)
    ups = (torch.randn(gates.shape, generator=gen(2)) * size).bfloat16()
    far = (-80 - 80 * torch.rand((64, N), generator=gen(3))).bfloat16()
    back = torch.exp(-far.double() - torch.rand((64, N), generator=gen(4)).double() * 60)
    back = back.clamp(max=3e38).bfloat16()
    return torch.cat((torch.cat((gates, far)), torch.cat((ups, back))), 1).contiguous(), N


def near_rounded(got, want, share, what):
    """got is want rounded to bf16, or, where want is within ``share`` of its size from the
    middle between two, either of them.  (Subnormal results: one of their steps, 2^-133.)"""
    got = got.detach().cpu().double()
    a, b = ((want * (1 + k * share)).float().bfloat16().double() for k in (-1, 1))
    low, high = torch.minimum(a, b), torch.maximum(a, b)
    small = want.abs() < 2 * TINY
    ok = torch.where(small, (got - want).abs() <= 2.0 ** -133 + UBF * want.abs(),
                     (got >= low) & (got <= high))
    assert bool(ok.all()), "%s: %d of %d off, first %r" % (
        what, int((~ok).sum()), ok.numel(), (float(got[~ok][0]), float(want[~ok][0])))


def test_activation_of_every_gate():
    announce("expert_swiglu of every gate")
    a, N = inputs()
    want, _ = ref.gate(a, N)
    near_rounded(ep.expert_swiglu(a.cuda()), want, ALONE * U32, "y")
    codes, scales = ep.expert_swiglu(a.cuda(), fp8=True)
    top = want.view(-1, 128).abs().amax(1, keepdim=True).clamp(min=1e-4) / 448
    within(scales.view(-1, 1), top, (ALONE + 4) * U32 * top, "scales")


@pytest.mark.parametrize("rows", [3, 130])
@pytest.mark.parametrize("fp8", [False, True])
def test_activation_behind_the_products(rows, fp8):
    """Rows that are 1 in one channel, whose sums are the weights themselves: in the few
    tasks of few rows and in tiles."""
    announce("expert_linear with the activation, every gate, rows=%d fp8=%d" % (rows, fp8))
    a, _ = inputs()
    gate, up = a[:, :128].reshape(-1), a[:, 128:].reshape(-1)
    N, I = gate.numel(), 128
    x = torch.zeros((rows, I))
    x[:, 5] = 1
    kw = {}
    w = torch.zeros((1, 2 * N, I), dtype=torch.bfloat16)
    if fp8:
        # codes of gates, a quarter each, and of ups with scales of 2^-8 to 2^23
        c = torch.arange(256, dtype=torch.int32).to(torch.uint8)
        c = c[(c & 0x7F) != 0x7F]
        N = 256 * 16
        g = gen(9)
        gc, uc = (c[torch.randint(0, c.numel(), (N,), generator=g)] for _ in range(2))
        gs, us = torch.full((N // 128,), 0.25), 2.0 ** torch.arange(-8, N // 128 - 8).float()
        w = torch.zeros((1, 2 * N, I), dtype=torch.uint8)
        w[0, :N, 5], w[0, N:, 5] = gc, uc
        kw = dict(x_scales=torch.ones((rows, 1)).cuda(),
                  weight_scales=torch.cat((gs, us)).view(1, -1, 1).cuda())
        x = x.to(torch.float8_e4m3fn).view(torch.uint8)
        v = lambda q, s: q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128)
        want, _ = ref.gate(torch.cat((v(gc, gs), v(uc, us))).view(1, -1), N)
    else:
        w[0, :N, 5], w[0, N:, 5] = gate, up
        x = x.bfloat16()
        want, _ = ref.gate(torch.cat((gate, up)).view(1, -1), N)
    cnt, off = device([rows], [0, rows])
    y = ep.expert_linear(x.cuda(), w.cuda(), cnt, expert_offsets=off, swiglu=True, **kw)
    near_rounded(y, want.expand(rows, -1), STEPS * U32, "y")


def test_gradient_of_every_gate():
    """As above for d up, a product of the same factors and two more; d gate is off by as much of
    grad_y up s (1 + |g| (1 - s)) and 6 more: its own sum, products and 1 - s."""
    announce("expert_swiglu_backward of every gate")
    a, N = inputs()
    gy = torch.randn((a.shape[0], N), generator=gen(6)).bfloat16()
    got = ep.expert_swiglu_backward(gy.cuda(), a.cuda()).cpu()
    g, u, d = a[:, :N].double(), a[:, N:].double(), gy.double()
    s = torch.sigmoid(g)
    near_rounded(got[:, N:], d * g * s, STEPS * U32, "d up")
    rest = torch.sigmoid(-g)
    want = d * u * s * (1 + g * rest)
    size = (d * u * s).abs() * (1 + g.abs() * rest)
    tol = (STEPS + 6) * U32 * size
    within(got[:, :N], want, tol * (1 + UBF) + UBF * want.abs() + 2.0 ** -133, "d gate")


def test_gradient_where_the_product_of_its_inputs_passes_the_range():
    """grad_y * up beyond fp32's range, and a sigmoid that brings it back (off by
    1.25 |g| + 20 half steps of fp32 at most)."""
    N = 128
    g = (-45 - 40 * torch.rand((8, N), generator=gen(11))).bfloat16()
    # sizes of 2^0 to 2^20 for the gradient
    e = (-g.double() * math.log2(math.e) + 20 * torch.rand((8, N), generator=gen(12)).double()) / 2
    u, gy = (torch.exp2(e + k).bfloat16() for k in (8, -8))
    u[0], gy[0] = 2.0 ** 70, 2.0 ** 70
    g[0] = -80
    got = ep.expert_swiglu_backward(gy.cuda(), torch.cat((g, u), 1).cuda()).cpu()
    gd, s = g.double(), torch.sigmoid(g.double())
    want = gy.double() * u.double() * s * (1 + gd * (1 - s))
    assert bool((want.abs() < 2.0 ** 120).all())
    within(got[:, :N], want, (128 * U32 + UBF) * 1.01 * want.abs(), "d gate")


def test_gates_that_are_not_numbers():
    """A NaN reaches every result of its element; +inf as the gate gives +-inf."""
    N = 8
    a, gy = torch.ones((2, 2 * N)).bfloat16(), torch.ones((2, N)).bfloat16()
    a[0, 1], a[0, 2], a[0, 3] = float("nan"), math.inf, -200.0
    a[0, N + 3] = 3e38
    y = ep.expert_swiglu(a.cuda()).cpu()
    d = ep.expert_swiglu_backward(gy.cuda(), a.cuda()).cpu()
    assert bool(torch.isnan(y[0, 1])) and bool(torch.isnan(d[0, 1])) and bool(torch.isnan(d[0, N + 1]))
    assert float(y[0, 2]) == math.inf and float(d[0, N + 2]) == math.inf
    assert float(y[0, 3]) == 0 and float(d[0, 3]) == 0 and float(d[0, N + 3]) == 0
    keep = [0, 4, 5, 6, 7]
    assert bool(torch.isfinite(y[0, keep]).all()) and bool(torch.isfinite(d[0, keep]).all())
    assert torch.equal(y[0, keep], y[1, keep])
