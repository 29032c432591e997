"""The gated activation far from zero."""
import math

import pytest
import torch

from combine_ep_get_dispatch_amd import binding as ep
from operator_refs import U32, UBF
from test_gpu_expert_linear import gen, within

pytestmark = pytest.mark.gpu


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
