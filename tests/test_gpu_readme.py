"""The training step that README.md shows, run as it stands there."""
import os
import re

import pytest
import torch

import layer_refs as ref
from combine_ep_get_dispatch_amd import binding as ep
from operator_refs import UBF
from parity import announce
from test_gpu_expert_linear import gen, layer_inputs, quantised

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def code(text, first):
    """The block of Python code in ``text`` that begins with ``first``."""
    blocks = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if b.startswith(first)]
    assert len(blocks) == 1
    return blocks[0]


def test_training_step_gives_every_gradient():
    """Against automatic differentiation in 64 bits with the same routing and the
    normed rows rounded to bf16 as stored: the router's logits are a function of
    them, so x and the norm's weight get a share by way of the router.  Eleven
    roundings to bf16 at most on the way to a result (one more than without the
    router: the sum of the two shares), UBF each over the 2-norm."""
    announce("the training step of README.md")
    T, H, F, E, P, K = 96, 256, 128, 16, 4, 8
    s = layer_inputs(T, H, F, E, 310)
    # a share of the router's as large as the experts': it is seen if it is lost
    w_router = torch.randn((E, H), generator=gen(311)) / 8
    q1, s1 = quantised(s["w1"])
    q2, s2 = quantised(s["w2"])
    names = dict(x=s["x"], res=s["res"], norm_weight=s["nw"], w1=s["w1"], w2=s["w2"],
                 grad_out=s["go"], w_router=w_router, q1=q1, s1=s1, q2=q2, s2=s2)
    names = {k: v.cuda() for k, v in names.items()}
    names.update(torch=torch, ep=ep, num_experts=E, num_partitions=P)
    with open(README) as f:
        exec(compile(code(f.read(), "nm = ep.rms_norm("), README, "exec"), names)
    torch.cuda.synchronize()
    idx = names["idx"].cpu()
    assert idx.shape == (T, K)

    hr = (s["x"].double() + s["res"].double()).bfloat16().double().requires_grad_(True)
    nw, w1, w2, wr = (t.double().requires_grad_(True) for t in (s["nw"], s["w1"], s["w2"], w_router))
    n = hr * (hr.square().mean(1, keepdim=True) + 1e-6).rsqrt() * nw
    n = n + (names["nm"].y.cpu().double() - n).detach()
    wt = torch.softmax((n @ wr.t()).gather(1, idx), 1)
    res = torch.zeros((T, H), dtype=torch.float64)
    for k in range(K):
        a = torch.einsum("th,tfh->tf", n, w1[idx[:, k]])
        res = res + wt[:, k, None] * torch.einsum("tf,thf->th", ref.silu(a[:, :F]) * a[:, F:],
                                                  w2[idx[:, k]])
    ((res + hr) * s["go"].double()).sum().backward()
    for name, want in [("out", res.detach()), ("grad_x", hr.grad), ("grad_norm", nw.grad),
                       ("grad_w1", w1.grad), ("grad_w2", w2.grad), ("grad_router", wr.grad)]:
        off = float((names[name].cpu().double() - want).norm() / want.norm())
        assert off <= 11 * UBF, (name, off)

    # the FP8 experts behind it: rows in E4M3 twice, weights as quantised
    v1, v2 = ref.weight_values(q1, s1, F), ref.weight_values(q2, s2, H)
    n, wt = n.detach(), wt.detach()
    res = torch.zeros((T, H), dtype=torch.float64)
    for k in range(K):
        a = torch.einsum("th,tfh->tf", n, v1[idx[:, k]])
        res += wt[:, k, None] * torch.einsum("tf,thf->th", ref.gate(a, F)[0], v2[idx[:, k]])
    got = ep.combine(names["y"], names["d"].dst_row, names["w"]).cpu().double()
    assert float((got - res).norm() / res.norm()) <= 2 * ref.U8 + 6 * UBF
