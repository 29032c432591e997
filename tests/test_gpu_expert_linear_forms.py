"""The experts' products: which calls take a row's sums in eight shares."""
import pytest
import torch

from combine_ep_get_dispatch_amd import binding as ep
from parity import announce
from test_gpu_expert_linear import device, gen, ints

pytestmark = pytest.mark.gpu


def both(I, fp8, tiles, n):
    """Results of n rows alone in the call's only expert with rows, and beside an
    expert of 300 rows, which keeps the call from taking sums in shares."""
    N = tiles * 256
    g = gen(I + N)
    off = [0, n, n + 300]
    w = torch.randn((2, N, I), generator=g)
    x = torch.randn((off[2], I), generator=g)
    kw = {}
    if fp8:
        x, w = ((t * 60).to(torch.float8_e4m3fn).view(torch.uint8) for t in (x, w))
        kw = dict(x_scales=torch.rand((off[2], I // 128), generator=g).cuda() + 0.1,
                  weight_scales=torch.rand((2, N // 128, I // 128), generator=g).cuda() + 0.1)
    else:
        x, w = x.bfloat16(), w.bfloat16()
    out = []
    for counts in ([n, 0], [n, 300]):
        cnt, d_off = device(counts, off)
        out.append(ep.expert_linear(x.cuda(), w.cuda(), cnt, expert_offsets=d_off, **kw)[:n].cpu())
    return out


@pytest.mark.parametrize("I,fp8", [(256, False), (1024, False), (1472, False), (512, True),
                                   (2048, True), (2944, True)])
@pytest.mark.parametrize("tiles", [33, 64])
@pytest.mark.parametrize("n", [4, 32])
def test_two_rounds_of_short_sums_are_not_shared(I, fp8, tiles, n):
    """More tasks than one round holds of rows of fewer than 24 steps of 128 bytes: in
    shares they take up to 1.8 times as long, so a row has the bits that it has in a
    larger call."""
    announce("expert_linear I=%d fp8=%d tiles=%d rows=%d" % (I, fp8, tiles, n))
    alone, beside = both(I, fp8, tiles, n)
    assert torch.equal(alone, beside)


@pytest.mark.parametrize("I,fp8,tiles", [(128, False, 32), (2048, False, 64), (256, True, 32),
                                         (3200, True, 64)])
def test_few_tasks_are_shared_and_near(I, fp8, tiles):
    """Shared sums are off by their roundings: I + 8 steps of 2 * 2^-24 of the sum of the
    terms' sizes on either side, and E4M3 products cut at 2^-13 of eight neighbours', then
    a rounding to bf16 on either side."""
    alone, beside = both(I, fp8, tiles, 9)
    a, b = alone.double(), beside.double()
    size = float(a.abs().max()) * 4
    # a sum of I terms of random signs is near I^-1/2 of the sum of their sizes
    terms = size * I ** 0.5
    tol = 2 * ((I + 8) * 2 * 2.0 ** -24 + (8 * 2.0 ** -13 if fp8 else 0)) * terms
    assert bool(((a - b).abs() <= tol + 2.0 ** -7 * a.abs()).all())


@pytest.mark.parametrize("n", [65, 129, 200, 256, 300, 600])
@pytest.mark.parametrize("I,N", [(256, 256), (520, 200), (72, 264), (1032, 520)])
def test_one_to_nine_tasks_in_pieces(n, I, N):
    """Calls of so few tasks that an XCD has one, whose rows its workgroups share: exact in
    small integers."""
    announce("expert_linear and gradients of %d rows %d -> %d" % (n, I, N))
    g = gen(n + I)
    x, w, gy = ints((n, I), g), ints((1, N, I), g, 2), ints((n, N), g, 2)
    cnt, off = device([n], [0, n])
    xb, wb, gb = (t.bfloat16().cuda() for t in (x, w, gy))
    y = ep.expert_linear(xb, wb, cnt, expert_offsets=off)
    assert torch.equal(y.cpu().double(), (x @ w[0].t()).bfloat16().double())
    gx, gw = ep.expert_linear_backward(gb, xb, wb, cnt, expert_offsets=off,
                                       grad_weight_dtype=torch.float32)
    assert torch.equal(gx.cpu().double(), (gy @ w[0]).bfloat16().double())
    assert torch.equal(gw[0].cpu().double(), gy.t() @ x)
    only = ep.expert_linear_backward(gb, xb, None, cnt, expert_offsets=off,
                                     grad_weight_dtype=torch.float32)[1]
    assert torch.equal(only, gw)
    if I % 128 == 0:
        q = lambda t: t.float().to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        y8 = ep.expert_linear(q(x), q(w), cnt, expert_offsets=off,
                              x_scales=torch.ones((n, I // 128), device="cuda"),
                              weight_scales=torch.ones((1, (N + 127) // 128, I // 128), device="cuda"))
        assert torch.equal(y8, y)
