"""The norm of rows whose squares lie outside fp32's range, and its gradient there."""
import math

import pytest
import torch

import layer_refs as ref
from combine_ep_get_dispatch_amd import binding as ep
from operator_refs import e4m3_values
from parity import announce
from test_gpu_expert_linear import gen, within

pytestmark = pytest.mark.gpu

# 1 / rms is subnormal in fp32 where rms passes 2^126: half a step of 2^-149 of at least 2^-128
SUBNORMAL = 2.0 ** -22


def rows(H, seed, scales):
    """Rows of about the size of each of ``scales``, which bf16 holds."""
    x = torch.randn((len(scales), H), generator=gen(seed)).clamp(-3.5, 3.5).double()
    x = (x * torch.tensor(scales, dtype=torch.float64)[:, None]).bfloat16()
    assert bool(torch.isfinite(x).all())
    return x


LARGE = [2.0 ** k for k in (126, 125, 100, 70, 64, 63, 60, 57, 56, 40, 0, -60)]
SMALL = [2.0 ** k for k in (-125, -110, -80, -76, -75, -74, -70, -64, -42, -41, -40, -39, -38, -10, 0)]


@pytest.mark.parametrize("w32", [False, True])
@pytest.mark.parametrize("H", [8, 128, 504, 2048, 7168, 24576])
@pytest.mark.parametrize("scales,eps", [(LARGE, 1e-6), (LARGE, 0.0), (SMALL, 0.0), (SMALL, 1e-38),
                                        (SMALL, 1e-6), (SMALL, 2.0 ** -81)])
def test_rows_of_any_size(scales, eps, H, w32):
    announce("rms_norm of rows %g..%g H=%d eps=%g w32=%d" % (min(scales), max(scales), H, eps, w32))
    x = rows(H, H + len(scales), scales)
    # one row of small channels beside a large one, whose squares are the sum
    x[4, 1:] = torch.randn(H - 1, generator=gen(H)).bfloat16()
    w = 1 + 0.3 * torch.randn(H, generator=gen(H + 1))
    w = w if w32 else w.bfloat16()
    fp8 = H % 128 == 0
    o = ep.rms_norm(x.cuda(), w.cuda(), eps=eps, fp8=fp8)
    e = float(torch.tensor(eps, dtype=torch.float32))
    y, tol, inv, itol = ref.norm(x, w, e)
    tol = tol + SUBNORMAL * y.abs()
    within(o.inv_rms, inv, itol + (ref.U32 + SUBNORMAL) * inv, "inv_rms")
    within(o.y, y, ref.bf16_tol(y, tol), "y")
    if fp8:
        s, stol, v, vtol = ref.to_e4m3(y, tol)
        within(o.scales, s, stol + ref.U32 * s, "scales")
        got = e4m3_values()[o.codes.cpu().long()] * o.scales.cpu().double().repeat_interleave(128, 1)
        within(got, v, vtol, "codes")
    for t in range(len(scales)):             # the way back
        gy = rows(H, 7 * H + t, [min(max(scales[t], 2.0 ** -60), 2.0 ** 60)])
        args = (gy, x[t:t + 1].contiguous(), w, o.inv_rms[t:t + 1].cpu())
        gx, gw = ep.rms_norm_backward(*(a.cuda() for a in args))
        wx, tx, ww, tw = ref.norm_backward(*args, None)
        within(gx, wx, ref.bf16_tol(wx, tx), "grad_x of row %d" % t)
        within(gw, ww, tw + ref.U32 * ww.abs(), "grad_weight of row %d" % t)


def test_residual_rows_of_any_size():
    """The sum of two large rows, as stored; one that passes bf16's range stays in its row."""
    H = 640
    x, res = rows(H, 5, LARGE), rows(H, 6, [2.0 ** -3 * s for s in LARGE])
    x[0, 9], res[0, 9] = 3e38, 2e38
    w = torch.ones(H)
    o = ep.rms_norm(x.cuda(), w.cuda(), residual=res.cuda())
    h = (x.double() + res.double()).bfloat16()
    assert torch.equal(o.residual.cpu(), h) and math.isinf(float(h[0, 9]))
    assert float(o.inv_rms[0]) == 0 and bool(torch.isnan(o.y[0, 9]))
    y, tol, inv, itol = ref.norm(h[1:], w, 1e-6)
    within(o.inv_rms[1:], inv, itol + (ref.U32 + SUBNORMAL) * inv, "inv_rms")
    within(o.y[1:], y, ref.bf16_tol(y, tol + SUBNORMAL * y.abs()), "y")


def test_rows_whose_inverse_passes_the_range():
    """With eps 0: rows of subnormals have y, and an inverse norm in fp32 up to
    2^128; a row of zeros has neither.  Of row 0, whole numbers up to 63 of even
    spread, the mean square is (63 + 1)(2 * 63 + 1) / 6 = 1355 of 2^-266, near
    2^-255.6, so the inverse is near 2^127.8; of row 2 it is 16 * 2^133."""
    H = 256
    x = torch.zeros((3, H), dtype=torch.bfloat16)
    x[0] = (torch.randint(1, 64, (H,), generator=gen(1)).double() * 2.0 ** -133).bfloat16()
    x[2, 3] = 2.0 ** -133
    w = torch.ones(H)
    o = ep.rms_norm(x.cuda(), w.cuda(), eps=0.0)
    y, tol, inv, itol = ref.norm(x, w, 0.0)
    for t in (0, 2):
        within(o.y[t], y[t], ref.bf16_tol(y, tol)[t], "y")
    within(o.inv_rms[:1], inv[:1], (itol + ref.U32 * inv)[:1], "inv_rms")
    assert float(o.inv_rms[2]) == math.inf
    assert bool(torch.isnan(o.y[1]).all())
