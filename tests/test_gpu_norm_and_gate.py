"""The root-mean-square norm, the gated activation and their gradients on the
GPU against plain 64-bit references (layer_refs.py derives the bounds)."""
import math

import pytest
import torch

import layer_refs as ref
from combine_ep_get_dispatch_amd import binding as ep
from operator_refs import e4m3_values
from parity import announce
from test_gpu_expert_linear import device, gen, place, poison, within

pytestmark = pytest.mark.gpu

NORM = [  # T, H, residual, bf16, fp8, fp32 weight
    (1, 8, False, True, False, False),
    (1, 128, True, True, True, True),
    (3, 128, False, False, True, False),
    (5, 504, True, True, False, False),
    (7, 512, True, True, True, False),
    (33, 520, False, True, False, True),
    (2, 2048, True, False, True, True),
    (9, 2056, True, True, False, False),
    (4, 4096, False, True, True, False),
    (600, 1152, True, True, True, False),
    (3, 7168, True, True, True, False),
    (2, 8200, True, True, False, True),
    (2, 16384, False, True, True, False),
    (3, 24576, True, True, True, True),
    (1, 32768, True, True, False, False),
]


def norm_inputs(T, H, residual, w32, seed):
    g = gen(seed)
    x = (torch.randn((T, H), generator=g) * torch.rand((T, 1), generator=g) * 3).bfloat16()
    res = torch.randn((T, H), generator=g).bfloat16() if residual else None
    w = 1 + 0.3 * torch.randn(H, generator=g)
    return x, res, w if w32 else w.bfloat16(), g


@pytest.mark.parametrize("T,H,residual,bf16,fp8,w32", NORM, ids=["%dx%d_%d%d%d%d" % c for c in NORM])
def test_norm(T, H, residual, bf16, fp8, w32):
    announce("rms_norm T=%d H=%d residual=%d bf16=%d fp8=%d w32=%d" % (T, H, residual, bf16, fp8, w32))
    x, res, w, _ = norm_inputs(T, H, residual, w32, T + H)
    if H > 200:
        x[0, :130] = 0                       # a group of zeros, or nearly
        if residual:
            res[0, :130] = 0
    eps = 1e-5
    o = ep.rms_norm(x.cuda(), w.cuda(), eps=eps, residual=None if res is None else res.cuda(),
                    bf16=bf16, fp8=fp8)
    torch.cuda.synchronize()
    h = x if res is None else (x.double() + res.double()).bfloat16()
    if residual:
        assert torch.equal(o.residual.cpu(), h)
    else:
        assert o.residual is None
    y, tol, inv, itol = ref.norm(h, w, eps)
    within(o.inv_rms, inv, itol + ref.U32 * inv, "inv_rms")
    assert (o.y is not None) == bf16 and (o.codes is not None) == fp8
    if bf16:
        within(o.y, y, ref.bf16_tol(y, tol), "y")
    if fp8:
        s, stol, v, vtol = ref.to_e4m3(y, tol)
        within(o.scales, s, stol + ref.U32 * s, "scales")
        got = e4m3_values()[o.codes.cpu().long()] * o.scales.cpu().double().repeat_interleave(128, 1)
        within(got, v, vtol, "codes")


def test_norm_of_rows_that_are_not_numbers():
    """A NaN or infinity stays in its row, whose codes are then S.1111.111 where
    y is not a number; a row of zeros gives zeros."""
    T, H = 6, 384
    x, _, w, _ = norm_inputs(T, H, False, False, 5)
    x[1, 3] = math.inf
    x[2, 200] = float("nan")
    x[4] = 0
    o = ep.rms_norm(x.cuda(), w.cuda(), fp8=True)
    y, codes, inv = o.y.cpu().float(), o.codes.cpu(), o.inv_rms.cpu()
    for t in (0, 3, 5):
        assert bool(torch.isfinite(y[t]).all()) and bool(((codes[t] & 0x7F) != 0x7F).all())
    assert bool((y[4] == 0).all()) and bool(((codes[4] & 0x7F) == 0).all())
    assert float(inv[1]) == 0 and bool(torch.isnan(inv[2]))
    assert bool(torch.isnan(y[1, 3])) and bool((y[1, 4:] == 0).all())
    assert int(codes[1, 3]) & 0x7F == 0x7F and bool(((codes[1, 4:] & 0x7F) == 0).all())
    assert bool(torch.isnan(y[2]).all()) and bool(((codes[2] & 0x7F) == 0x7F).all())


BACK = [(T, H, r, w32) for (T, H, w32) in
        [(1, 8, True), (2, 128, False), (5, 504, False), (513, 520, True), (700, 64, False),
         (1025, 256, False), (40, 2056, False), (3, 7168, True), (600, 4104, False),
         (2, 8200, False), (3, 16384, True), (2, 32768, False)] for r in (False, True)]


@pytest.mark.parametrize("T,H,residual,w32", BACK, ids=["%dx%d_%d_%d" % c for c in BACK])
def test_norm_backward(T, H, residual, w32):
    announce("rms_norm_backward T=%d H=%d residual=%d w32=%d" % (T, H, residual, w32))
    x, _, w, g = norm_inputs(T, H, False, w32, 3 * T + H)
    gy = torch.randn((T, H), generator=g).bfloat16()
    gres = torch.randn((T, H), generator=g).bfloat16() if residual else None
    inv = ref.norm(x, w, 1e-6)[2].float()
    args = (gy.cuda(), x.cuda(), w.cuda(), inv.cuda())
    kw = dict(grad_residual=None if gres is None else gres.cuda())
    gx, gw = ep.rms_norm_backward(*args, **kw)
    torch.cuda.synchronize()
    wx, tx, ww, tw = ref.norm_backward(gy, x, w, inv, gres)
    within(gx, wx, ref.bf16_tol(wx, tx), "grad_x")
    within(gw, ww, tw + ref.U32 * ww.abs(), "grad_weight")
    n = ep.rms_norm_backward_workspace_bytes(T, H)
    ws = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    again = ep.rms_norm_backward(*args, workspace=ws[:n], **kw)
    assert torch.equal(again[0], gx) and torch.equal(again[1], gw)
    assert bool((ws[n:] == 0xFF).all())


def test_norm_of_no_tokens():
    w = torch.ones(256, device="cuda")
    none = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    o = ep.rms_norm(none, w, residual=none, fp8=True)
    assert o.y.shape == (0, 256) and o.scales.shape == (0, 2)
    gx, gw = ep.rms_norm_backward(none, none, w, o.inv_rms)
    assert gx.shape == (0, 256) and bool((gw == 0).all())


def test_norm_gradient_against_differences():
    """grad_weight against differences of y (linear in the weight, y in bf16 is
    off by UBF of its size), grad_x against central differences of the 64-bit
    reference with a step of 2^-10: third derivatives times h^2 and y's
    cancellation stay under 1e-4 of the gradient's size here."""
    T, H, h = 3, 64, 2.0 ** -10
    x, _, w, g = norm_inputs(T, H, False, True, 77)
    gy = torch.randn((T, H), generator=g).bfloat16()
    o = ep.rms_norm(x.cuda(), w.cuda())
    gx, gw = ep.rms_norm_backward(gy.cuda(), x.cuda(), w.cuda(), o.inv_rms)
    up = ep.rms_norm(x.cuda(), (w + 1).cuda()).y.cpu().double()
    y = o.y.cpu().double()
    diff = ((up - y) * gy.double()).sum(0)
    tol = (ref.UBF * (up.abs() + y.abs()) * gy.double().abs()).sum(0)
    within(gw, diff, tol + 1e-5, "grad_weight")
    for t, i in [(0, 0), (1, 33), (2, 63)]:
        a, b = x.double().clone(), x.double().clone()
        a[t, i] += h
        b[t, i] -= h
        d = ((ref.norm(a, w, 1e-6)[0] - ref.norm(b, w, 1e-6)[0]) * gy.double()).sum() / (2 * h)
        size = float((gy.double() * y).abs().sum() / x[t].double().norm())
        assert abs(float(gx[t, i]) - float(d)) <= (ref.UBF + 1e-4) * size


GATE = [  # counts, N, form
    (None, 8, None), (None, 200, None), (None, 4096, None), ([1], 128, "offsets"),
    ([0, 3, 0, 70, 1], 64, "offsets"), ([5, 0, 64, 65, 63, 1], 1000, "aligned"),
    ([3, 40, 12], 264, "capacity"), ([2, 1] * 150, 128, "capacity"), ([700, 5], 136, "aligned"),
    ([130, 1], 8192, "offsets"), ([0, 0], 128, "offsets"),
]
GATE_IDS = ["%s_%d_%s" % ("all" if c is None else "E%d" % len(c), n, f) for c, n, f in GATE]


def gate_inputs(counts, N, form, seed):
    g = gen(seed)
    if counts is None:
        off, C, R, d_cnt, d_off, runs = None, 0, 61, None, None, [(0, 61)]
    else:
        off, C, R = place(counts, form)
        d_cnt, d_off = device(counts, off)
        runs = ref.ranges(counts, off, C, R)
    a = (torch.randn((R, 2 * N), generator=g) * 3).bfloat16()
    a, hold = poison(a, runs, float("nan"))
    b, n = max(runs, key=lambda v: v[1])
    if n > 0:                                # values far out
        a[b, :4] = torch.tensor([-200.0, 200.0, -88.0, -1e30])
        a[b, N:N + 4] = torch.tensor([3.0, 1e20, 100.0, 2.0])
    return a, hold, dict(num_tokens_per_expert=d_cnt, expert_offsets=d_off, capacity=C), R, g


@pytest.mark.parametrize("counts,N,form", GATE, ids=GATE_IDS)
def test_gate(counts, N, form):
    announce("expert_swiglu %s N=%d %s" % (counts if counts is None else len(counts), N, form))
    a, hold, rows, R, _ = gate_inputs(counts, N, form, N)
    want, tol = ref.gate(a, N)
    y = torch.full((R, N), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.expert_swiglu(a.cuda(), out=y, **rows)
    assert bool((y.cpu()[~hold] == 7.0).all())
    within(y.cpu()[hold], want[hold], ref.bf16_tol(want, tol)[hold], "y")
    if N % 128:
        return
    codes = torch.full((R, N), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((R, N // 128), 7.0, device="cuda")
    ep.expert_swiglu(a.cuda(), fp8=True, out=(codes, scales), **rows)
    c, s = codes.cpu(), scales.cpu()
    assert bool((c[~hold] == 0x55).all()) and bool((s[~hold] == 7.0).all())
    ws, ts, wv, tv = ref.to_e4m3(want, tol)
    within(s[hold], ws[hold], (ts + ref.U32 * ws)[hold], "scales")
    got = e4m3_values()[c.long()] * s.double().repeat_interleave(128, 1)
    within(got[hold], wv[hold], tv[hold], "codes")


@pytest.mark.parametrize("counts,N,form", GATE, ids=GATE_IDS)
def test_gate_backward(counts, N, form):
    announce("expert_swiglu_backward %s N=%d %s" % (counts if counts is None else len(counts), N,
                                                    form))
    a, hold, rows, R, g = gate_inputs(counts, N, form, N + 1)
    gy = torch.randn((R, N), generator=g).bfloat16()
    gy[~hold] = float("nan")
    out = torch.full((R, 2 * N), 7.0, dtype=torch.bfloat16, device="cuda")
    ep.expert_swiglu_backward(gy.cuda(), a.cuda(), out=out, **rows)
    want, tol = ref.gate_backward(gy, a, N)
    got = out.cpu()
    assert bool((got[~hold] == 7.0).all())
    within(got[hold], want[hold], ref.bf16_tol(want, tol)[hold], "gradient")


def test_gate_codes_of_values_that_are_not_numbers():
    N = 256
    a = torch.randn((3, 2 * N), generator=gen(2)).bfloat16()
    a[1, 5], a[1, N + 5] = math.inf, -1.0
    a[2, 130] = float("nan")
    c, s = (t.cpu() for t in ep.expert_swiglu(a.cuda(), fp8=True))
    assert int(c[1, 5]) == 0xFF and math.isinf(float(s[1, 0]))
    assert bool(((c[1, :128] & 0x7F) == 0)[torch.arange(128) != 5].all())
    assert int(c[2, 130]) & 0x7F == 0x7F and math.isfinite(float(s[2, 1]))
    assert bool(((c[0] & 0x7F) != 0x7F).all()) and bool(((c[2, :128] & 0x7F) != 0x7F).all())


def test_gate_gradient_against_differences():
    """Against central differences of the 64-bit reference, step 2^-12: third
    derivatives of silu are below 1, so h^2 of the terms' size; then UBF."""
    N, h = 16, 2.0 ** -12
    g = gen(8)
    a, gy = torch.randn((4, 2 * N), generator=g).bfloat16(), torch.randn((4, N), generator=g).bfloat16()
    got = ep.expert_swiglu_backward(gy.cuda(), a.cuda()).cpu().double()
    for r in range(4):
        for c in (0, 7, 15, 16, 20, 31):
            up, dn = a.double().clone(), a.double().clone()
            up[r, c] += h
            dn[r, c] -= h
            d = float(((ref.gate(up, N)[0] - ref.gate(dn, N)[0]) * gy.double()).sum() / (2 * h))
            size = float((gy[r, c % N].double() * a[r, N + c % N].double()).abs()) + abs(d)
            assert abs(float(got[r, c]) - d) <= ref.UBF * abs(d) + (h * h + 1e-8) * size + 1e-9


def test_operators_on_another_stream_and_unaligned_rows_of_a_buffer():
    """Outputs that are a slice of a larger buffer keep what lies beside them."""
    T, H = 9, 136
    x, res, w, g = norm_inputs(T, H, True, False, 4)
    big = torch.full((T + 2, H), 3.0, dtype=torch.bfloat16, device="cuda")
    hbuf = big.clone()
    inv = torch.empty(T, device="cuda")
    out = ep.RmsNormed(big[1:T + 1], None, None, hbuf[1:T + 1], inv)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ep.rms_norm(x.cuda(), w.cuda(), residual=res.cuda(), out=out)
    torch.cuda.synchronize()
    ref_o = ep.rms_norm(x.cuda(), w.cuda(), residual=res.cuda())
    assert torch.equal(big[1:T + 1], ref_o.y) and torch.equal(hbuf[1:T + 1], ref_o.residual)
    assert bool((big[[0, T + 1]] == 3.0).all()) and bool((hbuf[[0, T + 1]] == 3.0).all())
