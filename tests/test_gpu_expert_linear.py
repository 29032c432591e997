"""The experts' products in bf16 and E4M3 and their gradients on the GPU.

Most cases use small integers: every partial sum is then exact in fp32 in any
order, so the results have to be the reference's rounded once, bit for bit.
Rows of no expert hold NaN in every input and a sentinel in every output.
"""
import math

import pytest
import torch

import layer_refs as ref
from combine_ep_get_dispatch_amd import binding as ep
from operator_refs import UBF
from parity import announce

pytestmark = pytest.mark.gpu
NAN = float("nan")


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(got, want, tol, what=""):
    got = got.detach().cpu().double()
    look = ~torch.isnan(want)
    off = (got - want).abs()
    bad = look & ~(off <= tol)
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g over its bound" % (
        what, int(bad.sum()), bad.numel(), float((off / tol)[bad].nan_to_num(math.inf).max()))


def place(counts, form):
    """(offsets, capacity, R): runs one after the other, at multiples of 16 with
    two rows of nobody in front, or at multiples of a capacity that cuts the
    largest run."""
    if form == "capacity":
        C = max(1, max(counts) - 1)
        return None, C, len(counts) * C + 3
    step, at, off = (16, 2, []) if form == "aligned" else (1, 0, [])
    for n in counts:
        off.append(at)
        at += (n + step - 1) // step * step
    return off + [at], 0, at + 5


def ints(shape, g, top=4):
    return torch.randint(-top, top + 1, shape, generator=g).double()


def codes_of(v):
    """E4M3 codes of values that E4M3 holds."""
    t = v.float().to(torch.float8_e4m3fn)
    assert torch.equal(t.double(), v)
    return t.view(torch.uint8)


def device(counts, off):
    return (torch.tensor(counts, dtype=torch.int32).cuda(),
            None if off is None else torch.tensor(off, dtype=torch.int32).cuda())


def poison(t, runs, value):
    """t with ``value`` in the rows of no expert."""
    hold = torch.zeros(t.shape[0], dtype=torch.bool)
    for b, n in runs:
        hold[b:b + n] = True
    t[~hold] = value
    return t, hold


# counts that meet every row tile's edge
EDGES = [0, 1, 7, 15, 16, 17, 31, 33, 47, 48, 63, 64, 65, 0, 100, 127, 128, 129, 191, 192, 193,
         255, 256, 257, 320, 0]
# E, I, N, counts, form
SHAPES = [
    ([1], 8, 8, "offsets"),
    ([1], 2048, 520, "capacity"),
    ([0, 0, 3, 0], 64, 16, "offsets"),
    ([0, 0, 0], 64, 16, "offsets"),
    ([2, 3, 5, 1], 56, 264, "aligned"),
    ([16, 17, 40], 72, 1000, "capacity"),
    (EDGES, 136, 304, "offsets"),
    (EDGES, 64, 256, "aligned"),
    (EDGES[::-1], 1032, 72, "capacity"),
    ([300, 5, 700, 64], 520, 264, "aligned"),
    ([600], 256, 512, "offsets"),
    ([9, 1, 4] * 100, 128, 128, "offsets"),
    ([3] * 1024, 24, 8, "capacity"),
    ([200] * 24, 64, 1024, "offsets"),       # what is left of a round, in halves
    ([200] * 72 + [60], 64, 1032, "offsets"),    # a whole round and a rest, in quarters
    ([64] * 3, 1160, 520, "capacity"),       # few tasks, more steps than waves
    ([30, 31], 2056, 264, "offsets"),
]
IDS = ["E%d_%dto%d_%s" % (len(c), i, n, f) for c, i, n, f in SHAPES]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,I,N,form", SHAPES, ids=IDS)
def test_linear_bf16(counts, I, N, form, swiglu):
    announce("expert_linear bf16 E=%d I=%d N=%d %s swiglu=%d" % (len(counts), I, N, form, swiglu))
    g = gen(I + N)
    off, C, R = place(counts, form)
    runs = ref.ranges(counts, off, C, R)
    W = 2 * N if swiglu else N
    x, w = ints((R, I), g), ints((len(counts), W, I), g, 2)
    x, hold = poison(x, runs, NAN)
    for e, (_, n) in enumerate(runs):
        if n == 0:
            w[e] = NAN                       # weights that no row meets
    want, _ = ref.linear(x, w, runs, N, swiglu)
    d_cnt, d_off = device(counts, off)
    y = torch.full((R, N), 77.0, dtype=torch.bfloat16, device="cuda")
    kw = dict(expert_offsets=d_off, capacity=C, swiglu=swiglu)
    ep.expert_linear(x.bfloat16().cuda(), w.bfloat16().cuda(), d_cnt, out=y, **kw)
    torch.cuda.synchronize()
    got = y.cpu()
    assert bool((got[~hold] == 77.0).all())
    if swiglu:                               # the sums are exact; silu's own, |up| < 2^15
        gate, _ = ref.linear(x, w[:, :N], runs, N, False)
        tol = ref.silu_steps(gate) * ref.U32 * want.abs() + 2.0 ** 15 * ref.LOST
        within(got[hold], want[hold], ref.bf16_tol(want, tol)[hold], "y")
    else:
        assert torch.equal(got[hold].double(), want[hold].bfloat16().double())


FP8_SHAPES = [
    ([1], 128, 8, "offsets"),
    ([1, 0, 2], 2048, 136, "capacity"),
    ([5, 16, 17, 0, 40], 384, 1000, "aligned"),
    (EDGES, 256, 264, "offsets"),
    (EDGES, 128, 128, "capacity"),
    ([300, 5, 700, 64], 512, 512, "aligned"),
    ([9, 1, 4] * 100, 256, 64, "offsets"),
    ([200] * 24, 128, 1024, "offsets"),
    ([200] * 72 + [60], 128, 1032, "offsets"),
    ([64] * 3, 1152, 520, "capacity"),
    ([30, 31], 1920, 264, "offsets"),
    ([16], 1408, 200, "offsets"),
]


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts,I,N,form", FP8_SHAPES,
                         ids=["E%d_%dto%d_%s" % (len(c), i, n, f) for c, i, n, f in FP8_SHAPES])
def test_linear_fp8(counts, I, N, form, swiglu):
    """Integers up to 4 and scales of 1, 2 or 4: exact in any order."""
    announce("expert_linear fp8 E=%d I=%d N=%d %s swiglu=%d" % (len(counts), I, N, form, swiglu))
    g = gen(I * 3 + N)
    off, C, R = place(counts, form)
    runs = ref.ranges(counts, off, C, R)
    E, W, S = len(counts), N * (1 + swiglu), (N + 127) // 128 * (1 + swiglu)
    x, w = codes_of(ints((R, I), g)), codes_of(ints((E, W, I), g, 2))
    xs = 2.0 ** torch.randint(0, 3, (R, I // 128), generator=g).float()
    ws = 2.0 ** torch.randint(0, 3, (E, S, I // 128), generator=g).float()
    if swiglu:
        ws /= 64
    x, hold = poison(x, runs, 0x7F)
    xs, _ = poison(xs, runs, NAN)
    want, _ = ref.linear(ref.fp8_values(x, xs), ref.weight_values(w, ws, N), runs, N, swiglu)
    d_cnt, d_off = device(counts, off)
    y = torch.full((R, N), 77.0, dtype=torch.bfloat16, device="cuda")
    ep.expert_linear(x.cuda(), w.cuda(), d_cnt, expert_offsets=d_off, capacity=C,
                     x_scales=xs.cuda(), weight_scales=ws.cuda(), swiglu=swiglu, out=y)
    torch.cuda.synchronize()
    got = y.cpu()
    assert bool((got[~hold] == 77.0).all())
    if swiglu:                               # |up| < 2^15
        values = ref.weight_values(w, ws, N)[:, :N]
        gate, _ = ref.linear(ref.fp8_values(x, xs), values, runs, N, False)
        tol = ref.silu_steps(gate) * ref.U32 * want.abs() + 2.0 ** 15 * ref.LOST
        within(got[hold], want[hold], ref.bf16_tol(want, tol)[hold], "y")
    else:
        assert torch.equal(got[hold].double(), want[hold].bfloat16().double())


BACK = SHAPES + [([129, 64, 1], 1000, 200, "aligned"), ([70, 0, 513], 264, 520, "offsets")]


@pytest.mark.parametrize("gw", ["bf16", "fp32", "add"])
@pytest.mark.parametrize("counts,I,N,form", BACK,
                         ids=["E%d_%dto%d_%s" % (len(c), i, n, f) for c, i, n, f in BACK])
def test_linear_backward(counts, I, N, form, gw):
    announce("expert_linear_backward E=%d I=%d N=%d %s %s" % (len(counts), I, N, form, gw))
    g = gen(I + 7 * N)
    off, C, R = place(counts, form)
    runs = ref.ranges(counts, off, C, R)
    E = len(counts)
    x, gy, w = ints((R, I), g), ints((R, N), g, 2), ints((E, N, I), g, 2)
    x, hold = poison(x, runs, NAN)
    gy, _ = poison(gy, runs, math.inf)
    old = ints((E, N, I), g, 100) if gw == "add" else torch.full((E, N, I), NAN,
                                                                 dtype=torch.float64)
    want_x = torch.full((R, I), 55.0, dtype=torch.float64)
    want_w = torch.zeros((E, N, I), dtype=torch.float64)
    for e, (b, n) in enumerate(runs):
        if n == 0:
            w[e] = NAN
            continue
        want_x[b:b + n] = gy[b:b + n] @ w[e]
        want_w[e] = gy[b:b + n].t() @ x[b:b + n]
    if gw == "add":
        want_w += old
    dt = torch.bfloat16 if gw == "bf16" else torch.float32
    d_cnt, d_off = device(counts, off)
    gx = torch.full((R, I), 55.0, dtype=torch.bfloat16, device="cuda")
    gwt = old.to(dt).cuda()
    d = [t.bfloat16().cuda() for t in (gy, x, w)]
    ep.expert_linear_backward(*d, d_cnt, expert_offsets=d_off, capacity=C, accumulate=gw == "add",
                              out=(gx, gwt))
    torch.cuda.synchronize()
    assert torch.equal(gx.cpu().double(), want_x.bfloat16().double())
    assert torch.equal(gwt.cpu().double(), want_w.to(dt).double())
    if gw == "fp32":                         # each half by itself
        a = ep.expert_linear_backward(d[0], None, d[2], d_cnt, expert_offsets=d_off, capacity=C,
                                      out=(gx.clone().fill_(55.0), None))
        b = ep.expert_linear_backward(d[0], d[1], None, d_cnt, expert_offsets=d_off, capacity=C,
                                      grad_weight_dtype=torch.float32)
        assert a[1] is None and b[0] is None
        assert torch.equal(a[0], gx) and torch.equal(b[1], gwt)


def random_case(E, I, N, counts, seed, swiglu=False):
    g = gen(seed)
    off, C, R = place(counts, "aligned")
    x = torch.randn((R, I), generator=g)
    w = torch.randn((E, N * (1 + swiglu), I), generator=g) / math.sqrt(I)
    return off, C, R, x, w, g


@pytest.mark.parametrize("swiglu", [False, True])
def test_linear_of_random_values(swiglu):
    counts, I, N = [70, 3, 260, 18], 704, 200
    off, C, R, x, w, _ = random_case(4, I, N, counts, 3, swiglu)
    x, w = x.bfloat16(), w.bfloat16()
    runs = ref.ranges(counts, off, C, R)
    want, tol = ref.linear(x.double(), w.double(), runs, N, swiglu)
    d_cnt, d_off = device(counts, off)
    y = ep.expert_linear(x.cuda(), w.cuda(), d_cnt, expert_offsets=d_off, swiglu=swiglu)
    within(y, want, ref.bf16_tol(want, tol), "bf16")
    # the same product in E4M3, rows as dispatch's rule gives them
    I8 = 640
    xv, wv = x[:, :I8].double(), w[:, :, :I8].double()
    a = xv.view(R, I8 // 128, 128).abs().amax(2).clamp(min=1e-4)
    xs = (a / 448).float()
    xc = (xv.view(R, I8 // 128, 128) / xs.double()[..., None]).float()
    xc = xc.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(R, I8)
    S = (N + 127) // 128 * (1 + swiglu)
    ws = torch.rand((4, S, I8 // 128), generator=gen(4)) * 1e-3 + 1e-4
    wc = (torch.randn((4, N * (1 + swiglu), I8), generator=gen(5)) * 60).to(
        torch.float8_e4m3fn).view(torch.uint8)
    want, tol = ref.linear(ref.fp8_values(xc, xs), ref.weight_values(wc, ws, N), runs, N, swiglu,
                           cut=2.0 ** -13)
    y = ep.expert_linear(xc.cuda(), wc.cuda(), d_cnt, expert_offsets=d_off, x_scales=xs.cuda(),
                         weight_scales=ws.cuda(), swiglu=swiglu)
    within(y, want, ref.bf16_tol(want, tol), "fp8")


def test_large_sums_of_integers():
    """Many channels, many rows: long sums, exact."""
    counts, I, N = [1500, 37, 900], 4104, 1032
    g = gen(11)
    off, C, R = place(counts, "offsets")
    x = torch.randint(-2, 3, (R, I), generator=g).bfloat16().cuda()
    w = torch.randint(-2, 3, (3, N, I), generator=g).bfloat16().cuda()
    gy = torch.randint(-2, 3, (R, N), generator=g).bfloat16().cuda()
    d_cnt, d_off = device(counts, off)
    y = ep.expert_linear(x, w, d_cnt, expert_offsets=d_off)
    gx, gw = ep.expert_linear_backward(gy, x, w, d_cnt, expert_offsets=d_off,
                                       grad_weight_dtype=torch.float32)
    for e, n in enumerate(counts):
        r = slice(off[e], off[e] + n)
        assert torch.equal(y[r], (x[r].float() @ w[e].float().t().contiguous()).bfloat16())
        assert torch.equal(gx[r], (gy[r].float() @ w[e].float()).bfloat16())
        assert torch.equal(gw[e], gy[r].float().t().contiguous() @ x[r].float())
    again = ep.expert_linear(x, w, d_cnt, expert_offsets=d_off)
    assert torch.equal(again[:off[-1]], y[:off[-1]])


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_beside_a_row_do_not_change_its_bits(fp8):
    """The same rows alone in their expert and among many, in blocks of every
    size, give the same bits (many experts: sums are not taken in shares)."""
    E, I, N = 80, 640, 264
    g = gen(61)
    few, many = [9] * E, [9] * E
    many[0], many[1], many[2], many[3] = 300, 200, 100, 50
    w = torch.randn((E, N, I), generator=g)
    rows = torch.randn((sum(many), I), generator=g)
    keep, at = [], 0
    for n in many:
        keep += list(range(at, at + 9))
        at += n
    kw = {}
    if fp8:
        q = lambda t: (t * 60).to(torch.float8_e4m3fn).view(torch.uint8)
        w, rows = q(w), q(rows)
        xs = torch.rand((rows.shape[0], I // 128), generator=g) * 0.01 + 0.001
        kw["weight_scales"] = (torch.rand((E, 3, I // 128), generator=g) * 0.01).cuda()
    else:
        w, rows = w.bfloat16(), rows.bfloat16()
    out = []
    for counts, x in ((few, rows[keep]), (many, rows)):
        off = [0]
        for n in counts:
            off.append(off[-1] + n)
        cnt, d_off = device(counts, off)
        if fp8:
            kw["x_scales"] = (xs[keep] if x.shape[0] < rows.shape[0] else xs).contiguous().cuda()
        out.append(ep.expert_linear(x.contiguous().cuda(), w.cuda(), cnt, expert_offsets=d_off,
                                    **kw).cpu())
    assert torch.equal(out[0], out[1][keep])


def test_values_that_are_not_numbers_stay_in_their_row():
    """An infinity or NaN in a row or a weight reaches the results that use it
    and no others."""
    counts, I, N = [40, 200, 9], 200, 136
    off, C, R, x, w, _ = random_case(3, I, N, counts, 21)
    x[off[1] + 5, 7] = math.inf
    x[off[0] + 39, 199] = NAN
    w[2, 11, 3] = math.inf
    runs = ref.ranges(counts, off, C, R)
    x, _ = poison(x, runs, NAN)
    x, w = x.bfloat16(), w.bfloat16()
    d_cnt, d_off = device(counts, off)
    y = ep.expert_linear(x.cuda(), w.cuda(), d_cnt, expert_offsets=d_off).cpu()
    for e, (b, n) in enumerate(runs):
        for r in range(b, b + n):
            bad = torch.zeros(N, dtype=torch.bool)
            if r in (off[1] + 5, off[0] + 39):
                bad[:] = True
            if e == 2:
                bad[11] = True
            assert torch.equal(~torch.isfinite(y[r]), bad), r


@pytest.mark.parametrize("counts", [[40, 200, 9], [5, 20, 3]])
def test_codes_that_are_not_numbers_stay_in_their_row(counts):
    """The same in E4M3: a NaN code or an infinite scale of a row, a NaN code of a
    weight; in blocks and in the few tasks whose sums are taken in shares."""
    I, N = 256, 136
    g = gen(23)
    off, C, R = place(counts, "aligned")
    runs = ref.ranges(counts, off, C, R)
    x, w = codes_of(ints((R, I), g)), codes_of(ints((3, N, I), g, 2))
    xs, ws = torch.ones((R, I // 128)), torch.ones((3, 2, I // 128))
    x[off[1] + 5, 7] = 0x7F
    xs[off[0] + 2, 1] = math.inf
    w[2, 11, 200] = 0xFF
    x, _ = poison(x, runs, 0x7F)
    xs, _ = poison(xs, runs, NAN)
    d_cnt, d_off = device(counts, off)
    y = ep.expert_linear(x.cuda(), w.cuda(), d_cnt, expert_offsets=d_off, x_scales=xs.cuda(),
                         weight_scales=ws.cuda()).cpu()
    for e, (b, n) in enumerate(runs):
        for r in range(b, b + n):
            bad = torch.zeros(N, dtype=torch.bool)
            if r in (off[1] + 5, off[0] + 2):
                bad[:] = True
            if e == 2:
                bad[11] = True
            assert torch.equal(~torch.isfinite(y[r]), bad), r


def test_calls_on_two_streams_at_once():
    """Products, gradients, norm and activation of two sets of inputs, in flight
    on two streams at the same time, give what they give alone."""
    T, H, F, E, K = 300, 256, 128, 8, 2
    sets = [{k: v.cuda() for k, v in layer_inputs(T, H, F, E, 200 + i).items()} for i in range(2)]
    alone = [[t.clone() for t in training_step(s, E, K)] for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(training_step(s, E, K))
        torch.cuda.synchronize()
        for a, b in zip(got, alone):
            for u, v in zip(a, b):
                assert torch.equal(u, v)


def test_rows_past_the_end_and_empty_inputs():
    """Runs that reach past num_rows are cut; counts of zero and below are none;
    no rows at all leave gradients of 0."""
    I, N = 72, 40
    g = gen(31)
    x, w = ints((20, I), g).bfloat16().cuda(), ints((4, N, I), g).bfloat16().cuda()
    cnt = torch.tensor([3, 500, -4, 6], dtype=torch.int32).cuda()
    off = torch.tensor([-1, 10, 4, 20, 26], dtype=torch.int32).cuda()
    y = torch.full((22, N), 9.0, dtype=torch.bfloat16, device="cuda")
    ep.expert_linear(x, w, cnt, expert_offsets=off, out=y[:20])
    want = torch.full((22, N), 9.0)
    xf, wf = x.float().cpu(), w.float().cpu()
    want[0:2] = xf[0:2] @ wf[0].t()
    want[10:20] = xf[10:20] @ wf[1].t()
    assert torch.equal(y.cpu().float(), want.bfloat16().float())
    none = torch.empty((0, I), dtype=torch.bfloat16, device="cuda")
    assert ep.expert_linear(none, w, cnt, expert_offsets=off).shape == (0, N)
    gx, gw = ep.expert_linear_backward(none[:, :N].contiguous(), none, w, cnt, expert_offsets=off)
    assert gx.shape == (0, I) and bool((gw == 0).all())


def test_rows_and_weights_past_32_bits():
    """Rows and experts whose places pass 2^32 bytes, next to rows of nobody."""
    g = gen(51)
    R, I, N = 300000, 8192, 16
    cnt, off = device([3, 100], [5, R - 101, R - 1])
    x = torch.full((R, I), NAN, dtype=torch.bfloat16, device="cuda")
    gy = torch.full((R, N), NAN, dtype=torch.bfloat16, device="cuda")
    w = torch.randint(-1, 2, (2, N, I), generator=g).bfloat16().cuda()
    gx = torch.full((R, I), 3.0, dtype=torch.bfloat16, device="cuda")
    runs = [slice(5, 8), slice(R - 101, R - 1)]
    for r in runs:
        n = r.stop - r.start
        x[r] = torch.randint(-1, 2, (n, I), generator=g).bfloat16().cuda()
        gy[r] = torch.randint(-1, 2, (n, N), generator=g).bfloat16().cuda()
    y = ep.expert_linear(x, w, cnt, expert_offsets=off)
    _, gw = ep.expert_linear_backward(gy, x, w, cnt, expert_offsets=off,
                                      grad_weight_dtype=torch.float32, out=(gx, None))
    for e, r in enumerate(runs):
        assert torch.equal(y[r], (x[r].float() @ w[e].float().t().contiguous()).bfloat16())
        assert torch.equal(gx[r], (gy[r].float() @ w[e].float()).bfloat16())
        assert torch.equal(gw[e], gy[r].float().t().contiguous() @ x[r].float())
    assert bool((gx[8:20] == 3.0).all()) and bool((gx[R - 130:R - 101] == 3.0).all())
    assert bool((gx[R - 1] == 3.0).all())
    del x, gx, gy, w
    E, N, I = 520, 2048, 2112                # 4.5 GB of bf16 weights
    w = torch.empty((E, N, I), dtype=torch.bfloat16, device="cuda")
    w[E - 1] = torch.randint(-1, 2, (N, I), generator=g).bfloat16().cuda()
    cnt, off = device([0] * (E - 1) + [70], [0] * E + [70])
    x = torch.randint(-1, 2, (70, I), generator=g).bfloat16().cuda()
    gy = torch.randint(-1, 2, (70, N), generator=g).bfloat16().cuda()
    y = ep.expert_linear(x, w, cnt, expert_offsets=off)
    assert torch.equal(y, (x.float() @ w[E - 1].float().t().contiguous()).bfloat16())
    gx, gw = ep.expert_linear_backward(gy, x, w, cnt, expert_offsets=off)
    assert torch.equal(gx, (gy.float() @ w[E - 1].float()).bfloat16())
    assert torch.equal(gw[E - 1], (gy.float().t().contiguous() @ x.float()).bfloat16())
    assert bool((gw[0] == 0).all()) and bool((gw[E - 2] == 0).all())


def test_gradient_against_differences():
    """expert_linear's gradients against differences of its own results: in
    steps of 1 of integer inputs the product is linear and exact."""
    counts, I, N = [5, 3], 16, 8
    g = gen(41)
    off, _, R = place(counts, "offsets")
    R = off[-1]
    x, w, gy = ints((R, I), g, 3), ints((2, N, I), g, 3), ints((R, N), g, 2)
    d_cnt, d_off = device(counts, off)
    y0 = None

    def loss(x, w):
        y = ep.expert_linear(x.bfloat16().cuda(), w.bfloat16().cuda(), d_cnt,
                             expert_offsets=d_off)
        return float((y.cpu().double() * gy).sum())

    y0 = loss(x, w)
    gx, gw = ep.expert_linear_backward(gy.bfloat16().cuda(), x.bfloat16().cuda(),
                                       w.bfloat16().cuda(), d_cnt, expert_offsets=d_off,
                                       grad_weight_dtype=torch.float32)
    for r, i in [(0, 0), (4, 15), (5, 3), (7, 8)]:
        up = x.clone()
        up[r, i] += 1
        assert loss(up, w) - y0 == float(gx[r, i])
    for e, n, i in [(0, 0, 0), (1, 7, 15), (0, 5, 2)]:
        up = w.clone()
        up[e, n, i] += 1
        assert loss(x, up) - y0 == float(gw[e, n, i])


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def layer_inputs(T, H, F, E, seed):
    g = gen(seed)
    bf = lambda *s: torch.randn(s, generator=g).bfloat16()
    return dict(x=bf(T, H), res=bf(T, H), nw=(1 + 0.1 * torch.randn(H, generator=g)),
                lg=torch.randn((T, E), generator=g),
                w1=(torch.randn((E, 2 * F, H), generator=g) / math.sqrt(H)).bfloat16(),
                w2=(torch.randn((E, H, F), generator=g) / math.sqrt(F)).bfloat16(),
                go=bf(T, H))


def training_step(s, E, K, shares=None):
    """norm -> route -> dispatch -> gate/up -> activation -> down -> combine, and
    all the way back.  Gradients: of x, the norm's weight, w1, w2, the logits."""
    T, H = s["x"].shape
    nm = ep.rms_norm(s["x"], s["nw"], residual=s["res"])
    idx, wt = ep.route(s["lg"], K, normalize=True)
    lay, d = ep.layout_dispatch(nm.y, idx, E, 1)
    rows = dict(expert_offsets=lay.expert_offsets)
    cnt = lay.num_tokens_per_expert
    a = ep.expert_linear(d.recv_x, s["w1"], cnt, **rows)
    h = ep.expert_swiglu(a, cnt, **rows)
    y = ep.expert_linear(h, s["w2"], cnt, **rows)
    out = ep.combine(y, d.dst_row, wt)
    gy, gwt = ep.combine_backward(s["go"], y, d.dst_row, wt)
    gh, gw2 = ep.expert_linear_backward(gy, h, s["w2"], cnt, grad_weight_dtype=torch.float32,
                                        **rows)
    ga = ep.expert_swiglu_backward(gh, a, cnt, **rows)
    gr, gw1 = ep.expert_linear_backward(ga, d.recv_x, s["w1"], cnt,
                                        grad_weight_dtype=torch.float32, **rows)
    gn = ep.dispatch_backward(gr, d.dst_row)
    gx, gnw = ep.rms_norm_backward(gn, nm.residual, s["nw"], nm.inv_rms, grad_residual=s["go"])
    gl = ep.route_backward(s["lg"], idx, gwt, normalize=True)
    return out, gx, gnw, gw1, gw2, gl, idx


def test_training_step_gradients():
    """The whole step against automatic differentiation in 64 bits with the same
    routing.  Roundings to bf16 on the way to each result: the normed rows, a, h
    and y forward, then the gradients of y, h, a, the rows and the token, and
    the result: at most ten, UBF each over the 2-norm (the maps between them
    pass an error's share on as they do the value's)."""
    T, H, F, E, K = 150, 256, 136, 8, 2
    s = layer_inputs(T, H, F, E, 90)
    s["lg"][7] = -math.inf
    d = {k: v.cuda() for k, v in s.items()}
    out, gx, gnw, gw1, gw2, gl, idx = training_step(d, E, K)
    torch.cuda.synchronize()
    idx = idx.cpu()

    hr = (s["x"].double() + s["res"].double()).bfloat16().double().requires_grad_(True)
    nw = s["nw"].double().requires_grad_(True)
    lg = torch.where(torch.isfinite(s["lg"]), s["lg"].double(), -1e4).requires_grad_(True)
    w1, w2 = (s[k].double().requires_grad_(True) for k in ("w1", "w2"))
    n = hr * (hr.square().mean(1, keepdim=True) + 1e-6).rsqrt() * nw
    ok = idx >= 0
    wt = torch.where(ok, torch.softmax(torch.where(ok, lg.gather(1, idx.clamp(min=0)), -1e4), 1),
                     0.0)
    res = torch.zeros((T, H), dtype=torch.float64)
    for k in range(K):
        e = idx[:, k].clamp(min=0)
        a = torch.einsum("th,tfh->tf", n, w1[e])
        y = torch.einsum("tf,thf->th", ref.silu(a[:, :F]) * a[:, F:], w2[e])
        res = res + wt[:, k, None] * y
    ((res + hr) * s["go"].double()).sum().backward()
    for got, want, name in [(out, res.detach(), "out"), (gx, hr.grad, "grad_x"),
                            (gnw, nw.grad, "norm weight"), (gw1, w1.grad, "w1"),
                            (gw2, w2.grad, "w2"), (gl, lg.grad, "logits")]:
        off = float((got.cpu().double() - want).norm() / want.norm())
        assert off <= 10 * UBF, (name, off)
    assert bool((out[7] == 0).all()) and torch.equal(gx[7].cpu(), s["go"][7])


def fp8_prefill(s, E, K, q1, qs1, q2, qs2):
    nm = ep.rms_norm(s["x"], s["nw"], residual=s["res"], fp8=True)
    idx, wt = ep.route(s["lg"], K, normalize=True)
    lay, d = ep.layout_dispatch_aligned(nm.y, idx, E, 1, 16, fp8=True)
    rows = dict(expert_offsets=lay.expert_offsets)
    cnt = lay.num_tokens_per_expert
    a = ep.expert_linear(d.recv_x, q1, cnt, x_scales=d.recv_scales, weight_scales=qs1, **rows)
    h, hs = ep.expert_swiglu(a, cnt, fp8=True, **rows)
    y = ep.expert_linear(h, q2, cnt, x_scales=hs, weight_scales=qs2, **rows)
    out = ep.combine(y, d.dst_row, wt)
    T = s["x"].shape[0]
    one = torch.full((1,), T, dtype=torch.int32, device=out.device)
    shared = ep.expert_linear(nm.codes, q1[:1], one, capacity=T, x_scales=nm.scales,
                              weight_scales=qs1[:1], swiglu=False)
    return out, shared, idx


def quantised(w):
    """E4M3 codes and scales per 128 x 128 block of w [E, W, I] (whole blocks)."""
    E, W, I = w.shape
    b = w.float().view(E, W // 128, 128, I // 128, 128)
    s = b.abs().amax((2, 4)).clamp(min=1e-4) / 448
    q = (b / s[:, :, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(E, W, I), s


def test_fp8_prefill():
    """norm -> FP8 dispatch -> FP8 products with an FP8 activation -> combine, and
    an expert shared by all tokens from the norm's own FP8 rows, against 64 bits
    with the quantised weights.  E4M3 rows are off by at most U8 of their values
    each (the input's and the activation's), over the 2-norm; bf16 roundings as
    above."""
    T, H, F, E, K = 200, 256, 128, 8, 2
    s = layer_inputs(T, H, F, E, 95)
    q1, qs1 = quantised(s["w1"])
    q2, qs2 = quantised(s["w2"])
    d = {k: v.cuda() for k, v in s.items()}
    out, shared, idx = fp8_prefill(d, E, K, q1.cuda(), qs1.cuda(), q2.cuda(), qs2.cuda())
    torch.cuda.synchronize()
    idx = idx.cpu()
    v1 = ref.weight_values(q1, qs1, 2 * F)
    v2 = ref.weight_values(q2, qs2, H)
    h = (s["x"].double() + s["res"].double()).bfloat16()
    n, _, _, _ = ref.norm(h, s["nw"], 1e-6)
    wt = torch.softmax(s["lg"].double().gather(1, idx), 1)
    res = torch.zeros((T, H), dtype=torch.float64)
    for k in range(K):
        a = torch.einsum("th,tfh->tf", n, v1[idx[:, k]])
        res += wt[:, k, None] * torch.einsum("tf,thf->th", ref.gate(a, F)[0], v2[idx[:, k]])
    for got, want in ((out, res), (shared, n @ v1[0].t())):
        off = float((got.cpu().double() - want).norm() / want.norm())
        assert off <= 2 * ref.U8 + 6 * UBF, off


def test_captured_steps_replayed_beside_eager_calls():
    """Two training steps captured into graphs of their own and replayed in turn
    with eager calls between, on another stream too: every replay gives the
    eager result."""
    T, H, F, E, K = 96, 128, 64, 8, 2
    sets = [{k: v.cuda() for k, v in layer_inputs(T, H, F, E, 100 + i).items()} for i in range(2)]
    eager = [[t.clone() for t in training_step(s, E, K)] for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = training_step(sets[0], E, K)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(on_side, eager[0]):
        assert torch.equal(a, b)
    graphs = []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = training_step(s, E, K)
        graphs.append((graph, res))
    for rep in range(4):
        for i in (rep % 2, 1 - rep % 2):
            for t in graphs[i][1]:
                t.zero_()
            graphs[i][0].replay()
            other = training_step(sets[1 - i], E, K)
            torch.cuda.synchronize()
            for a, b in zip(graphs[i][1], eager[i]):
                assert torch.equal(a, b), (rep, i)
            for a, b in zip(other, eager[1 - i]):
                assert torch.equal(a, b), (rep, i)
