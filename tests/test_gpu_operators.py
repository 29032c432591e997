"""The router and its gradient, the gradients of dispatch and combine, and the
experts' 4-bit products on the GPU, each against a plain 64-bit reference
(operator_refs.py holds the references and derives the bounds), then together
as a training step and a decode step use them.
"""
import math

import pytest
import torch

import operator_refs as ref
from combine_ep_get_dispatch_amd import binding as ep
from parity import announce

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


def within(got, want, tol, what=""):
    """got (any device) within tol of want, elementwise; NaN in want: not looked at."""
    got = got.detach().cpu().double()
    look = ~torch.isnan(want)
    off = (got - want).abs()
    bad = look & ~(off <= tol)
    assert not bool(bad.any()), "%s: %d of %d off, worst %.3g over its bound" % (
        what, int(bad.sum()), bad.numel(), float((off / tol)[bad].nan_to_num(math.inf).max()))


# ---------------------------------------------------------------------------
# router
# ---------------------------------------------------------------------------

ROUTE = [
    # T, E, K, dtype, score, groups, topk_groups, bias, normalize, scale
    (1, 1, 1, "fp32", "softmax", 1, 1, False, False, 1.0),
    (1, 256, 8, "fp32", "sigmoid", 8, 4, True, True, 2.5),
    (67, 256, 8, "bf16", "sigmoid", 8, 4, True, True, 2.5),
    (33, 256, 8, "fp32", "softmax", 8, 3, False, False, 1.0),
    (40, 160, 6, "bf16", "softmax", 8, 3, True, False, 16.0),
    (129, 8, 2, "fp32", "softmax", 1, 1, False, True, 1.0),
    (130, 7, 7, "bf16", "softmax", 1, 1, False, True, 1.0),
    (65, 64, 4, "fp32", "sigmoid", 1, 1, False, False, 1.0),
    (31, 63, 5, "bf16", "sigmoid", 1, 1, True, False, 1.0),
    (17, 100, 10, "fp32", "softmax", 1, 1, True, True, 1.0),
    (19, 128, 8, "bf16", "softmax", 1, 1, False, False, 1.0),
    (9, 257, 3, "fp32", "sigmoid", 1, 1, True, True, 1.0),
    (9, 512, 16, "bf16", "softmax", 64, 8, False, True, 1.0),
    (5, 1000, 64, "fp32", "softmax", 4, 2, True, False, 1.0),
    (6, 1024, 33, "bf16", "sigmoid", 1, 1, False, True, 1.0),
    (12, 64, 1, "fp32", "softmax", 64, 1, False, True, 1.0),
    (8, 24, 12, "fp32", "sigmoid", 3, 2, True, True, 1.0),
    (11, 256, 9, "bf16", "softmax", 64, 12, True, True, 1.0),
]


def route_logits(T, E, dtype, seed, special=True):
    """Logits with masked experts, padded tokens, exact ties and extreme values."""
    g = gen(seed)
    l = torch.randn((T, E), generator=g) * 1.5
    if special:
        l[torch.rand((T, E), generator=g) < 0.1] = -math.inf
        l[torch.rand((T, E), generator=g) < 0.02] = math.nan
        if T > 1:
            l[1] = -math.inf                               # a padded token
        if T > 2:
            l[2] = torch.randint(0, 3, (E,), generator=g).float()   # many ties
        if T > 3:
            l[3] = -math.inf
            l[3, E // 2] = 0.25                            # one expert left
        if T > 4:
            l[4, : max(1, E // 2)] = torch.finfo(torch.float32).min   # lowest value as a mask
        if T > 5:
            l[5] = 0.0
            l[5, ::2] = -0.0                               # equal zeros of both signs
        if T > 6:
            l[6, E - 1] = math.inf
        if T > 7:
            l[7] = torch.finfo(torch.float32).min
    return l.to(torch.bfloat16 if dtype == "bf16" else torch.float32)


@pytest.mark.parametrize("T,E,K,dtype,score,ng,tg,bias,norm,scale", ROUTE,
                         ids=["T%d_E%d_K%d_%s_%s_g%d" % c[:6] for c in ROUTE])
def test_route(T, E, K, dtype, score, ng, tg, bias, norm, scale):
    announce("route T=%d E=%d K=%d %s %s groups=%d" % (T, E, K, dtype, score, ng))
    l = route_logits(T, E, dtype, T * 31 + E)
    b = None
    if bias:
        b = torch.randn(E, generator=gen(E)) * 0.1
        if E > 3:
            b[1], b[3] = -math.inf, math.nan               # never available
    kw = dict(score=score, num_groups=ng, topk_groups=tg, normalize=norm, scale=scale)
    idx, w = ep.route(l.cuda(), K, expert_bias=None if b is None else b.cuda(), **kw)
    torch.cuda.synchronize()
    ri, rw = ref.route(l, K, bias=b, **kw)
    assert torch.equal(idx.cpu(), ri)
    within(w, rw, ref.route_weight_tol(rw, E), "weights")
    again = ep.route(l.cuda(), K, expert_bias=None if b is None else b.cuda(), **kw)
    assert torch.equal(again[0], idx) and torch.equal(again[1], w)


LARGE = [(2100, 5, 2, "bf16", "softmax", 1, 1, False), (2300, 40, 4, "fp32", "sigmoid", 5, 2, True),
         (2200, 100, 8, "bf16", "softmax", 1, 1, False), (2049, 256, 8, "fp32", "sigmoid", 8, 4, True),
         (2500, 160, 6, "bf16", "sigmoid", 8, 3, True), (2100, 400, 12, "fp32", "softmax", 4, 2, False),
         (2048, 256, 8, "bf16", "sigmoid", 64, 9, True), (2060, 256, 8, "fp32", "softmax", 64, 9, False)]


@pytest.mark.parametrize("T,E,K,dtype,score,ng,tg,bias", LARGE,
                         ids=["T%d_E%d_K%d_%s_%s_g%d" % c[:6] for c in LARGE])
def test_route_and_gradient_of_large_batches(T, E, K, dtype, score, ng, tg, bias):
    """Batches past where a token has a wave of its own: the same tokens in
    small calls give the same bits, and a sample of them the reference's."""
    announce("route T=%d E=%d K=%d %s %s groups=%d" % (T, E, K, dtype, score, ng))
    l = route_logits(T, E, dtype, T + E)
    b = torch.randn(E, generator=gen(E)) * 0.1 if bias else None
    kw = dict(score=score, num_groups=ng, topk_groups=tg, normalize=True, scale=1.5)
    db = None if b is None else b.cuda()
    idx, w = ep.route(l.cuda(), K, expert_bias=db, **kw)
    parts = [ep.route(p.cuda(), K, expert_bias=db, **kw) for p in l.split(1000)]
    assert torch.equal(idx, torch.cat([p[0] for p in parts]))
    some = torch.cat([torch.arange(12), torch.randint(0, T, (28,), generator=gen(1)),
                      torch.arange(T - 4, T)])
    ri, rw = ref.route(l[some], K, bias=b, **kw)
    assert torch.equal(idx.cpu()[some], ri)
    within(w.cpu()[some], rw, ref.route_weight_tol(rw, E), "weights")
    gw = torch.randn((T, K), generator=gen(E))
    for norm in (False, True):
        got = ep.route_backward(l.cuda(), idx, gw.cuda(), score=score, normalize=norm, scale=1.5)
        g, size = ref.route_backward(l, idx.cpu(), gw, score, norm, 1.5)
        within(got, g, ref.route_backward_tol(g, size, E, l.dtype), "grad_logits")


def test_route_at_unaligned_rows_and_in_given_outputs():
    """Logits that start at an odd element, and outputs that are part of a
    larger buffer whose other rows stay as they are."""
    T, E, K = 21, 256, 8
    flat = torch.randn(T * E + 1, generator=gen(3)).cuda()
    l = flat[1:].view(T, E)
    big_i = torch.full((T + 2, K), 77, dtype=torch.int64, device="cuda")
    big_w = torch.full((T + 2, K), 7.0, device="cuda")
    ep.route(l, K, score="sigmoid", out=(big_i[1:T + 1], big_w[1:T + 1]))
    torch.cuda.synchronize()
    ri, rw = ref.route(l.cpu(), K, score="sigmoid")
    assert torch.equal(big_i[1:T + 1].cpu(), ri)
    within(big_w[1:T + 1], rw, ref.route_weight_tol(rw, E))
    assert bool((big_i[[0, T + 1]] == 77).all()) and bool((big_w[[0, T + 1]] == 7.0).all())
    bf = flat.bfloat16()[1:].view(T, E)
    grad = torch.full((T * E + 3,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = grad[1:T * E + 1].view(T, E)
    i, _ = ep.route(bf, K)
    gw = torch.randn((T, K), generator=gen(4))
    ep.route_backward(bf, i, gw.cuda(), out=out)
    g, size = ref.route_backward(bf.cpu(), i.cpu(), gw, "softmax", False, 1.0)
    within(out, g, ref.route_backward_tol(g, size, E, torch.bfloat16))
    assert float(grad[0]) == 5.0 and bool((grad[-2:] == 5.0).all())


def test_route_of_no_tokens():
    idx, w = ep.route(torch.empty((0, 16), device="cuda"), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    g = ep.route_backward(torch.empty((0, 16), device="cuda"), idx, w)
    assert g.shape == (0, 16)


BACK = [(T, E, K, d, s, n) for T, E, K, d in
        [(1, 1, 1, "fp32"), (70, 8, 2, "bf16"), (33, 63, 5, "fp32"), (40, 128, 8, "bf16"),
         (35, 256, 8, "fp32"), (18, 160, 6, "bf16"), (9, 500, 20, "fp32"), (7, 1024, 64, "bf16")]
        for s in ("softmax", "sigmoid") for n in (False, True)]


@pytest.mark.parametrize("T,E,K,dtype,score,norm", BACK,
                         ids=["T%d_E%d_K%d_%s_%s_%d" % c for c in BACK])
def test_route_backward(T, E, K, dtype, score, norm):
    announce("route backward T=%d E=%d K=%d %s %s %d" % (T, E, K, dtype, score, norm))
    l = route_logits(T, E, dtype, T * 17 + E)
    idx, _ = ref.route(l, K, score=score)
    if T > 8 and K > 1:
        idx[8, 1] = idx[8, 0]                # the same expert twice
        idx[0, K - 1] = E + 5                # not an expert: skipped
    gw = torch.randn((T, K), generator=gen(E))
    got = ep.route_backward(l.cuda(), idx.cuda(), gw.cuda(), score=score, normalize=norm,
                            scale=2.5)
    torch.cuda.synchronize()
    g, size = ref.route_backward(l, idx, gw, score, norm, 2.5)
    assert got.dtype == l.dtype
    within(got, g, ref.route_backward_tol(g, size, E, l.dtype), "grad_logits")


@pytest.mark.parametrize("score,norm", [("softmax", False), ("softmax", True),
                                        ("sigmoid", False), ("sigmoid", True)])
def test_route_gradient_against_differences(score, norm):
    """The kernels' gradient against differences of the kernels' own weights:
    the loss is linear in the weights, so with a step h the difference is off
    by the weights' fp32 rounding over h and by third derivatives times h^2."""
    T, E, K, h = 6, 16, 3, 2.0 ** -7
    l = torch.randn((T, E), generator=gen(9))
    l = (l * 64).round() / 64                # steps of h stay exact in fp32
    gw = torch.randn((T, K), generator=gen(10))
    idx, _ = ep.route(l.cuda(), K, score=score, normalize=norm)
    grad = ep.route_backward(l.cuda(), idx, gw.cuda(), score=score, normalize=norm).cpu()
    ri = idx.cpu()
    for e in range(E):
        w = []
        for sign in (1, -1):
            s = l.clone()
            s[:, e] += sign * h
            # the weights of the experts selected at l, whatever is selected at s
            allidx, allw = ep.route(s.cuda(), E, score=score)
            full = torch.zeros((T, E)).scatter_(1, allidx.cpu(), allw.cpu()).double()
            v = full.gather(1, ri)
            w.append(v / v.sum(1, keepdim=True) if norm else v)
        diff = ((w[0] - w[1]) * gw.double()).sum(1) / (2 * h)
        # |third derivative| of the shares is below 1; fp32 weights below 1
        tol = gw.abs().sum(1).double() * (h * h / 6 * 2 + 40 * ref.U32 / h)
        assert bool(((diff - grad[:, e].double()).abs() <= tol).all()), (e, score, norm)


# ---------------------------------------------------------------------------
# gradients of combine and dispatch
# ---------------------------------------------------------------------------

BACKWARD = [
    # T, H, K, extra rows, masked share
    (1, 8, 1, 0, 0.0), (1, 7168, 8, 0, 0.0), (3, 136, 2, 5, 0.0), (50, 512, 8, 0, 0.1),
    (33, 520, 6, 7, 0.3), (20, 1032, 4, 0, 0.0), (7, 4096, 10, 3, 0.2), (11, 2048, 3, 0, 0.5),
    (4, 9000, 8, 0, 0.0), (2, 18440, 5, 0, 0.0), (5, 256, 64, 2, 0.2), (9, 1024, 1, 0, 1.0),
    (1100, 264, 8, 0, 0.05), (300, 64, 2, 0, 0.0),
]


def slots(T, K, extra, masked, seed):
    """dst_row: distinct rows in a shuffled order, some slots without a row or
    with one past the end; the first token has none where slots are masked."""
    g = gen(seed)
    R = T * K + extra
    dst = torch.randperm(R, generator=g)[:T * K].to(torch.int32).view(T, K)
    u = torch.rand((T, K), generator=g)
    dst[u < masked] = -1
    dst[u < masked / 3] = R + 3
    if masked:
        dst[0] = -1
    return dst, R


@pytest.mark.parametrize("T,H,K,extra,masked", BACKWARD,
                         ids=["T%d_H%d_K%d" % c[:3] for c in BACKWARD])
def test_combine_and_dispatch_backward(T, H, K, extra, masked):
    announce("backward T=%d H=%d K=%d" % (T, H, K))
    g = gen(T + H)
    dst, R = slots(T, K, extra, masked, H + K)
    go = torch.randn((T, H), generator=g).bfloat16()
    y = torch.randn((R, H), generator=g).bfloat16()
    w = torch.rand((T, K), generator=g)
    d_go, d_y, d_dst, d_w = go.cuda(), y.cuda(), dst.cuda(), w.cuda()
    keep = torch.full((R, H), 3.5, dtype=torch.bfloat16, device="cuda")
    gw_buf = torch.full((T, K), 9.0, device="cuda")
    gy, gw = ep.combine_backward(d_go, d_y, d_dst, d_w, out=(keep, gw_buf))
    torch.cuda.synchronize()
    rgy, rgw, size = ref.combine_backward(go, y, dst, w)
    named = torch.zeros(R, dtype=torch.bool)
    named[dst[(dst >= 0) & (dst < R)].long()] = True
    # fp32 product, then bf16
    within(gy.cpu()[named], rgy[named], (ref.UBF + 2 * ref.U32) * rgy[named].abs() + ref.TINY,
           "grad_y")
    assert bool((gy.cpu()[~named] == 3.5).all())
    # at most 64 roundings on any path of the sum for H <= 40000: 8 per chunk
    # and lane, the lanes, the waves
    within(gw, rgw, 64 * ref.U32 * size + ref.TINY, "grad_weights")
    assert bool((gw.cpu()[(dst < 0) | (dst >= R)] == 0).all())
    again = ep.combine_backward(d_go, d_y, d_dst, d_w, out=(keep.clone(), None))
    assert torch.equal(again[0], gy) and torch.equal(again[1], gw)
    # each half alone
    only_y, none = ep.combine_backward(d_go, None, d_dst, d_w, out=(torch.full_like(keep, 3.5),
                                                                    None))
    assert none is None and torch.equal(only_y, gy)
    none, only_w = ep.combine_backward(d_go, d_y, d_dst, None)
    assert none is None and torch.equal(only_w, gw)

    gx = ep.dispatch_backward(d_y, d_dst)
    torch.cuda.synchronize()
    rgx, size = ref.dispatch_backward(y, dst)
    within(gx, rgx, ref.UBF * rgx.abs() + K * 2 * ref.U32 * size + ref.TINY, "grad_x")


@pytest.mark.parametrize("T,H,K,masked", [(2048, 4104, 8, 0.1), (4099, 4096, 4, 0.0),
                                          (2900, 4608, 6, 0.02), (1100, 5000, 17, 0.05)])
def test_combine_backward_of_large_batches(T, H, K, masked):
    """Batches that run in tiles (ragged tail tiles and chunks among them),
    against the two halves alone, which run one workgroup per token: the rows
    bit for bit, the sums within the roundings of both orders."""
    announce("backward tiles T=%d H=%d K=%d" % (T, H, K))
    dst, R = slots(T, K, 3, masked, H + K)
    g = torch.Generator(device="cuda").manual_seed(T)
    go = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    y = torch.randn((R, H), device="cuda", generator=g).bfloat16()
    w = torch.rand((T, K), device="cuda", generator=g)
    d_dst = dst.cuda()
    both = ep.combine_backward(go, y, d_dst, w, out=(torch.full_like(y, 2.5), None))
    gy, _ = ep.combine_backward(go, None, d_dst, w, out=(torch.full_like(y, 2.5), None))
    _, gw = ep.combine_backward(go, y, d_dst, None)
    torch.cuda.synchronize()
    assert torch.equal(both[0], gy)
    ok = (d_dst >= 0) & (d_dst < R)
    for k in range(K):
        rows = y[d_dst[:, k].clamp(0, R - 1).long()].double() * go.double()
        want = torch.where(ok[:, k], rows.sum(1), 0.0)
        tol = 64 * ref.U32 * rows.abs().sum(1) + ref.TINY
        for got in (both[1][:, k], gw[:, k]):
            assert bool(((got.double() - want).abs() <= tol).all()), k
    again = ep.combine_backward(go, y, d_dst, w, out=(torch.full_like(y, 2.5), None))
    assert torch.equal(again[0], both[0]) and torch.equal(again[1], both[1])


def test_backward_without_rows_or_tokens():
    dst = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    go = torch.ones((3, 16), dtype=torch.bfloat16, device="cuda")
    none = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    gy, gw = ep.combine_backward(go, none, dst, torch.ones((3, 2), device="cuda"))
    assert gy.shape == (0, 16) and bool((gw == 0).all())
    assert bool((ep.dispatch_backward(none, dst) == 0).all())
    gy, gw = ep.combine_backward(go, None, dst, torch.ones((3, 2), device="cuda"), num_rows=0)
    assert gy.shape == (0, 16) and gw is None
    gy, gw = ep.combine_backward(go, none, dst, None)
    assert gy is None and bool((gw == 0).all())
    empty = dst[:0]
    gy, gw = ep.combine_backward(go[:0], go, empty, torch.ones((0, 2), device="cuda"))
    assert gw.shape == (0, 2) and ep.dispatch_backward(go, empty).shape == (0, 16)


def test_combine_gradient_against_differences():
    """The loss sum(out * c) is linear in each input: with inputs of few bits
    the forward is exact, so its differences are the gradient."""
    T, H, K = 5, 64, 3
    g = gen(21)
    small = lambda *s: torch.randint(-2, 3, s, generator=g).float()
    dst = torch.randperm(T * K, generator=g).to(torch.int32).view(T, K).cuda()
    y, w, c = small(T * K, H), small(T, K), small(T, H)

    def loss(y, w):
        out = ep.combine(y.bfloat16().cuda(), dst, w.cuda())
        return float((out.double().cpu() * c).sum())

    gy, gw = ep.combine_backward(c.bfloat16().cuda(), y.bfloat16().cuda(), dst, w.cuda())
    for r, h in [(0, 0), (7, 63), (14, 31), (3, 8)]:
        up, dn = y.clone(), y.clone()
        up[r, h] += 1
        dn[r, h] -= 1
        assert (loss(up, w) - loss(dn, w)) / 2 == float(gy[r, h])
    for t in range(T):
        for k in range(K):
            up, dn = w.clone(), w.clone()
            up[t, k] += 1
            dn[t, k] -= 1
            assert (loss(y, up) - loss(y, dn)) / 2 == float(gw[t, k])


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------

EXPERT = [
    # E, C, counts, I, N, G, fp8, zeros, swiglu, offsets
    (1, 1, [1], 32, 8, 32, False, False, False, False),
    (1, 4, [3], 128, 16, 128, True, False, False, False),
    (3, 8, [0, 8, 5], 256, 64, 64, False, True, False, False),
    (4, 17, [17, 0, 1, 16], 384, 72, 128, True, True, False, True),
    (2, 40, [33, 40], 160, 24, 32, False, False, True, False),
    (2, 70, [70, 65], 512, 136, 32, True, True, True, True),
    (5, 3, [9, 2, 0, 3, 1], 1440, 40, 32, False, True, False, False),   # counts past C
    (3, 20, [4, 0, 19], 192, 200, 64, False, True, True, True),
    (2, 130, [129, 7], 1024, 56, 64, True, False, True, False),
    (8, 2, [0] * 8, 128, 16, 128, False, False, False, False),
    (1, 300, [290], 896, 64, 128, False, False, False, True),
    (2, 16, [16, 11], 7168, 64, 128, True, False, True, False),
    (2, 16, [3, 11], 7168, 40, 64, False, True, False, False),
    # many experts, few and many rows among them
    (70, 20, [(7 * e) % 23 for e in range(70)], 128, 40, 64, False, True, False, False),
    (130, 36, [(11 * e) % 37 for e in range(130)], 256, 72, 128, True, False, True, True),
    (66, 18, [0] * 64 + [17, 2], 96, 16, 32, False, True, False, True),
    (400, 18, [(5 * e) % 19 if e > 250 else 0 for e in range(400)], 64, 16, 32, False, False, False,
     False),
    # more input channels than the scales of one round
    (2, 20, [20, 9], 8320, 24, 128, True, True, False, False),
    (2, 20, [4, 18], 4192, 72, 32, False, True, True, False),
    (1, 40, [40], 16576, 16, 64, False, False, False, True),
    (2, 3, [3, 2], 4224, 16, 32, True, True, False, False),
]


def expert_inputs(E, C, I, N, G, fp8, zeros, swiglu, seed):
    g = gen(seed)
    R = E * C
    W = 2 * N if swiglu else N
    x = torch.randn((R, I), generator=g)
    xs = None
    if fp8:
        a = x.view(R, I // 128, 128).abs().amax(2).clamp(min=1e-4)
        xs = a / 448.0
        x = (x.view(R, I // 128, 128) * (448.0 / a)[..., None]).to(torch.float8_e4m3fn)
        x = x.view(torch.uint8).view(R, I)
        x.view(-1)[: min(256, R * I)] = (torch.arange(min(256, R * I)) % 127).to(torch.uint8)
    else:
        x = x.bfloat16()
    w = torch.randint(0, 256, (E, W, I // 2), dtype=torch.uint8, generator=g)
    s = ((torch.rand((E, I // G, W), generator=g) + 0.5) * (0.3 / math.sqrt(I))).bfloat16()
    z = torch.randint(0, 16, (E, I // G, W), dtype=torch.uint8, generator=g) if zeros else None
    return x, xs, w, s, z


@pytest.mark.parametrize("E,C,counts,I,N,G,fp8,zeros,swiglu,offsets", EXPERT,
                         ids=["E%d_C%d_I%d_N%d_G%d_%s" % (c[0], c[1], c[3], c[4], c[5],
                                                          "fp8" if c[6] else "bf16")
                              for c in EXPERT])
def test_expert_linear_w4(E, C, counts, I, N, G, fp8, zeros, swiglu, offsets):
    announce("expert_linear_w4 E=%d C=%d I=%d N=%d G=%d fp8=%s swiglu=%s" % (E, C, I, N, G, fp8,
                                                                            swiglu))
    x, xs, w, s, z = expert_inputs(E, C, I, N, G, fp8, zeros, swiglu, I + N)
    R = E * C
    cnt = torch.tensor(counts, dtype=torch.int32)
    if offsets:
        off = torch.zeros(E + 1, dtype=torch.int32)
        off[1:] = cnt.cumsum(0).to(torch.int32)
        ranges = [(int(off[e]), counts[e]) for e in range(E)]
    else:
        off = None
        ranges = [(e * C, min(counts[e], C)) for e in range(E)]
    y = torch.full((R, N), 6.5, dtype=torch.bfloat16, device="cuda")
    cu = lambda t: None if t is None else t.cuda()
    got = ep.expert_linear_w4(cu(x), cu(w), cu(s), cu(cnt), expert_offsets=cu(off),
                              capacity=0 if offsets else C, x_scales=cu(xs), zeros=cu(z),
                              swiglu=swiglu, out=y)
    torch.cuda.synchronize()
    want, err = ref.expert_linear(x, xs, w, s, z, ranges, N, swiglu)
    within(got, want, err * (1 + ref.UBF) + ref.UBF * want.abs() + ref.TINY, "y")
    held = ~torch.isnan(want[:, 0])
    assert bool((got.cpu()[~held] == 6.5).all())
    if bool(held.any()):
        d = (got.cpu().double() - want)[held]
        # every element is rounded once: together at most half a step of the whole
        assert float(d.norm()) <= ref.UBF * float(want[held].norm())
    again = ep.expert_linear_w4(cu(x), cu(w), cu(s), cu(cnt), expert_offsets=cu(off),
                                capacity=0 if offsets else C, x_scales=cu(xs), zeros=cu(z),
                                swiglu=swiglu, out=torch.full_like(y, 6.5))
    assert torch.equal(again, got)


def test_expert_linear_ignores_rows_outside_the_buffer():
    """Offsets and counts that leave [0, num_rows) touch only rows inside it."""
    E, I, N, G, R = 4, 128, 16, 32, 10
    x, _, w, s, _ = expert_inputs(1, R, I, N, G, False, False, False, 5)
    w, s = w.repeat(E, 1, 1), s.repeat(E, 1, 1)
    off = torch.tensor([-3, 4, 8, 50, 50], dtype=torch.int32)
    cnt = torch.tensor([5, -2, 9, 4], dtype=torch.int32)
    y = torch.full((R, N), 6.5, dtype=torch.bfloat16, device="cuda")
    got = ep.expert_linear_w4(x.cuda(), w.cuda(), s.cuda(), cnt.cuda(), expert_offsets=off.cuda(),
                              out=y)
    torch.cuda.synchronize()
    want, err = ref.expert_linear(x, None, w, s, None, [(0, 2), (0, 0), (8, 2), (0, 0)], N, False)
    within(got, want, err * (1 + ref.UBF) + ref.UBF * want.abs() + ref.TINY, "y")
    assert bool((got.cpu()[torch.isnan(want[:, 0])] == 6.5).all())


@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33, 48, 64, 65])
def test_expert_linear_row_counts_share_their_rows_results(n):
    """A row's result does not depend on how many rows stand beside it by more
    than the sums' roundings, and not at all on what stands in the rows after
    the expert's last one."""
    C, I, N, G = 70, 512, 40, 128
    x, xs, w, s, _ = expert_inputs(1, C, I, N, G, True, False, False, 11)
    full = ep.expert_linear_w4(x.cuda(), w.cuda(), s.cuda(),
                               torch.tensor([C], dtype=torch.int32, device="cuda"), capacity=C,
                               x_scales=xs.cuda())
    x2, xs2 = x.clone(), xs.clone()
    x2[n:] = 0x7f                                     # NaN codes past the rows held
    xs2[n:] = math.nan
    part = ep.expert_linear_w4(x2.cuda(), w.cuda(), s.cuda(),
                               torch.tensor([n], dtype=torch.int32, device="cuda"), capacity=C,
                               x_scales=xs2.cuda(), out=torch.full_like(full, 6.5))
    want, err = ref.expert_linear(x, xs, w, s, None, [(0, n)], N, False)
    for got in (full, part):
        within(got, want, err * (1 + ref.UBF) + ref.UBF * want.abs() + ref.TINY, "y")
    assert bool((part.cpu()[n:] == 6.5).all())


def test_expert_linear_with_exact_numbers():
    """Integers small enough that every sum is exact in fp32 and the result in
    bf16: the kernel's output equals the definition's bit for bit."""
    E, C, I, N, G = 2, 5, 256, 32, 64
    g = gen(77)
    x = torch.zeros((E * C, I))
    for r in range(E * C):
        at = torch.randperm(I, generator=g)[:6]
        x[r, at] = torch.randint(-2, 3, (6,), generator=g).float()
    w = torch.randint(0, 256, (E, N, I // 2), dtype=torch.uint8, generator=g)
    s = torch.ones((E, I // G, N), dtype=torch.bfloat16)
    z = torch.randint(4, 12, (E, I // G, N), dtype=torch.uint8, generator=g)
    cnt = torch.tensor([C, C - 2], dtype=torch.int32)
    got = ep.expert_linear_w4(x.bfloat16().cuda(), w.cuda(), s.cuda(), cnt.cuda(), capacity=C,
                              zeros=z.cuda())
    want, _ = ref.expert_linear(x, None, w, s, z, [(0, C), (C, C - 2)], N, False)
    held = ~torch.isnan(want[:, 0])
    assert torch.equal(got.cpu().double()[held], want[held])


def test_expert_linear_of_the_largest_capacity():
    """A capacity of almost 2^31 rows, of which a few hold a token (the others
    need no memory: they are neither read nor written)."""
    I, N, G, n = 64, 16, 32, 5
    x, _, w, s, _ = expert_inputs(1, n, I, N, G, False, False, False, 9)
    x, w, s = x.cuda(), w.cuda(), s.cuda()
    cnt = torch.tensor([n], dtype=torch.int32, device="cuda")
    y = torch.zeros((n, N), dtype=torch.bfloat16, device="cuda")
    ep._launch("ep_expert_linear_w4", x, x.data_ptr(), None, ep.EP_DTYPE_BF16, 2**31 - 1, None,
               cnt.data_ptr(), 2**31 - 1, 1, I, N, G, w.data_ptr(), s.data_ptr(), None, 0,
               y.data_ptr())
    assert torch.equal(y, ep.expert_linear_w4(x, w, s, cnt, capacity=n))


def at_the_end(t):
    """t's copy in the last bytes of a device allocation of its own."""
    if t is None:
        return None
    whole = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    v = whole[whole.numel() - t.numel() * t.element_size():].view(t.dtype).view(t.shape)
    return v.copy_(t)


@pytest.mark.parametrize("I,G,fp8,zeros", [(32, 32, False, True), (64, 32, False, False),
                                           (64, 64, False, True), (96, 32, False, True),
                                           (192, 64, False, False), (128, 128, False, True),
                                           (128, 32, True, True), (256, 128, True, False)])
@pytest.mark.parametrize("n", [3, 20])
def test_expert_linear_with_operands_at_the_ends_of_their_memory(I, G, fp8, zeros, n):
    announce("expert_linear_w4 at the ends of memory: I=%d G=%d fp8=%s n=%d" % (I, G, fp8, n))
    E, N = 2, 24
    x, xs, w, s, z = expert_inputs(E, n, I, N, G, fp8, zeros, False, I + n)
    cnt = torch.tensor([n, n], dtype=torch.int32)
    y = at_the_end(torch.zeros((E * n, N), dtype=torch.bfloat16))
    got = ep.expert_linear_w4(at_the_end(x), at_the_end(w), at_the_end(s), at_the_end(cnt),
                              capacity=n, x_scales=at_the_end(xs), zeros=at_the_end(z), out=y)
    torch.cuda.synchronize()
    want, err = ref.expert_linear(x, xs, w, s, z, [(0, n), (n, n)], N, False)
    within(got, want, err * (1 + ref.UBF) + ref.UBF * want.abs() + ref.TINY, "y")


def test_expert_linear_of_no_rows():
    _, _, w, s, _ = expert_inputs(2, 1, 64, 8, 32, False, False, False, 1)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    y = ep.expert_linear_w4(x, w.cuda(), s.cuda(), off[:2].clone(), expert_offsets=off)
    assert y.shape == (0, 8)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_training_step_gradients():
    """router -> dispatch -> experts (a product each, torch) -> combine and all
    the way back, against automatic differentiation of the same layer in 64
    bits with the same routing.  The layer runs in bf16, so each gradient is
    compared over its 2-norm: the roundings met on the way are four of bf16
    (x or y, out's gradient, the rows' gradient, the result) at UBF each."""
    T, H, E, P, K = 96, 256, 16, 4, 4
    g = gen(50)
    x = (torch.randn((T, H), generator=g)).bfloat16()
    lg = torch.randn((T, E), generator=g)
    lg[5] = -math.inf                                       # a padded token
    We = (torch.randn((E, H, H), generator=g) / math.sqrt(H)).bfloat16()
    go = torch.randn((T, H), generator=g).bfloat16()
    kw = dict(score="softmax", normalize=True, scale=1.5)
    d_x, d_lg = x.cuda(), lg.cuda()
    idx, w = ep.route(d_lg, K, **kw)
    lay, d = ep.layout_dispatch(d_x, idx, E, P)
    off = lay.expert_offsets.cpu().tolist()
    n = off[-1]
    y = torch.zeros((T * K, H), dtype=torch.bfloat16, device="cuda")
    d_We = We.cuda().float()
    for e in range(E):
        a, b = off[e], off[e + 1]
        y[a:b] = (d.recv_x[a:b].float() @ d_We[e]).bfloat16()
    out = ep.combine(y, d.dst_row, w)
    gy, gw = ep.combine_backward(go.cuda(), y, d.dst_row, w)
    gr = torch.zeros_like(gy)
    for e in range(E):
        a, b = off[e], off[e + 1]
        gr[a:b] = (gy[a:b].float() @ d_We[e].t().contiguous()).bfloat16()
    gx = ep.dispatch_backward(gr, d.dst_row)
    gl = ep.route_backward(d_lg, idx, gw, **kw)
    torch.cuda.synchronize()
    assert n == (T - 1) * K

    rx = x.double().requires_grad_(True)
    rl = torch.where(torch.isfinite(lg), lg.double(), -1e4).requires_grad_(True)
    ri = idx.cpu()
    ok = ri >= 0
    lw = torch.where(ok, rl.gather(1, ri.clamp(min=0)), -1e4)
    rw = torch.where(ok, torch.softmax(lw, 1), 0.0) * 1.5
    ry = torch.bmm(rx[:, None, :].expand(T, K, H).reshape(T * K, 1, H),
                   We.double()[ri.clamp(min=0).view(-1)]).view(T, K, H)
    ro = (ry * rw[..., None]).sum(1)
    (ro * go.double()).sum().backward()
    for got, want, name in [(out, ro.detach(), "out"), (gx, rx.grad, "grad_x"),
                            (gl, rl.grad, "grad_logits")]:
        off_by = float((got.cpu().double() - want).norm() / want.norm())
        assert off_by <= 4 * ref.UBF, (name, off_by)
    assert bool((gx[5] == 0).all()) and bool((gl[5] == 0).all()) and bool((out[5] == 0).all())


def decode_step(x, lg, bias, E, K, C, w1, s1, w2, s2):
    idx, w = ep.route(lg, K, expert_bias=bias, score="sigmoid", num_groups=4, topk_groups=2,
                      normalize=True, scale=2.5)
    d = ep.low_latency_dispatch(x, idx, E, C, fp8=True)
    h = ep.expert_linear_w4(d.recv_x, w1, s1, d.num_tokens_per_expert, capacity=C,
                            x_scales=d.recv_scales, swiglu=True)
    y = ep.expert_linear_w4(h, w2, s2, d.num_tokens_per_expert, capacity=C)
    return ep.combine(y, d.dst_row, w), idx, d, h, y


def decode_inputs(T, H, F, E, seed):
    g = gen(seed)
    x = torch.randn((T, H), generator=g).bfloat16()
    lg = torch.randn((T, E), generator=g)
    bias = torch.randn(E, generator=g) * 0.05
    _, _, w1, s1, _ = expert_inputs(E, 1, H, F, 128, False, False, True, seed + 1)
    _, _, w2, s2, _ = expert_inputs(E, 1, F, H, 64, False, False, False, seed + 2)
    return [t.cuda() for t in (x, lg, bias, w1, s1, w2, s2)]


def test_decode_step():
    """router -> fixed-capacity FP8 dispatch -> gate/up -> down -> combine, each
    stage's output against the definition on the stage's own inputs."""
    T, H, F, E, K, C = 24, 512, 320, 16, 4, 24
    x, lg, bias, w1, s1, w2, s2 = decode_inputs(T, H, F, E, 60)
    out, idx, d, h, y = decode_step(x, lg, bias, E, K, C, w1, s1, w2, s2)
    torch.cuda.synchronize()
    ri, rw = ref.route(lg.cpu(), K, bias=bias.cpu(), score="sigmoid", num_groups=4, topk_groups=2,
                       normalize=True, scale=2.5)
    assert torch.equal(idx.cpu(), ri)
    cnt = d.num_tokens_per_expert.cpu().tolist()
    ranges = [(e * C, min(cnt[e], C)) for e in range(E)]
    wh, eh = ref.expert_linear(d.recv_x.cpu(), d.recv_scales.cpu(), w1.cpu(), s1.cpu(), None,
                               ranges, F, True)
    within(h, wh, eh * (1 + ref.UBF) + ref.UBF * wh.abs() + ref.TINY, "gate/up")
    wy, ey = ref.expert_linear(h.cpu(), None, w2.cpu(), s2.cpu(), None, ranges, H, False)
    within(y, wy, ey * (1 + ref.UBF) + ref.UBF * wy.abs() + ref.TINY, "down")
    rows = y.cpu().double()[d.dst_row.cpu().long().clamp(min=0)]
    want = (rows * rw[..., None]).sum(1)
    size = (rows.abs() * rw[..., None]).sum(1)
    within(out, want, ref.UBF * want.abs() + 64 * ref.U32 * size + ref.TINY, "out")


def test_two_captured_steps_replayed_beside_eager_calls():
    """Two decode steps and a backward captured into graphs of their own, then
    replayed in turn with eager calls between: every replay gives the eager
    result (the calls keep no state that two graphs could share)."""
    T, H, F, E, K, C = 12, 256, 128, 8, 2, 12
    sets = [decode_inputs(T, H, F, E, 70 + i) for i in range(2)]
    go = torch.randn((T, H), generator=gen(80)).bfloat16().cuda()

    def step(s):
        x, lg, bias, w1, s1, w2, s2 = s
        out, idx, d, h, y = decode_step(x, lg, bias, E, K, C, w1, s1, w2, s2)
        idx2, w = ep.route(lg, K, normalize=True)
        gy = torch.zeros((E * C, H), dtype=torch.bfloat16, device="cuda")
        gy, gw = ep.combine_backward(go, y, d.dst_row, w, out=(gy, None))
        gx = ep.dispatch_backward(gy, d.dst_row)
        gl = ep.route_backward(lg, idx2, gw, normalize=True)
        return out, gw, gx, gl

    eager = [[t.clone() for t in step(s)] for s in sets]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = step(sets[0])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(on_side, eager[0]):
        assert torch.equal(a, b)
    graphs = []
    for s in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = step(s)
        graphs.append((graph, res))
    for rep in range(4):
        for i in (rep % 2, 1 - rep % 2):
            for t in graphs[i][1]:
                t.zero_()
            graphs[i][0].replay()
            other = step(sets[1 - i])
            torch.cuda.synchronize()
            for a, b in zip(graphs[i][1], eager[i]):
                assert torch.equal(a, b), (rep, i)
            for a, b in zip(other, eager[1 - i]):
                assert torch.equal(a, b), (rep, i)
