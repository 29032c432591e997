"""The router, its gradient, the gradients of combine and the experts' 4-bit
products where results are small differences of large numbers, where inputs are
large, and where the same numbers are summed by another variant of a kernel.
"""
import math
from decimal import Decimal, getcontext

import pytest
import torch

import operator_refs as ref
from combine_ep_get_dispatch_amd import binding as ep
from parity import announce

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ---------------------------------------------------------------------------
# the router's gradient of confident tokens
# ---------------------------------------------------------------------------

def decimal_route_backward(logits, topk_idx, gw, score, normalize, scale):
    """(gradient, size of what it is added up from) with 60 digits, from
    d_i = share_i (c_i - sum of the shares' c) [(1 - s_i) for sigmoid scores];
    size = share_i sum_j share_j |c_i - c_j|."""
    getcontext().prec = 60
    T, E = logits.shape
    K = topk_idx.shape[1]
    grad = torch.zeros((T, E), dtype=torch.float64)
    size = torch.zeros((T, E), dtype=torch.float64)
    for t in range(T):
        l = [Decimal(float(v)) for v in logits[t]]
        e = [int(i) for i in topk_idx[t]]
        c = [Decimal(float(gw[t, k])) * Decimal(float(scale)) for k in range(K)]
        sig = [1 / (1 + (-v).exp()) for v in l]
        if score == "softmax" and not normalize:
            u = [v.exp() for v in l]
            total = sum(u)
            ci = [sum((c[k] for k in range(K) if e[k] == i), Decimal(0)) for i in range(E)]
            for i in range(E):
                mean = sum(u[j] / total * ci[j] for j in set(e))
                grad[t, i] = float(u[i] / total * (ci[i] - mean))
                size[t, i] = float(u[i] / total * sum(u[j] / total * abs(ci[i] - ci[j])
                                                      for j in range(E)))
            continue
        u = [l[i].exp() if score == "softmax" else sig[i] for i in e]
        total = sum(u)
        for k in range(K):
            one = 1 - sig[e[k]] if score == "sigmoid" else Decimal(1)
            if normalize:
                mean = sum(u[j] / total * c[j] for j in range(K))
                grad[t, e[k]] += float(u[k] / total * (c[k] - mean) * one)
                size[t, e[k]] += float(u[k] / total * one * sum(u[j] / total * abs(c[k] - c[j])
                                                               for j in range(K)))
            else:
                grad[t, e[k]] += float(c[k] * u[k] * one)
                size[t, e[k]] += float(abs(c[k] * u[k] * one))
    return grad, size


@pytest.mark.parametrize("score,norm", [("softmax", False), ("softmax", True),
                                        ("sigmoid", False), ("sigmoid", True)])
@pytest.mark.parametrize("K", [1, 3])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("E,many", [(64, False), (256, False), (256, True)])
def test_gradient_of_confident_tokens(score, norm, K, dtype, E, many):
    """The top logit leads by 10 to 60: its expert's gradient is its share times
    what the others hold, down to 1e-26 of c, and right relative to itself.

    fp64 throughout: a share is off by exp's 2 units and the rounding of its
    argument, at most 2^-53 * 128, and by at most 1100 additions, so each term
    is off by less than 2^-42 of itself; taking the c relative to that of the
    largest share, at least 1/256, adds 2 + 2 * 256 roundings of 2^-53 of the
    size.  Together less than 2^-41 of the size.
    Then one rounding to fp32, and for bf16 one more."""
    announce("confident tokens E=%d K=%d %s %s %s many=%s" % (E, K, dtype, score, norm, many))
    leads = [10.0, 15.0, 18.0, 20.0, 25.0, 30.0, 60.0]
    T = len(leads)
    l = torch.randn((T, E), generator=gen(E + K)) * 1.5
    top = torch.randint(0, E, (T,), generator=gen(3))
    for t, lead in enumerate(leads):
        l[t, top[t]] = float(l[t].max()) + lead
    if score == "sigmoid":
        l -= 12.0                                 # shares that are far apart
    l = l.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    gw = torch.randn((T, K), generator=gen(K))
    idx = l.float().sort(dim=1, descending=True, stable=True).indices[:, :K].contiguous()
    # with a large batch a token has fewer lanes
    n = 2100 // T + 1 if many else 1
    got = ep.route_backward(l.repeat(n, 1).cuda(), idx.repeat(n, 1).cuda(), gw.repeat(n, 1).cuda(),
                            score=score, normalize=norm, scale=2.5)
    torch.cuda.synchronize()
    want, size = decimal_route_backward(l, idx, gw, score, norm, 2.5)
    tol = 2.0 ** -41 * size + ref.U32 * want.abs() * (1 + ref.UBF) + ref.TINY
    if dtype == "bf16":
        tol = tol + ref.UBF * want.abs()
    got = got.cpu().double().view(n, T, E)
    assert bool((got == got[0]).all())
    off = (got[0] - want).abs()
    assert bool((off <= tol).all()), "worst %.3g of the result" % float(
        (off / want.abs().clamp(min=1e-37)).max())


def test_gradient_of_repeated_and_tied_slots():
    """Slots that name one expert together, and equal c: the sums are exact zeros
    or the formula's, not what their roundings leave."""
    l = torch.tensor([[30.0, 1.0, 0.0, -1.0], [4.0, 4.0, 4.0, 4.0], [25.0, 2.0, 1.0, 0.0]])
    idx = torch.tensor([[0, 0, 1], [0, 1, 2], [0, 1, 0]])
    gw = torch.tensor([[0.3, -0.7, 0.2], [0.25, 0.25, 0.25], [1e-3, 1e-3, 1e-3]])
    for score, norm in (("softmax", False), ("softmax", True), ("sigmoid", True)):
        got = ep.route_backward(l.cuda(), idx.cuda(), gw.cuda(), score=score, normalize=norm).cpu()
        want, size = decimal_route_backward(l, idx, gw, score, norm, 1.0)
        tol = 2.0 ** -41 * size + 2 * ref.U32 * want.abs() + ref.TINY
        assert bool(((got.double() - want).abs() <= tol).all()), (score, norm)
        if norm:
            assert bool((got[1:] == 0).all()), (score, norm)


@pytest.mark.parametrize("T,E,K,dtype", [(2100, 5, 2, "fp32"), (4097, 40, 40, "fp32"),
                                         (2200, 100, 8, "bf16"), (3000, 160, 6, "bf16"),
                                         (2049, 256, 8, "fp32"), (2100, 400, 64, "fp32"),
                                         (2060, 512, 12, "bf16")])
def test_softmax_weights_are_the_same_bits_in_batches_of_any_size(T, E, K, dtype):
    """A token's softmax weights in a large batch (few lanes a token) and in
    small ones (a wave a token), without normalisation: the same bits, and within
    the roundings of the exponents' arguments (at most ln E half steps on average
    over the shares), expf's (4) and the result's (1): their sum adds none."""
    announce("softmax weights T=%d E=%d K=%d %s" % (T, E, K, dtype))
    l = torch.randn((T, E), generator=gen(T + E)) * 3
    l[::7, :: 3] = -math.inf
    l[11] = -math.inf
    l[12] += 30000.0
    l = l.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    idx, w = ep.route(l.cuda(), K, scale=2.5)
    parts = [ep.route(p.cuda(), K, scale=2.5) for p in l.split(701)]
    torch.cuda.synchronize()
    assert torch.equal(idx, torch.cat([p[0] for p in parts]))
    assert torch.equal(w, torch.cat([p[1] for p in parts]))
    s = ref.scores(l, "softmax")
    want = torch.where(idx.cpu() >= 0, s.gather(1, idx.cpu().clamp(min=0)), 0.0) * 2.5
    tol = (math.log(E) + 4 + 1 + 1) * ref.U32 * want + ref.TINY
    assert bool(((w.cpu().double() - want).abs() <= tol).all())


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------

def expert_inputs(R, I, N, G, fp8, zeros, swiglu, seed, mean=0.0):
    """One expert's rows, weights, scales and zero points."""
    g = gen(seed)
    W = 2 * N if swiglu else N
    x = torch.randn((R, I), generator=g) + mean
    xs = None
    if fp8:
        a = x.view(R, I // 128, 128).abs().amax(2)
        xs = a / 448.0
        x = (x.view(R, I // 128, 128) * (448.0 / a)[..., None]).to(torch.float8_e4m3fn)
        x = x.view(torch.uint8).view(R, I)
    else:
        x = x.bfloat16()
    w = torch.randint(0, 256, (1, W, I // 2), dtype=torch.uint8, generator=g)
    s = ((torch.rand((1, I // G, W), generator=g) + 0.5) * (0.3 / math.sqrt(I))).bfloat16()
    z = torch.randint(0, 16, (1, I // G, W), dtype=torch.uint8, generator=g) if zeros else None
    return x, xs, w, s, z


def expert(x, xs, w, s, z, n, swiglu=False, out=None):
    cu = lambda t: None if t is None else t.cuda()
    return ep.expert_linear_w4(cu(x), cu(w), cu(s), torch.tensor([n], dtype=torch.int32).cuda(),
                               capacity=x.shape[0], x_scales=cu(xs), zeros=cu(z), swiglu=swiglu,
                               out=out)


@pytest.mark.parametrize("fp8,G,zeros,swiglu", [
    (True, 128, False, True), (True, 128, True, False), (True, 64, True, False),
    (True, 32, False, False), (False, 128, False, False), (False, 128, True, True),
    (False, 64, False, False), (False, 32, True, False)])
@pytest.mark.parametrize("blocks", [1, 3, 4, 5, 7, 8, 9, 12, 13, 16, 56, 65, 77])
def test_a_rows_bits_do_not_depend_on_the_rows_beside_it(fp8, G, zeros, swiglu, blocks):
    """A row's result is the same bits however many rows stand beside it: of bf16
    rows always, of E4M3 rows among experts of up to 16 rows and among larger
    ones (whose blocks of input channels are added up in another order)."""
    announce("bits by rows: fp8=%s G=%d blocks=%d" % (fp8, G, blocks))
    R, N = 40, 40
    args = expert_inputs(R, blocks * 128, N, G, fp8, zeros, swiglu, blocks)
    full = expert(*args, R, swiglu).cpu()
    want, err = ref.expert_linear(*args[:5], [(0, R)], N, swiglu)
    off = (full.double() - want).abs()
    assert bool((off <= err * (1 + ref.UBF) + ref.UBF * want.abs() + ref.TINY).all())
    few = expert(*args, 16, swiglu).cpu()
    assert bool(((few[:16].double() - want[:16]).abs() <= (err * (1 + ref.UBF) + ref.UBF * want.abs()
                                                           + ref.TINY)[:16]).all())
    for n in (1, 7, 16, 17, 32, 33):
        part = expert(*args, n, swiglu).cpu()
        assert torch.equal(part[:n], (few if n <= 16 else full)[:n]), n
    if not fp8:
        assert torch.equal(few[:16], full[:16])


# ---------------------------------------------------------------------------
# combine's gradient
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("T,H,K", [(2050, 4104, 8), (2100, 8192, 8), (1100, 8200, 17), (2048, 9224, 8),
                                   (4100, 16896, 4), (520, 20000, 33), (600, 9224, 8)])
def test_weight_gradients_are_the_same_bits_with_and_without_row_gradients(T, H, K):
    """Large batches write both gradients in tiles, the weights' alone in a
    workgroup per token: the sums are added up in the same order."""
    announce("weight gradients T=%d H=%d K=%d" % (T, H, K))
    g = torch.Generator(device="cuda").manual_seed(T)
    go = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    R = 3000                                       # (every row once: T * K rows are much memory)
    y = torch.randn((R, H), device="cuda", generator=g).bfloat16()
    dst = torch.full((T * K,), -1, dtype=torch.int32)
    at = torch.randperm(T * K, generator=gen(K))[:R]
    dst[at] = torch.arange(R, dtype=torch.int32)
    dst = dst.view(T, K).cuda()
    w = torch.rand((T, K), device="cuda", generator=g)
    _, both = ep.combine_backward(go, y, dst, w)
    _, alone = ep.combine_backward(go, y, dst, None)
    torch.cuda.synchronize()
    assert torch.equal(both, alone)
    ok = dst >= 0
    t = ok.nonzero()[:, 0]
    terms = go[t].double() * y[dst[ok].long()].double()
    assert bool(((both[ok].double() - terms.sum(1)).abs()
                 <= 64 * ref.U32 * terms.abs().sum(1) + ref.TINY).all())
    assert bool((both[~ok] == 0).all())


# ---------------------------------------------------------------------------
# experts: large rows, rows with a common mean
# ---------------------------------------------------------------------------

def close(got, want, err, what):
    """Within the sums' bound and the result's one rounding; over the whole, a
    rounding error is uniform, at most 2^-8 / sqrt(3) of the power of two below
    the value, so 0.6 half steps of the 2-norm leave the sums 0.16 of them."""
    got = got.cpu().double()
    off = (got - want).abs()
    bad = ~(off <= err * (1 + ref.UBF) + ref.UBF * want.abs() + ref.TINY)
    assert not bool(bad.any()), "%s: %d of %d off" % (what, int(bad.sum()), bad.numel())
    scale = float(want.abs().max())
    if want.numel() >= 1000:
        assert float((off / scale).norm()) <= 0.6 * ref.UBF * float((want / scale).norm()), what


@pytest.mark.parametrize("G,zeros", [(32, False), (32, True), (64, True), (128, False), (128, True)])
@pytest.mark.parametrize("n", [5, 20])
def test_rows_of_one_sign_just_below_the_largest(G, zeros, n):
    """bf16 rows of up to 2^113, all of one sign: a group's sums come up to
    143 * 128 * 2^113 < 2^128 and stay finite."""
    announce("large rows G=%d n=%d" % (G, n))
    x, _, w, s, z = expert_inputs(20, 512, 64, G, False, zeros, False, G + n)
    x = ((x.float().abs() / 8).clamp(0.5, 0.998) * 2.0 ** 112).bfloat16() * 2
    x[1] = -x[1]
    x[2] = 255 * 2.0 ** 105                          # the largest bf16 number below 2^113
    s = (s.float() * 2.0 ** -20).bfloat16()
    got = expert(x, None, w, s, z, n)
    torch.cuda.synchronize()
    assert float(x.float().abs().max()) < 2.0 ** 113
    want, err = ref.expert_linear(x, None, w, s, z, [(0, n)], 64, False)
    off = (got.cpu().double() - want).abs()[:n]
    assert bool((off <= (err * (1 + ref.UBF) + ref.UBF * want.abs() + ref.TINY)[:n]).all())


@pytest.mark.parametrize("G", [32, 128])
def test_e4m3_rows_of_the_largest_scales(G):
    announce("large E4M3 rows G=%d" % G)
    n, I, N = 18, 512, 64
    x, xs, w, s, z = expert_inputs(n, I, N, G, True, True, False, G)
    x[0] = 0x7e                                      # 448 everywhere
    xs = torch.full_like(xs, 2.0 ** 103)
    s = (s.float() * 2.0 ** -20).bfloat16()
    want, err = ref.expert_linear(x, xs, w, s, z, [(0, n)], N, False)
    close(expert(x, xs, w, s, z, n), want, err, "y")


@pytest.mark.parametrize("fp8,G,zeros", [(False, 128, False), (False, 128, True), (False, 32, True),
                                         (True, 128, True), (True, 32, False)])
@pytest.mark.parametrize("mean", [1.0, -30.0, 1000.0])
@pytest.mark.parametrize("n", [10, 24])
def test_rows_with_a_common_mean(fp8, G, zeros, mean, n):
    """Rows far from zero: what the codes' offset adds and the zero points take
    off again is then much larger than the result."""
    announce("common mean %g fp8=%s G=%d n=%d" % (mean, fp8, G, n))
    x, xs, w, s, z = expert_inputs(n, 2048, 128, G, fp8, zeros, False, G + n, mean)
    want, err = ref.expert_linear(x, xs, w, s, z, [(0, n)], 128, False)
    close(expert(x, xs, w, s, z, n), want, err, "y")


def e4m3_bound(x, xs, s, zeros, G):
    """Bound on a row's E4M3 sums.  Of eight neighbouring channels the matrix
    instruction cuts what lies below 2^-13 of the largest product's exponents'
    power of two: with codes of up to 15 below 2^-10 of the largest |x|'s power,
    which a code's last place reaches where |x| is under 2^-7 of that; in the
    sum of x (by ones, times a zero point of up to 15) below 2^-13, reached
    under 2^-10.  Then the eights' sums are added in fp32, in at most G / 8 + 8
    steps a group at a full step of at most 30 |x| each, and the groups."""
    R, I = x.shape
    v = ref.e4m3_values()[x.long()].abs()
    eight = v.view(R, I // 8, 8)
    top = torch.exp2(torch.floor(torch.log2(eight.amax(2, keepdim=True).clamp(min=2.0 ** -6))))
    # E4M3's last place stops at 2^-9: exponents below -6 count as -6
    power = torch.exp2(torch.floor(torch.log2(eight.clamp(min=2.0 ** -6))))
    cut = ((eight > 0) & (power < top * 2.0 ** -7)) * top * 2.0 ** -10
    cut = cut + ((eight > 0) & (power < top * 2.0 ** -10)) * top * 2.0 ** -13 * 15
    each = cut.view(R, I) + (G / 8 + 8) * 2 * ref.U32 * 30 * v
    return (each * xs.double().repeat_interleave(128, 1)) @ \
        s[0].t().double().repeat_interleave(G, 1).t().abs()


@pytest.mark.parametrize("G,zeros", [(32, False), (32, True), (64, False), (128, False), (128, True)])
@pytest.mark.parametrize("n", [1, 13, 30])
@pytest.mark.parametrize("I", [128, 1024, 7168])
@pytest.mark.parametrize("spread", [0.0, 2.0])
def test_e4m3_sums_within_what_their_codes_leave(G, zeros, n, I, spread):
    """E4M3 rows against a bound made for them; spread: channels of sizes far
    apart, so that small codes stand beside large ones."""
    announce("E4M3 bound G=%d n=%d I=%d spread=%g" % (G, n, I, spread))
    N = 128
    x, xs, w, s, z = expert_inputs(n, I, N, G, True, zeros, False, I + n)
    if spread:
        size = torch.exp(torch.randn((n, I), generator=gen(n)) * spread).clamp(max=40.0)
        v = (ref.e4m3_values()[x.long()] * size / 40.0).float()
        x = v.to(torch.float8_e4m3fn).view(torch.uint8)
    want, _ = ref.expert_linear(x, xs, w, s, z, [(0, n)], N, False)
    size = ref.e4m3_values()[x.long()].abs() * xs.double().repeat_interleave(128, 1)
    groups = (I / G + 64) * ref.U32 * 15 * size @ s[0].t().double().repeat_interleave(G, 1).t()
    close(expert(x, xs, w, s, z, n), want, e4m3_bound(x, xs, s, z, G) + groups, "y")


# ---------------------------------------------------------------------------
# the binding's checks of GPU tensors
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("name", ["gradients", "routers", "experts"])
def test_binding_refuses_wrong_gpu_tensors(name, monkeypatch):
    """The refusals of test_operators_cpu.py with tensors on the GPU, which the
    checks' short way looks at first; nothing is launched."""
    import test_operators_cpu as cpu

    def called(name, *args):
        raise AssertionError("the binding called %s" % name)
    monkeypatch.setattr(ep, "_launch", called)
    monkeypatch.setattr(ep, "_is_gpu", lambda t: True)      # (of tensors elsewhere: "must be on")
    with torch.device("cuda"):
        getattr(cpu, "test_binding_refuses_what_is_wrong_with_the_%s_tensors" % name)(None)


# ---------------------------------------------------------------------------
# batches of more threads than one launch holds
# ---------------------------------------------------------------------------

def test_gradients_of_more_tokens_than_one_launch_holds():
    """2^26 and a few tokens of 8 channels: a wave for each of them would be more
    than the 2^32 threads of a launch."""
    T, H = (1 << 26) + 5, 8
    announce("gradients of %d tokens" % T)
    g = torch.Generator(device="cuda").manual_seed(1)
    go = torch.randint(-8, 9, (T, H), device="cuda", generator=g, dtype=torch.int8).bfloat16()
    y = torch.randint(-8, 9, (T, H), device="cuda", generator=g, dtype=torch.int8).bfloat16()
    w = torch.randint(-4, 5, (T, 1), device="cuda", generator=g, dtype=torch.int8).float()
    dst = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda").view(T, 1)
    gy, gw = ep.combine_backward(go, y, dst, w)
    for a in range(0, T, 1 << 24):                  # (small whole numbers: every sum is exact)
        b = min(a + (1 << 24), T)
        rows = y[T - b:T - a].flip(0).float()
        assert torch.equal(gw[a:b, 0], (rows * go[a:b].float()).sum(1)), a
        assert torch.equal(gy[T - b:T - a].flip(0).float(), go[a:b].float() * w[a:b]), a
    del gy, gw
    gx = ep.dispatch_backward(y, dst)
    assert torch.equal(gx, y.flip(0))
    del gx
    out = ep.combine(y, dst, w)
    assert torch.equal(out, (y.flip(0).float() * w).bfloat16())


def test_router_of_more_tokens_than_one_launch_holds():
    """2^29 and a few tokens of one expert, of 8 lanes each."""
    T = (1 << 29) + 5
    announce("router of %d tokens" % T)
    g = torch.Generator(device="cuda").manual_seed(2)
    l = torch.randn((T, 1), device="cuda", generator=g, dtype=torch.bfloat16)
    l[::1000003] = -math.inf
    idx, w = ep.route(l, 1, score="sigmoid")
    step = 1 << 26
    for a in range(0, T, step):
        p = l[a:a + step].double()
        assert torch.equal(idx[a:a + step], torch.where(p > -math.inf, 0, -1)), a
        want = torch.sigmoid(p)
        assert bool(((w[a:a + step].double() - want).abs() <= 2 * ref.U32 * want).all()), a
    gl = ep.route_backward(l, idx, w, score="sigmoid")
    for a in range(0, T, step):
        p = l[a:a + step].double()
        want = w[a:a + step].double() * torch.sigmoid(p) * torch.sigmoid(-p)
        want = torch.where(p > -math.inf, want, 0.0)
        off = (gl[a:a + step].double() - want).abs()
        assert bool((off <= (ref.UBF + 2 * ref.U32) * want.abs()).all()), a


def test_expert_counts_whose_blocks_pass_32_bits():
    """128 experts that each claim 2^31 - 1 rows: more tasks than any rows have.
    Nothing is read or written."""
    announce("expert counts past 32 bits")
    E, I, N, G = 128, 32, 8, 32
    x = torch.zeros((8, I), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((E, N, I // 2), dtype=torch.uint8, device="cuda")
    s = torch.zeros((E, 1, N), dtype=torch.bfloat16, device="cuda")
    cnt = torch.full((E,), 2**31 - 1, dtype=torch.int32, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    y = torch.full((8, N), 6.5, dtype=torch.bfloat16, device="cuda")
    ep._launch("ep_expert_linear_w4", x, x.data_ptr(), None, ep.EP_DTYPE_BF16, 2**31 - 1,
               off.data_ptr(), cnt.data_ptr(), 0, E, I, N, G, w.data_ptr(), s.data_ptr(), None, 0,
               y.data_ptr())
    torch.cuda.synchronize()
    assert bool((y == 6.5).all())


@pytest.mark.parametrize("T,H,K", [(30, 264, 3), (9, 9000, 12), (2050, 4104, 8), (1100, 8200, 17)])
def test_slots_without_a_row_get_0_whatever_their_tokens_gradient_holds(T, H, K):
    """Infinities and NaN in the gradients of padded tokens, and of tokens that
    have some of their slots: a slot without a row gets exactly 0."""
    announce("masked slots T=%d H=%d K=%d" % (T, H, K))
    g = torch.Generator(device="cuda").manual_seed(T)
    R = 500
    go = torch.randn((T, H), device="cuda", generator=g).bfloat16()
    y = torch.randn((R, H), device="cuda", generator=g).bfloat16()
    dst = torch.full((T * K,), -1, dtype=torch.int32)
    at = torch.randperm(T * K, generator=gen(K))
    n = min(R, T * K // 2)
    dst[at[:n]] = torch.arange(n, dtype=torch.int32)
    dst[at[n:n + 5]] = R + 7
    dst = dst.view(T, K)
    dst[::3] = -1
    dst = dst.cuda()
    go[::2, 5], go[::3], go[1, -1] = math.inf, math.nan, -math.inf
    w = torch.rand((T, K), device="cuda", generator=g)
    gy, both = ep.combine_backward(go, y, dst, w, out=(torch.full_like(y, 2.5), None))
    _, alone = ep.combine_backward(go, y, dst, None)
    ok = (dst >= 0) & (dst < R)
    assert bool((~ok).any()) and bool(ok.any())
    for gw in (both, alone):
        assert bool((gw[~ok] == 0).all())
    named = torch.zeros(R, dtype=torch.bool, device="cuda")
    named[dst[ok].long()] = True
    assert bool((gy[~named] == 2.5).all())
    t = ok.nonzero()[:, 0]
    assert torch.equal(torch.isnan(gy[dst[ok].long()].float()),
                       torch.isnan(go[t].float() * w[ok][:, None]))
