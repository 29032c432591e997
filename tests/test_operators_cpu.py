"""The router, the gradients of dispatch and combine, and the experts' 4-bit
products without a GPU: every refusal of their C entry points and of the
binding, and the references that the GPU tests compare with.

No call here reaches a kernel.  Pointers are placeholders that the host checks
look at and never follow (real buffers where a GPU is present).
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import operator_refs as ref
from combine_ep_get_dispatch_amd import binding as b
from combine_ep_get_dispatch_amd import workloads as wl
from test_abi_cpu import Bufs, INVALID, UNSUPPORTED, _NoLaunch

BAD16 = ctypes.c_void_p(0x100008)


@pytest.fixture
def buf():
    return Bufs()


def test_combine_backward_rejects_bad_arguments(buf):
    L = b.lib()
    go, y, dst, w, gy, gw = (buf() for _ in range(6))

    def call(go=go, y=y, rows=8, dst=dst, w=w, T=4, K=2, H=256, gy=gy, gw=gw):
        return L.ep_combine_backward(go, y, rows, dst, w, T, K, H, gy, gw, None)

    for kw in [dict(go=None), dict(y=None), dict(dst=None), dict(w=None), dict(gy=None, gw=None),
               dict(rows=-1), dict(T=-1), dict(K=0), dict(H=0), dict(H=12), dict(T=1 << 28, K=8),
               dict(go=BAD16), dict(y=BAD16), dict(gy=BAD16)]:
        assert call(**kw) == INVALID, kw
    assert call(K=65) == UNSUPPORTED


def test_dispatch_backward_rejects_bad_arguments(buf):
    L = b.lib()
    g, dst, gx = (buf() for _ in range(3))

    def call(g=g, rows=8, dst=dst, T=4, K=2, H=256, gx=gx):
        return L.ep_dispatch_backward(g, rows, dst, T, K, H, gx, None)

    for kw in [dict(g=None), dict(dst=None), dict(gx=None), dict(rows=-1), dict(T=-1), dict(K=0),
               dict(H=0), dict(H=20), dict(T=1 << 28, K=8), dict(g=BAD16), dict(gx=BAD16)]:
        assert call(**kw) == INVALID, kw
    assert call(K=65) == UNSUPPORTED


def test_route_rejects_bad_arguments(buf):
    L = b.lib()
    lg, bias, idx, w = (buf() for _ in range(4))

    def call(lg=lg, dt=2, bias=bias, T=4, E=16, K=2, sc=1, ng=4, tg=2, nm=1, scale=1.0, idx=idx,
             w=w):
        return L.ep_route(lg, dt, bias, T, E, K, sc, ng, tg, nm, scale, idx, w, None)

    for kw in [dict(lg=None), dict(idx=None), dict(w=None), dict(dt=1), dict(dt=3), dict(dt=-1),
               dict(T=-1), dict(E=0), dict(K=0), dict(K=17), dict(sc=2), dict(sc=-1), dict(ng=0),
               dict(ng=3), dict(tg=0), dict(tg=5), dict(K=9, tg=2), dict(ng=-4),
               dict(scale=math.inf), dict(scale=math.nan), dict(T=1 << 28, K=8),
               dict(lg=ctypes.c_void_p(0x100002)), dict(lg=ctypes.c_void_p(0x100001), dt=0)]:
        assert call(**kw) == INVALID, kw
    assert call(E=2048, ng=1, tg=1) == UNSUPPORTED
    assert call(E=128, K=65, ng=1, tg=1) == UNSUPPORTED
    assert call(E=130, ng=65, tg=65) == UNSUPPORTED
    assert b.MAX_ROUTE_GROUPS == 64


def test_route_backward_rejects_bad_arguments(buf):
    L = b.lib()
    lg, idx, gw, gl = (buf() for _ in range(4))

    def call(lg=lg, dt=2, idx=idx, gw=gw, T=4, E=16, K=2, sc=0, nm=0, scale=1.0, gl=gl):
        return L.ep_route_backward(lg, dt, idx, gw, T, E, K, sc, nm, scale, gl, None)

    for kw in [dict(lg=None), dict(idx=None), dict(gw=None), dict(gl=None), dict(dt=1),
               dict(T=-1), dict(E=0), dict(K=0), dict(K=17), dict(sc=2), dict(scale=-math.inf),
               dict(lg=ctypes.c_void_p(0x100002)), dict(gl=ctypes.c_void_p(0x100001), dt=0)]:
        assert call(**kw) == INVALID, kw
    assert call(E=2048) == UNSUPPORTED
    assert call(E=128, K=65) == UNSUPPORTED


def test_expert_linear_rejects_bad_arguments(buf):
    L = b.lib()
    x, xs, off, cnt, w, s, z, y = (buf() for _ in range(8))

    def call(x=x, xs=xs, dt=1, rows=64, off=None, cnt=cnt, C=16, E=4, I=256, N=64, G=128, w=w,
             s=s, z=None, act=0, y=y):
        return L.ep_expert_linear_w4(x, xs, dt, rows, off, cnt, C, E, I, N, G, w, s, z, act, y,
                                     None)

    for kw in [dict(x=None), dict(xs=None), dict(cnt=None), dict(w=None), dict(s=None),
               dict(y=None), dict(dt=2), dict(dt=-1), dict(rows=-1), dict(rows=1 << 31),
               dict(C=0), dict(C=17), dict(C=-1), dict(E=0), dict(I=0), dict(I=200),
               dict(I=160, G=32), dict(N=0), dict(N=12), dict(G=16), dict(G=0), dict(G=256),
               dict(x=BAD16), dict(w=BAD16), dict(y=BAD16), dict(s=ctypes.c_void_p(0x100004)),
               dict(z=ctypes.c_void_p(0x100002))]:
        assert call(**kw) == INVALID, kw
    assert call(E=2048, C=1, rows=4096) == UNSUPPORTED
    assert call(I=1 << 20, N=1 << 12) == UNSUPPORTED
    assert call(I=1 << 20, N=1 << 11, act=1) == UNSUPPORTED
    assert call(I=(1 << 24) + 128, N=8) == UNSUPPORTED


@pytest.fixture
def stand_in(monkeypatch):
    """CPU tensors stand in for GPU ones; a call into the library fails."""
    monkeypatch.setattr(b, "_is_gpu", lambda t: True)
    monkeypatch.setattr(b, "lib", lambda: _NoLaunch())


def test_binding_checks_the_gradients_tensors(stand_in):
    T, K, H, R = 4, 2, 16, 8
    bf = torch.bfloat16
    go, y = torch.zeros((T, H), dtype=bf), torch.zeros((R, H), dtype=bf)
    dst, w = torch.zeros((T, K), dtype=torch.int32), torch.zeros((T, K))
    gy, gw = torch.zeros((R, H), dtype=bf), torch.zeros((T, K))
    for args, kw in [((go[:2], y, dst, w), {}), ((go.float(), y, dst, w), {}),
                     ((go, y[:, :8], dst, w), {}), ((go, y, dst.long(), w), {}),
                     ((go, y, dst, w.double()), {}), ((go, y, dst, w[:2]), {}),
                     ((go, y, dst, w), dict(out=(gy[:4], gw))),
                     ((go, y, dst, w), dict(out=(gy, gw[:2]))),
                     ((go, y, dst, w), dict(out=(gy.t().contiguous().t(), gw))),
                     ((go, None, dst, None), {}), ((go, None, dst, w), {}),
                     ((go, None, dst, w), dict(out=(gy, gw))),
                     ((go, y, dst, None), dict(out=(gy, gw))),
                     ((go, y.to("meta"), dst, w), {})]:
        with pytest.raises((ValueError, TypeError)):
            b.combine_backward(*args, **kw)
    for args, kw in [((y, dst.long()), {}), ((y.float(), dst), {}), ((y[:, 0], dst), {}),
                     ((y, dst), dict(out=go[:2])), ((y.t(), dst), {})]:
        with pytest.raises((ValueError, TypeError)):
            b.dispatch_backward(*args, **kw)


def test_binding_checks_the_routers_tensors(stand_in):
    T, E, K = 4, 16, 2
    lg = torch.zeros((T, E))
    idx, w = torch.zeros((T, K), dtype=torch.int64), torch.zeros((T, K))
    for args, kw in [((lg.double(), K), {}), ((lg.half(), K), {}), ((lg[0], K), {}),
                     ((lg.t(), K), {}), ((lg[:, ::2], K), {}),
                     ((lg, K), dict(expert_bias=torch.zeros(E - 1))),
                     ((lg, K), dict(expert_bias=torch.zeros(E, dtype=torch.float64))),
                     ((lg, K), dict(score="relu")), ((lg, K), dict(out=(idx.int(), w))),
                     ((lg, K), dict(out=(idx, w[:, :1])))]:
        with pytest.raises((ValueError, TypeError, AssertionError)) as e:
            b.route(*args, **kw)
        assert not isinstance(e.value, AssertionError), (args, kw)
    for args, kw in [((lg, idx.int(), w), {}), ((lg, idx, w[:2]), {}), ((lg, idx[:, 0], w), {}),
                     ((lg, idx, w), dict(score="max")),
                     ((lg, idx, w), dict(out=lg.bfloat16())), ((lg, idx[:3], w[:3]), {})]:
        with pytest.raises((ValueError, TypeError)):
            b.route_backward(*args, **kw)


def test_binding_checks_the_experts_tensors(stand_in):
    E, C, I, N, G = 3, 4, 256, 16, 64
    x = torch.zeros((E * C, I), dtype=torch.bfloat16)
    q = torch.zeros((E * C, I), dtype=torch.uint8)
    xs = torch.zeros((E * C, I // 128))
    w = torch.zeros((E, N, I // 2), dtype=torch.uint8)
    s = torch.zeros((E, I // G, N), dtype=torch.bfloat16)
    z = torch.zeros((E, I // G, N), dtype=torch.uint8)
    cnt = torch.zeros(E, dtype=torch.int32)
    off = torch.zeros(E + 1, dtype=torch.int32)
    for args, kw in [((x.float(), w, s, cnt), dict(capacity=C)),
                     ((q, w, s, cnt), dict(capacity=C)),
                     ((q, w, s, cnt), dict(capacity=C, x_scales=xs[:, :1])),
                     ((x, w, s, cnt), dict(capacity=C, x_scales=xs)),
                     ((x, w[:, :, :64], s, cnt), dict(capacity=C)),
                     ((x, w, s[:, :3], cnt), dict(capacity=C)),
                     ((x, w, s.float(), cnt), dict(capacity=C)),
                     ((x, w, s, cnt.long()), dict(capacity=C)),
                     ((x, w, s, cnt[:2]), dict(capacity=C)),
                     ((x, w, s, cnt), dict(capacity=C, zeros=z.int())),
                     ((x, w, s, cnt), dict(capacity=C, expert_offsets=off)),
                     ((x, w, s, cnt), dict(expert_offsets=off[:E])),
                     ((x, w, s, cnt), dict(capacity=C, out=x)),
                     ((x, w[0], s, cnt), dict(capacity=C)),
                     ((x, w[:, :15].contiguous(), s[:, :, :15].contiguous(), cnt),
                      dict(capacity=C, swiglu=True))]:
        with pytest.raises((ValueError, TypeError)):
            b.expert_linear_w4(*args, **kw)


@pytest.mark.parametrize("name", ["tiny", "decode", "prefill"])
def test_router_reference_agrees_with_the_workloads_gating(name):
    """The seeded workloads draw their routing with a gating of their own
    (numpy); on the same logits the router's reference gives the same."""
    cfg = wl.CONFIGS[name]
    T = 48
    idx, w, _ = wl.route(cfg, T)
    lg = torch.from_numpy(wl._rng(100 + cfg["c"]).standard_normal((T, cfg["E"])))
    ri, rw = ref.route(lg, cfg["K"], score="softmax" if cfg["gating"] == "softmax" else "sigmoid",
                       num_groups=cfg.get("n_groups", 1), topk_groups=cfg.get("topk_groups", 1),
                       normalize=True)
    assert np.array_equal(ri.numpy(), idx)
    assert np.allclose(rw.numpy(), w, rtol=1e-6)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
def test_router_gradient_reference_against_differences(score, normalize):
    """The reference gradient against central differences of the reference
    router's weights, the selected experts held fixed."""
    g = torch.Generator().manual_seed(5)
    T, E, K, h = 3, 7, 3, 1e-5
    lg = torch.randn((T, E), generator=g, dtype=torch.float64)
    gw = torch.randn((T, K), generator=g, dtype=torch.float64)
    idx, _ = ref.route(lg, K, score=score, normalize=normalize, scale=1.5)

    def loss(l):
        v = ref.scores(l, score).gather(1, idx)
        if normalize:
            v = v / v.sum(1, keepdim=True)
        return float((v * 1.5 * gw).sum())

    grad, _ = ref.route_backward(lg, idx, gw, score, normalize, 1.5)
    for t in range(T):
        for e in range(E):
            up, dn = lg.clone(), lg.clone()
            up[t, e] += h
            dn[t, e] -= h
            assert abs((loss(up) - loss(dn)) / (2 * h) - float(grad[t, e])) < 1e-8


def test_e4m3_values_are_the_formats():
    v = ref.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.nan_to_num(v, nan=1e9), torch.nan_to_num(t, nan=1e9))


@pytest.fixture
def no_call(monkeypatch):
    """CPU tensors stand in for GPU ones; a call that passes the checks fails
    the test, on a machine with a GPU and a loaded library too."""
    def called(name, *args):
        raise AssertionError("the binding called %s before rejecting its arguments" % name)
    monkeypatch.setattr(b, "_is_gpu", lambda t: True)
    monkeypatch.setattr(b, "_launch", called)


def refused(why, fn, *args, **kw):
    with pytest.raises((ValueError, TypeError), match=why):
        fn(*args, **kw)


def test_binding_refuses_what_is_wrong_with_the_gradients_tensors(no_call):
    T, K, H, R = 4, 2, 16, 8
    bf = torch.bfloat16
    go, y = torch.zeros((T, H), dtype=bf), torch.zeros((R, H), dtype=bf)
    dst, w = torch.zeros((T, K), dtype=torch.int32), torch.zeros((T, K))
    gy, gw = torch.zeros((R, H), dtype=bf), torch.zeros((T, K))
    cb = b.combine_backward
    with pytest.raises(AssertionError, match="ep_combine_backward"):
        cb(go, y, dst, w, out=(gy, gw))                  # nothing wrong: it is called
    refused("grad_out must have shape", cb, go[:2], y, dst, w)
    refused("grad_out must be torch.bfloat16", cb, go.float(), y, dst, w)
    refused("y must have shape", cb, go, y[:, :8].contiguous(), dst, w)
    refused("y must be contiguous", cb, go, torch.zeros((R, 2 * H), dtype=bf)[:, ::2], dst, w)
    refused("y must be on", cb, go, y.to("meta"), dst, w)
    refused("dst_row must be torch.int32", cb, go, y, dst.long(), w)
    refused("dst_row must be on", cb, go, y, dst.to("meta"), w)
    refused("topk_weights must be torch.float32", cb, go, y, dst, w.double())
    refused("topk_weights must have shape", cb, go, y, dst, w[:2])
    refused("grad_y must have shape", cb, go, y, dst, w, out=(gy[:4], gw))
    refused("grad_y must be contiguous", cb, go, y, dst, w,
            out=(gy.t().contiguous().t(), gw))
    refused("grad_weights must have shape", cb, go, y, dst, w, out=(gy, gw[:2]))
    refused("needs y or topk_weights", cb, go, None, dst, None)
    refused("needs num_rows", cb, go, None, dst, w)
    refused("grad_weights needs y", cb, go, None, dst, w, out=(gy, gw))
    refused("grad_y needs topk_weights", cb, go, y, dst, None, out=(gy, gw))
    db = b.dispatch_backward
    with pytest.raises(AssertionError, match="ep_dispatch_backward"):
        db(y, dst, out=go)
    refused("dst_row must be torch.int32", db, y, dst.long())
    refused("grad_recv_x must be torch.bfloat16", db, y.float(), dst)
    refused("grad_recv_x must be .R, H.", db, y[:, 0], dst)
    refused("grad_recv_x must be contiguous", db, y.t(), dst)
    refused("out must have shape", db, y, dst, out=go[:2])
    refused("out must be on", db, y, dst, out=go.to("meta"))


def test_binding_refuses_what_is_wrong_with_the_routers_tensors(no_call):
    T, E, K = 4, 16, 2
    lg = torch.zeros((T, E))
    idx, w = torch.zeros((T, K), dtype=torch.int64), torch.zeros((T, K))
    with pytest.raises(AssertionError, match="ep_route"):
        b.route(lg, K, expert_bias=torch.zeros(E), out=(idx, w))
    for bad in (lg.double(), lg.half()):
        refused("logits must be float32 or bfloat16", b.route, bad, K)
        refused("logits must be float32 or bfloat16", b.route_backward, bad, idx, w)
    refused("logits must be .T, E.", b.route, lg[0], K)
    refused("logits must be contiguous", b.route, lg.t(), K)
    refused("logits must be contiguous", b.route, lg[:, ::2], K)
    refused("expert_bias must have shape", b.route, lg, K, expert_bias=torch.zeros(E - 1))
    refused("expert_bias must be torch.float32", b.route, lg, K, expert_bias=torch.zeros(E).double())
    refused("expert_bias must be on", b.route, lg, K, expert_bias=torch.zeros(E, device="meta"))
    refused("score must be one of", b.route, lg, K, score="relu")
    refused("topk_idx must be torch.int64", b.route, lg, K, out=(idx.int(), w))
    refused("topk_weights must have shape", b.route, lg, K, out=(idx, w[:, :1].contiguous()))
    with pytest.raises(AssertionError, match="ep_route_backward"):
        b.route_backward(lg, idx, w, out=torch.zeros_like(lg))
    refused("topk_idx must be torch.int64", b.route_backward, lg, idx.int(), w)
    refused("topk_idx must have shape", b.route_backward, lg, idx[:3], w[:3])
    refused("topk_idx must be .T, K.", b.route_backward, lg, idx[:, 0], w)
    refused("grad_weights must have shape", b.route_backward, lg, idx, w[:2])
    refused("grad_weights must be on", b.route_backward, lg, idx, w.to("meta"))
    refused("score must be one of", b.route_backward, lg, idx, w, score="max")
    refused("out must be torch.float32", b.route_backward, lg, idx, w, out=lg.bfloat16())


def test_binding_refuses_what_is_wrong_with_the_experts_tensors(no_call):
    E, C, I, N, G = 3, 4, 256, 16, 64
    x = torch.zeros((E * C, I), dtype=torch.bfloat16)
    q = torch.zeros((E * C, I), dtype=torch.uint8)
    xs = torch.zeros((E * C, I // 128))
    w = torch.zeros((E, N, I // 2), dtype=torch.uint8)
    s = torch.zeros((E, I // G, N), dtype=torch.bfloat16)
    z = torch.zeros((E, I // G, N), dtype=torch.uint8)
    cnt = torch.zeros(E, dtype=torch.int32)
    off = torch.zeros(E + 1, dtype=torch.int32)
    y = torch.zeros((E * C, N), dtype=torch.bfloat16)
    fn = b.expert_linear_w4
    for a, kw in (((x, w, s, cnt), dict(capacity=C, zeros=z)),
                  ((q, w, s, cnt), dict(expert_offsets=off, x_scales=xs))):
        with pytest.raises(AssertionError, match="ep_expert_linear_w4"):
            fn(*a, out=y, **kw)
    refused("x must be torch.bfloat16", fn, x.float(), w, s, cnt, capacity=C)
    refused("codes need x_scales", fn, q, w, s, cnt, capacity=C)
    refused("x_scales must have shape", fn, q, w, s, cnt, capacity=C, x_scales=xs[:, :1].contiguous())
    refused("x_scales must be torch.float32", fn, q, w, s, cnt, capacity=C, x_scales=xs.bfloat16())
    refused("x_scales belong to E4M3", fn, x, w, s, cnt, capacity=C, x_scales=xs)
    refused("weight must have shape", fn, x, w[:, :, :64].contiguous(), s, cnt, capacity=C)
    refused("weight must be contiguous", fn, x, w.transpose(1, 2).contiguous().transpose(1, 2), s, cnt,
            capacity=C)
    refused("weight .E, W, I/2.", fn, x, w[0], s, cnt, capacity=C)
    refused("weight must be on", fn, x, w.to("meta"), s, cnt, capacity=C)
    refused("I/G groups", fn, x, w, s[:, :3].contiguous(), cnt, capacity=C)
    refused("scales must be torch.bfloat16", fn, x, w, s.float(), cnt, capacity=C)
    refused("scales must have shape", fn, x, w, s[:2], cnt, capacity=C)
    refused("zeros must be torch.uint8", fn, x, w, s, cnt, capacity=C, zeros=z.int())
    refused("zeros must have shape", fn, x, w, s, cnt, capacity=C, zeros=z[:, :2].contiguous())
    refused("num_tokens_per_expert must be torch.int32", fn, x, w, s, cnt.long(), capacity=C)
    refused("num_tokens_per_expert must have shape", fn, x, w, s, cnt[:2], capacity=C)
    refused("expert_offsets or capacity", fn, x, w, s, cnt, capacity=C, expert_offsets=off)
    refused("expert_offsets must have shape", fn, x, w, s, cnt, expert_offsets=off[:E])
    refused("out must have shape", fn, x, w, s, cnt, capacity=C, out=x)
    refused("even number of weight channels", fn, x, w[:, :15].contiguous(), s[:, :, :15].contiguous(),
            cnt, capacity=C, swiglu=True)


def test_combine_and_gradients_reject_rows_past_the_largest(buf):
    L = b.lib()
    go, y, dst, w, gy, gw = (buf() for _ in range(6))
    for H in (2**31 - 504, 2**31 - 8):
        assert L.ep_combine_backward(go, y, 1, dst, w, 1, 1, H, gy, gw, None) == UNSUPPORTED
        assert L.ep_dispatch_backward(go, 1, dst, 1, 1, H, gy, None) == UNSUPPORTED
        assert L.ep_combine(y, 1, dst, w, 1, 1, H, gy, None) == UNSUPPORTED


def test_binding_refuses_sizes_that_32_bits_would_cut(no_call):
    """ctypes cuts an int argument to 32 bits without an error: 2^32 + 1 groups
    would be 1 group, 2^32 + 3 tokens 3 tokens."""
    big = (1 << 32) + 1
    why = "below 2.31"
    lg = torch.zeros((4, 16))
    refused(why, b.route, lg, 2, num_groups=big)
    refused(why, b.route, lg, 2, topk_groups=big)
    refused(why, b.route, lg[:0], big)
    row = lambda n, t: torch.empty((n, 1), dtype=t, device="meta")
    refused(why, b.route, row(big, torch.bfloat16), 1)
    refused(why, b.route_backward, row(big, torch.float32), row(big, torch.int64),
            row(big, torch.float32))
    bf = torch.bfloat16
    y = torch.empty((8, 16), dtype=bf, device="meta")
    refused(why, b.combine_backward, torch.empty((big, 16), dtype=bf, device="meta"), y,
            row(big, torch.int32), row(big, torch.float32))
    refused(why, b.dispatch_backward, y, row(big, torch.int32))
    x = torch.zeros((12, 64), dtype=bf)
    w = torch.zeros((3, 16, 32), dtype=torch.uint8)
    s = torch.zeros((3, 1, 16), dtype=bf)
    cnt = torch.zeros(3, dtype=torch.int32)
    for c in (big, 1 << 31):
        refused(why, b.expert_linear_w4, x, w, s, cnt, capacity=c)
