"""The experts' products, the gated activation and the norm without a GPU: every
refusal of their C entry points and of the binding, and the references that the
GPU tests compare with.  No call here reaches a kernel.
"""
import ctypes
import math

import pytest
import torch

import layer_refs as ref
from combine_ep_get_dispatch_amd import binding as b
from test_abi_cpu import Bufs, INVALID, UNSUPPORTED, WORKSPACE

BAD16 = ctypes.c_void_p(0x100008)
BIG = (1 << 22) + 128


@pytest.fixture
def buf():
    return Bufs()


ROWS = [dict(cnt=None), dict(rows=-1), dict(rows=1 << 31), dict(C=0), dict(C=17), dict(C=-1),
        dict(E=0), dict(E=-1)]


def test_expert_linear_rejects_bad_arguments(buf):
    L = b.lib()
    x, xs, off, cnt, w, ws, y = (buf() for _ in range(7))

    def call(x=x, xs=xs, dt=1, rows=64, off=None, cnt=cnt, C=16, E=4, I=256, N=64, w=w, ws=ws,
             act=0, y=y):
        return L.ep_expert_linear(x, xs, dt, rows, off, cnt, C, E, I, N, w, ws, act, y, None)

    for kw in ROWS + [dict(x=None), dict(xs=None), dict(w=None), dict(ws=None), dict(y=None),
                      dict(dt=2), dict(dt=-1), dict(I=0), dict(I=200), dict(I=12, dt=0),
                      dict(I=-8, dt=0), dict(N=0), dict(N=12), dict(N=-8), dict(x=BAD16),
                      dict(w=BAD16), dict(y=BAD16)]:
        assert call(**kw) == INVALID, kw
    assert call(E=2048, C=1, rows=4096) == UNSUPPORTED
    assert call(I=BIG) == UNSUPPORTED and call(N=BIG) == UNSUPPORTED
    assert call(N=(1 << 21) + 8, act=1) == UNSUPPORTED


def test_expert_linear_backward_rejects_bad_arguments(buf):
    L = b.lib()
    gy, x, w, off, cnt, gx, gw = (buf() for _ in range(7))

    def call(gy=gy, x=x, w=w, rows=64, off=None, cnt=cnt, C=16, E=4, I=256, N=64, gx=gx, gw=gw,
             dt=0, add=0):
        return L.ep_expert_linear_backward(gy, x, w, rows, off, cnt, C, E, I, N, gx, gw, dt, add,
                                           None)

    for kw in ROWS + [dict(gy=None), dict(x=None), dict(w=None), dict(gx=None, gw=None),
                      dict(dt=1), dict(dt=3), dict(add=1), dict(I=0), dict(I=12), dict(N=0),
                      dict(N=20), dict(gy=BAD16), dict(x=BAD16), dict(w=BAD16), dict(gx=BAD16),
                      dict(gw=BAD16)]:
        assert call(**kw) == INVALID, kw
    assert call(E=2048, C=1, rows=4096) == UNSUPPORTED
    assert call(I=BIG) == UNSUPPORTED and call(N=BIG) == UNSUPPORTED


def test_expert_swiglu_rejects_bad_arguments(buf):
    L = b.lib()
    a, gy, off, cnt, y, s = (buf() for _ in range(6))

    def call(a=a, rows=64, off=None, cnt=cnt, C=16, E=4, N=128, dt=1, y=y, s=s):
        return L.ep_expert_swiglu(a, rows, off, cnt, C, E, N, dt, y, s, None)

    def back(gy=gy, a=a, rows=64, off=None, cnt=cnt, C=16, E=4, N=128, y=y):
        return L.ep_expert_swiglu_backward(gy, a, rows, off, cnt, C, E, N, y, None)

    rows = [kw for kw in ROWS if "cnt" not in kw]
    for kw in rows + [dict(a=None), dict(y=None), dict(s=None), dict(dt=2), dict(dt=-1), dict(N=0),
                      dict(N=136), dict(N=12, dt=0), dict(N=-8, dt=0), dict(a=BAD16),
                      dict(y=BAD16), dict(cnt=None, rows=-1)]:
        assert call(**kw) == INVALID, kw
    for kw in rows + [dict(gy=None), dict(a=None), dict(y=None), dict(N=0), dict(N=12),
                      dict(gy=BAD16), dict(a=BAD16), dict(y=BAD16), dict(cnt=None, rows=1 << 31)]:
        assert back(**kw) == INVALID, kw
    assert call(E=2048, C=1, rows=4096) == UNSUPPORTED and call(N=BIG) == UNSUPPORTED
    assert back(E=2048, C=1, rows=4096) == UNSUPPORTED and back(N=BIG) == UNSUPPORTED


def test_rms_norm_rejects_bad_arguments(buf):
    L = b.lib()
    x, res, w, y, c, s, ro, inv = (buf() for _ in range(8))

    def call(x=x, res=res, w=w, dt=2, T=2, H=256, eps=1e-6, y=y, c=c, s=s, ro=ro, inv=inv):
        return L.ep_rms_norm(x, res, w, dt, T, H, eps, y, c, s, ro, inv, None)

    for kw in [dict(x=None), dict(w=None), dict(dt=1), dict(dt=-1), dict(T=-1), dict(H=0),
               dict(H=-8), dict(H=12), dict(H=200), dict(eps=-1e-6), dict(eps=math.inf),
               dict(eps=math.nan), dict(y=None, c=None), dict(s=None), dict(ro=None),
               dict(res=None), dict(x=BAD16), dict(res=BAD16), dict(w=BAD16), dict(y=BAD16),
               dict(c=BAD16), dict(ro=BAD16)]:
        assert call(**kw) == INVALID, kw
    assert call(H=32768 + 128) == UNSUPPORTED


def test_rms_norm_backward_rejects_bad_arguments(buf):
    L = b.lib()
    gy, x, w, inv, gr, gx, gw, ws = (buf() for _ in range(8))
    need = L.ep_rms_norm_backward_workspace_bytes(2, 256)
    assert need >= 2 * 256 * 4 and L.ep_rms_norm_backward_workspace_bytes(0, 256) > 0
    for bad in [(-1, 256), (2, 0), (2, 12), (2, 32776)]:
        assert L.ep_rms_norm_backward_workspace_bytes(*bad) == 0

    def call(gy=gy, x=x, w=w, dt=0, inv=inv, gr=gr, T=2, H=256, gx=gx, gw=gw, ws=ws, n=need):
        return L.ep_rms_norm_backward(gy, x, w, dt, inv, gr, T, H, gx, gw, ws, n, None)

    for kw in [dict(gy=None), dict(x=None), dict(w=None), dict(inv=None), dict(gx=None),
               dict(gw=None), dict(ws=None), dict(dt=1), dict(T=-1), dict(H=0), dict(H=12),
               dict(gy=BAD16), dict(x=BAD16), dict(w=BAD16), dict(gr=BAD16), dict(gx=BAD16),
               dict(gw=BAD16), dict(ws=BAD16)]:
        assert call(**kw) == INVALID, kw
    assert call(n=need - 1) == WORKSPACE
    assert call(H=32776) == UNSUPPORTED


@pytest.fixture
def no_call(monkeypatch):
    """CPU tensors stand in for GPU ones; a call that passes the checks fails the
    test, on a machine with a GPU and a loaded library too."""
    def called(name, *args):
        raise AssertionError("the binding called %s" % name)
    monkeypatch.setattr(b, "_is_gpu", lambda t: True)
    monkeypatch.setattr(b, "_launch", called)


def refused(why, fn, *args, **kw):
    with pytest.raises((ValueError, TypeError), match=why):
        fn(*args, **kw)


def passes(name, fn, *args, **kw):
    with pytest.raises(AssertionError, match="called %s$" % name):
        fn(*args, **kw)


def test_binding_checks_the_products_tensors(no_call):
    E, C, I, N = 3, 4, 256, 136
    bf, u8 = torch.bfloat16, torch.uint8
    x, w = torch.zeros((E * C, I), dtype=bf), torch.zeros((E, N, I), dtype=bf)
    q, qw = torch.zeros((E * C, I), dtype=u8), torch.zeros((E, N, I), dtype=u8)
    xs, ws = torch.zeros((E * C, I // 128)), torch.zeros((E, 2, I // 128))
    cnt, off = torch.zeros(E, dtype=torch.int32), torch.zeros(E + 1, dtype=torch.int32)
    y = torch.zeros((E * C, N), dtype=bf)
    fn = b.expert_linear
    passes("ep_expert_linear", fn, x, w, cnt, capacity=C, out=y)
    passes("ep_expert_linear", fn, x, w, cnt, expert_offsets=off, swiglu=True)
    passes("ep_expert_linear", fn, q, qw, cnt, capacity=C, x_scales=xs, weight_scales=ws)
    passes("ep_expert_linear", fn, q, qw, cnt, capacity=C, x_scales=xs, weight_scales=ws,
           swiglu=True)                      # one block of scales a half
    refused("x must be torch.bfloat16", fn, x.float(), w, cnt, capacity=C)
    refused("x must be .R, I.", fn, x[0], w, cnt, capacity=C)
    refused("x must be contiguous", fn, torch.zeros((E * C, 2 * I), dtype=bf)[:, ::2], w, cnt,
            capacity=C)
    refused("weight must be torch.bfloat16", fn, x, qw, cnt, capacity=C)
    refused("weight must be torch.uint8", fn, q, w, cnt, capacity=C, x_scales=xs, weight_scales=ws)
    refused("weight must have shape", fn, x, w[:, :, :128].contiguous(), cnt, capacity=C)
    refused("weight must be on", fn, x, w.to("meta"), cnt, capacity=C)
    refused("weight must be contiguous", fn, x, w.transpose(1, 2).contiguous().transpose(1, 2),
            cnt, capacity=C)
    refused("codes need x_scales and weight_scales", fn, q, qw, cnt, capacity=C, x_scales=xs)
    refused("x_scales must have shape", fn, q, qw, cnt, capacity=C, x_scales=xs[:, :1].contiguous(),
            weight_scales=ws)
    refused("weight_scales must have shape", fn, q, qw, cnt, capacity=C, x_scales=xs,
            weight_scales=ws[:, :1].contiguous())
    refused("weight_scales must be torch.float32", fn, q, qw, cnt, capacity=C, x_scales=xs,
            weight_scales=ws.to(bf))
    refused("belong to E4M3", fn, x, w, cnt, capacity=C, weight_scales=ws)
    refused("num_tokens_per_expert must be torch.int32", fn, x, w, cnt.long(), capacity=C)
    refused("num_tokens_per_expert must have shape", fn, x, w, cnt[:2], capacity=C)
    refused("expert_offsets or capacity", fn, x, w, cnt, capacity=C, expert_offsets=off)
    refused("expert_offsets must have shape", fn, x, w, cnt, expert_offsets=off[:E])
    refused("out must have shape", fn, x, w, cnt, capacity=C, out=x)
    refused("even number of weight channels", fn, x, w[:, :15].contiguous(), cnt, capacity=C,
            swiglu=True)
    refused("below 2.31", fn, x, w, cnt, capacity=1 << 32)


def test_binding_checks_the_products_gradients_tensors(no_call):
    E, C, I, N = 3, 4, 64, 16
    bf = torch.bfloat16
    x, w = torch.zeros((E * C, I), dtype=bf), torch.zeros((E, N, I), dtype=bf)
    gy, gw = torch.zeros((E * C, N), dtype=bf), torch.zeros((E, N, I))
    cnt, off = torch.zeros(E, dtype=torch.int32), torch.zeros(E + 1, dtype=torch.int32)
    fn, name = b.expert_linear_backward, "ep_expert_linear_backward"
    passes(name, fn, gy, x, w, cnt, capacity=C)
    passes(name, fn, gy, None, w, cnt, expert_offsets=off)
    passes(name, fn, gy, x, None, cnt, capacity=C, grad_weight_dtype=torch.float32)
    passes(name, fn, gy, x, w, cnt, capacity=C, accumulate=True, out=(None, gw))
    refused("needs x or weight", fn, gy, None, None, cnt, capacity=C)
    refused("grad_y must be torch.bfloat16", fn, gy.float(), x, w, cnt, capacity=C)
    refused("grad_y must be .R, N.", fn, gy[0], x, w, cnt, capacity=C)
    refused("x must have shape", fn, gy, x[:4], w, cnt, capacity=C)
    refused("weight must have shape", fn, gy, x, w[:, :8].contiguous(), cnt, capacity=C)
    refused("weight must be torch.bfloat16", fn, gy, x, w.float(), cnt, capacity=C)
    refused("grad_x must have shape", fn, gy, x, w, cnt, capacity=C, out=(gy, None))
    refused("grad_x needs weight", fn, gy, x, None, cnt, capacity=C, out=(x, None))
    refused("grad_weight needs x", fn, gy, None, w, cnt, capacity=C, out=(None, gw))
    refused("grad_weight must have shape", fn, gy, x, w, cnt, capacity=C, out=(None, gw[:2]))
    refused("grad_weight must be float32 or bfloat16", fn, gy, x, w, cnt, capacity=C,
            grad_weight_dtype=torch.float64)
    refused("grad_weight must be float32 to accumulate", fn, gy, x, w, cnt, capacity=C,
            accumulate=True, out=(None, gw.to(bf)))
    refused("accumulate needs", fn, gy, x, w, cnt, capacity=C, accumulate=True)
    refused("num_tokens_per_expert must have shape", fn, gy, x, w, cnt[:2], capacity=C)
    refused("expert_offsets or capacity", fn, gy, x, w, cnt, capacity=C, expert_offsets=off)
    refused("below 2.31", fn, gy, x, w, cnt, capacity=1 << 32)


def test_binding_checks_the_activations_tensors(no_call):
    E, C, N = 3, 4, 128
    bf = torch.bfloat16
    a, gy = torch.zeros((E * C, 2 * N), dtype=bf), torch.zeros((E * C, N), dtype=bf)
    cnt, off = torch.zeros(E, dtype=torch.int32), torch.zeros(E + 1, dtype=torch.int32)
    codes, scales = torch.zeros((E * C, N), dtype=torch.uint8), torch.zeros((E * C, 1))
    fn = b.expert_swiglu
    passes("ep_expert_swiglu", fn, a)
    passes("ep_expert_swiglu", fn, a, cnt, capacity=C, out=gy)
    passes("ep_expert_swiglu", fn, a, cnt, expert_offsets=off, fp8=True, out=(codes, scales))
    refused("gate_up must be .R, 2N.", fn, a[:, :5])
    refused("gate_up must be torch.bfloat16", fn, a.float())
    refused("gate_up must be contiguous", fn, a.t().contiguous().t())
    refused("need num_tokens_per_expert", fn, a, capacity=C)
    refused("need num_tokens_per_expert", fn, a, expert_offsets=off)
    refused("expert_offsets or capacity", fn, a, cnt, capacity=C, expert_offsets=off)
    refused("expert_offsets must have shape", fn, a, cnt, expert_offsets=off[:2])
    refused("out must have shape", fn, a, out=a)
    refused("codes must have shape", fn, a, fp8=True, out=(codes[:3], scales))
    refused("scales must have shape", fn, a, fp8=True, out=(codes, scales[:3]))
    refused("below 2.31", fn, a, cnt, capacity=1 << 32)
    fn = b.expert_swiglu_backward
    passes("ep_expert_swiglu_backward", fn, gy, a, cnt, capacity=C)
    refused("grad_y must have shape", fn, a, a)
    refused("grad_y must be torch.bfloat16", fn, gy.float(), a)
    refused("gate_up must be .R, 2N.", fn, gy, a[0])
    refused("out must have shape", fn, gy, a, out=gy)


def test_binding_checks_the_norms_tensors(no_call):
    T, H = 4, 256
    bf = torch.bfloat16
    x, w, inv = torch.zeros((T, H), dtype=bf), torch.zeros(H), torch.zeros(T)
    fn = b.rms_norm
    passes("ep_rms_norm", fn, x, w)
    passes("ep_rms_norm", fn, x, w.to(bf), residual=x, fp8=True)
    refused("x must be .T, H.", fn, x[0], w)
    refused("x must be torch.bfloat16", fn, x.float(), w)
    refused("x must be contiguous", fn, x.t(), w[:T])
    refused("weight must be float32 or bfloat16", fn, x, w.half())
    refused("weight must have shape", fn, x, w[:8])
    refused("residual must have shape", fn, x, w, residual=x[:2])
    refused("residual must be torch.bfloat16", fn, x, w, residual=x.float())
    refused("needs bf16 or fp8", fn, x, w, bf16=False)
    refused("y must be a torch.Tensor", fn, x, w, out=b.RmsNormed(None, None, None, None, inv))
    refused("out.residual must be", fn, x, w, residual=x,
            out=b.RmsNormed(x, None, None, None, inv))
    refused("codes must be", fn, x, w, fp8=True, out=b.RmsNormed(x, x, None, None, inv))
    refused("inv_rms must have shape", fn, x, w, out=b.RmsNormed(x, None, None, None, inv[:2]))
    refused("below 2.31", fn, torch.empty(((1 << 32) + 1, 1), dtype=bf, device="meta"), w)
    fn = b.rms_norm_backward
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    passes("ep_rms_norm_backward", fn, x, x, w, inv, grad_residual=x, workspace=ws)
    refused("x must have shape", fn, x, x[:2], w, inv)
    refused("inv_rms must have shape", fn, x, x, w, inv[:2])
    refused("inv_rms must be torch.float32", fn, x, x, w, inv.to(bf))
    refused("weight must have shape", fn, x, x, w[:8], inv)
    refused("grad_residual must have shape", fn, x, x, w, inv, grad_residual=x[:1])
    refused("workspace must be torch.uint8", fn, x, x, w, inv, workspace=ws.float())
    refused("grad_x must have shape", fn, x, x, w, inv, workspace=ws, out=(x[:1], w))
    refused("grad_weight must be torch.float32", fn, x, x, w, inv, workspace=ws,
            out=(x, w.to(bf)))


def test_references_against_automatic_differentiation():
    g = torch.Generator().manual_seed(1)
    T, H, N = 5, 24, 8
    randn = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    x, w, gy = randn(T, H).requires_grad_(True), randn(H).requires_grad_(True), randn(T, H)
    y, _, inv, _ = ref.norm(x, w, 1e-6)
    y.backward(gy)
    gx, _, gw, _ = ref.norm_backward(gy, x.detach(), w.detach(), inv.detach(), None)
    assert torch.allclose(gx, x.grad) and torch.allclose(gw, w.grad)
    a, ga = randn(T, 2 * N).requires_grad_(True), randn(T, N)
    ref.gate(a, N)[0].backward(ga)
    assert torch.allclose(ref.gate_backward(ga, a.detach(), N)[0], a.grad)
