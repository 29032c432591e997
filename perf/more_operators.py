"""Cases of the layer's operators for prefill and training: the experts' products over
ragged runs of rows (bf16 and FP8) with their gradients, the gated activation between two
of them with its gradient, and the root-mean-square norm ahead of the layer with the
residual's addition, an FP8 output and its gradient.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits), or,
where ``own`` is set, through the framework's entry points.  ``exact`` computes the same
outputs from the definitions in 64 bits.

Notation: E experts, R receive rows, I input and W output channels of an expert's weight
(W = 2N with the activation: gate channels, then up channels), T tokens, H hidden size.
FP8 rows are E4M3 codes with one fp32 scale per 128 channels, as dispatch writes them; FP8
weights have one scale per block of 128 x 128 (of each half, with the activation).
"""
from __future__ import annotations

import math

import torch

own = False


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------

def listed():
    return [
        # One token in decode: its 8 experts among this GPU's 32, down projection in bf16;
        # the fewest rows an expert can have.
        dict(name="linear one token", op="linear", E=32, rows=8, I=2048, N=7168, fp8=False,
             act=False, form="capacity", skew=0.3),
        # A prefill chunk through this GPU's 32 experts: FP8 rows and weights, gate and up
        # projection with the activation behind them.
        dict(name="linear prefill fp8", op="linear", E=32, rows=16384, I=7168, N=2048, fp8=True,
             act=True, form="offsets", skew=1.5),
        # Training step of coarse experts (32768 tokens, top-2 of 8), bf16: the largest product.
        dict(name="linear train bf16", op="linear", E=8, rows=65521, I=4096, N=2048, fp8=False,
             act=False, form="offsets", skew=1.5),
        # The way back of that step: the rows' gradient.
        dict(name="linear grad rows", op="linear_backward", E=8, rows=65521, I=4096, N=2048,
             want="x", gw="bf16", form="offsets", skew=1.5),
        # ... and the weights' gradient, in fp32 for an optimizer that keeps it so.
        dict(name="linear grad weight", op="linear_backward", E=8, rows=65521, I=4096, N=2048,
             want="w", gw="fp32", form="offsets", skew=1.5),
        # Both gradients of many small experts: odd widths, uneven runs that start at aligned
        # rows, more weights than rows.
        dict(name="linear grads ragged", op="linear_backward", E=40, rows=6001, I=1032, N=1000,
             want="xw", gw="bf16", form="aligned", skew=0.3),
        # One decode batch ahead of the layer: residual added, rows in bf16 for the router and
        # in FP8 for an expert that all tokens share.
        dict(name="norm decode", op="norm", T=128, H=7168, residual=True, bf16=True, fp8=True),
        # A prefill batch.
        dict(name="norm prefill", op="norm", T=4099, H=7168, residual=True, bf16=True, fp8=True),
        # The way back of a training step through the norm.
        dict(name="norm grad", op="norm_backward", T=4096, H=7168, residual=True),
        # Coarse experts' width, odd token count, no residual.
        dict(name="norm grad odd", op="norm_backward", T=32767, H=4104, residual=False),
        # Between the products of an FP8 prefill: activation and quantisation in one pass.
        dict(name="gate prefill fp8", op="gate", E=32, rows=32768, N=2048, fp8=True,
             form="aligned", skew=0.3),
        # Its gradient in a training step of coarse experts.
        dict(name="gate grad", op="gate_backward", E=8, rows=65521, N=1024, form="offsets",
             skew=1.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "linear_backward", "norm",
                     "norm_backward", "gate", "gate_backward"])
    if op in ("norm", "norm_backward"):
        fp8 = op == "norm" and rng.random() < 0.5
        H = 128 * _log(rng, 1, 96) if fp8 else 8 * _log(rng, 8, 1536)
        T = min(_log(rng, 1, 65536), 130_000_000 // H)
        case = dict(op=op, T=T, H=H, residual=rng.random() < 0.6)
        if op == "norm":
            case.update(fp8=fp8, bf16=not fp8 or rng.random() < 0.5)
        return case
    E = _log(rng, 1, 64)
    form = rng.choice(["offsets", "aligned", "capacity"])
    skew = rng.choice([0.3, 1.5])
    if op in ("gate", "gate_backward"):
        fp8 = op == "gate" and rng.random() < 0.5
        N = 128 * _log(rng, 1, 32) if fp8 else 8 * _log(rng, 8, 512)
        case = dict(op=op, E=E, rows=min(_log(rng, 1, 65536), 60_000_000 // N), N=N, form=form,
                    skew=skew)
        if op == "gate":
            case["fp8"] = fp8
        return case
    fp8 = op == "linear" and rng.random() < 0.5
    act = op == "linear" and rng.random() < 0.4
    I = 128 * _log(rng, 1, 56) if fp8 else 8 * _log(rng, 8, 896)
    N = 8 * _log(rng, 8, 512)
    W = 2 * N if act else N
    E = max(1, min(E, 400_000_000 // (I * W)))
    rows = min(_log(rng, 1, 65536), 250_000_000_000 // (I * W))
    case = dict(op=op, E=E, rows=rows, I=I, N=N, form=form, skew=skew)
    if op == "linear":
        case.update(fp8=fp8, act=act)
    else:
        case.update(want=rng.choice(["x", "w", "xw"]), gw=rng.choice(["bf16", "fp32"]))
    return case


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _most(case):
    """No expert has more rows than this."""
    mean = case["rows"] / case["E"]
    return int(mean * (1.7 if case["skew"] < 1 else 1.3)) + 2


def _places(case, g):
    """Rows per expert, uneven as a router fills them, and where each expert's run starts:
    one after the other, at multiples of 16, or at multiples of a capacity."""
    E, rows, C = case["E"], case["rows"], _most(case)
    if rows < 4 * E:               # few rows: one each for as many experts
        cnt = torch.zeros(E, dtype=torch.int64, device="cuda")
        at = torch.rand(E, device="cuda", generator=g).argsort()
        cnt[at[torch.arange(rows, device="cuda") % E]] = 1
        for i in range(1, -(-rows // E)):
            cnt[at[: min(E, rows - i * E)]] += 1
    else:
        p = torch.rand(E, device="cuda", generator=g) + case["skew"]
        cnt = (p / p.sum() * rows).round().long()
    cnt = cnt.clamp(max=C)
    if case["form"] == "capacity":
        return cnt.to(torch.int32), None, C, E * C
    step = 16 if case["form"] == "aligned" else 1
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = ((cnt + step - 1) // step * step).cumsum(0).to(torch.int32)
    return cnt.to(torch.int32), off, 0, rows + E * step


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 6007 + 29)
    return g


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    dev, bf = "cuda", torch.bfloat16
    randn = lambda *n: torch.randn(n, device=dev, generator=g)
    if case["op"] in ("norm", "norm_backward"):
        T, H = case["T"], case["H"]
        s["x"] = (randn(T, H) * (0.5 + torch.rand((T, 1), device=dev, generator=g))).to(bf)
        s["weight"] = (1.0 + 0.2 * randn(H)).to(bf)
        if case["op"] == "norm":
            s["res"] = randn(T, H).to(bf) if case["residual"] else None
        else:
            s["inv_rms"] = (s["x"].double().square().mean(1) + 1e-6).rsqrt().float()
            s["grad_y"] = (randn(T, H) * 0.01).to(bf)
            s["grad_residual"] = (randn(T, H) * 0.01).to(bf) if case["residual"] else None
        return s
    s["counts"], s["offsets"], s["C"], R = _places(case, g)
    N = case["N"]
    if case["op"] in ("gate", "gate_backward"):
        s["gate_up"] = (randn(R, 2 * N) * 1.5).to(bf)
        if case["op"] == "gate_backward":
            s["grad_y"] = (randn(R, N) * 0.01).to(bf)
            s["out"] = torch.zeros((R, 2 * N), dtype=bf, device=dev)
        elif case["fp8"]:
            s["out"] = (torch.zeros((R, N), dtype=torch.uint8, device=dev),
                        torch.zeros((R, N // 128), device=dev))
        else:
            s["out"] = torch.zeros((R, N), dtype=bf, device=dev)
        return s
    E, I = case["E"], case["I"]
    if case["op"] == "linear_backward":
        s["x"] = randn(R, I).to(bf)
        s["grad_y"] = (randn(R, N) * 0.01).to(bf)
        s["weight"] = (randn(E, N, I) / math.sqrt(I)).to(bf)
        s["grad_x"] = torch.zeros((R, I), dtype=bf, device=dev)
        s["grad_weight"] = torch.zeros((E, N, I), device=dev,
                                       dtype=bf if case["gw"] == "bf16" else torch.float32)
        return s
    W = 2 * N if case["act"] else N
    s["y"] = torch.zeros((R, N), dtype=bf, device=dev)
    s["x_scales"] = s["weight_scales"] = None
    if not case["fp8"]:
        s["x"] = randn(R, I).to(bf)
        s["weight"] = (randn(E, W, I) / math.sqrt(I)).to(bf)
        return s
    x = randn(R, I // 128, 128)
    a = x.abs().amax(dim=2).clamp(min=1e-4)
    s["x_scales"] = a / 448.0
    s["x"] = ((x * (448.0 / a)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
              .view(R, I))
    # weights of either half, padded to whole blocks for their scales
    halves = 2 if case["act"] else 1
    NB = (N + 127) // 128
    w = torch.zeros((E * halves, NB * 128, I), device=dev)
    w[:, :N] = randn(E * halves, N, I)
    w = w.view(E * halves, NB, 128, I // 128, 128)
    a = w.abs().amax(dim=(2, 4)).clamp(min=1e-4)
    w *= (448.0 / a)[:, :, None, :, None]
    s["weight_scales"] = (a / (448.0 * math.sqrt(I))).view(E, halves * NB, I // 128)
    s["weight"] = (w.view(E * halves, NB * 128, I)[:, :N].to(torch.float8_e4m3fn)
                   .view(torch.uint8).reshape(E, W, I))
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"linear": _linear, "linear_backward": _linear_backward, "norm": _norm,
            "norm_backward": _norm_backward, "gate": _gate,
            "gate_backward": _gate_backward}[s["op"]](s)


def _run_own(s):
    from combine_ep_get_dispatch_amd import binding as ep
    op = s["op"]
    if op == "norm":
        o = ep.rms_norm(s["x"], s["weight"], residual=s["res"], bf16=s["bf16"], fp8=s["fp8"])
        codes = None if o.codes is None else o.codes.view(torch.float8_e4m3fn)
        return [v for v in (o.y, codes, o.scales, o.residual, o.inv_rms) if v is not None]
    if op == "norm_backward":
        return ep.rms_norm_backward(s["grad_y"], s["x"], s["weight"], s["inv_rms"],
                                    grad_residual=s["grad_residual"])
    rows = dict(expert_offsets=s["offsets"], capacity=s["C"])
    if op == "gate":
        o = ep.expert_swiglu(s["gate_up"], s["counts"], fp8=s["fp8"], out=s["out"], **rows)
        return (o[0].view(torch.float8_e4m3fn), o[1]) if s["fp8"] else o
    if op == "gate_backward":
        return ep.expert_swiglu_backward(s["grad_y"], s["gate_up"], s["counts"], out=s["out"],
                                         **rows)
    if op == "linear_backward":
        gx, gw = "x" in s["want"], "w" in s["want"]
        o = ep.expert_linear_backward(
            s["grad_y"], s["x"] if gw else None, s["weight"] if gx else None, s["counts"],
            out=(s["grad_x"] if gx else None, s["grad_weight"] if gw else None), **rows)
        return [v for v in o if v is not None]
    return ep.expert_linear(s["x"], s["weight"], s["counts"], x_scales=s["x_scales"],
                            weight_scales=s["weight_scales"], swiglu=s["act"], out=s["y"],
                            **rows)


def _rows_of(s):
    """[E, C] receive row of each place, C at least the most rows of an expert, and whether
    the place holds a row."""
    C = _most(s)
    j = torch.arange(C, device="cuda")
    begin = (s["offsets"][:-1].long() if s["offsets"] is not None
             else torch.arange(s["E"], device="cuda") * C)
    held = j[None, :] < s["counts"][:, None]
    return torch.where(held, begin[:, None] + j[None, :], 0), held


def _padded(t, rows, held):
    return torch.where(held[..., None], t[rows].float(), 0.0)


def _values(codes, scales, group):
    """fp32 values of E4M3 codes with a scale per ``group`` channels."""
    n = codes.shape[-1]
    v = codes.view(torch.float8_e4m3fn).float().view(*codes.shape[:-1], n // group, group)
    return (v * scales[..., None]).view(codes.shape)


def _to_e4m3(v):
    """(values in E4M3, scales) of v [rows, channels], a scale per 128 channels."""
    b = v.view(v.shape[0], -1, 128)
    a = b.abs().amax(dim=2).clamp(min=1e-4)
    return (b * (448.0 / a)[..., None]).to(torch.float8_e4m3fn).view(v.shape), a / 448.0


def _silu(v):
    return v / (1.0 + torch.exp(-v))


def _linear(s):
    rows, held = _rows_of(s)
    N = s["N"]
    x, w = s["x"], s["weight"]
    if s["fp8"]:
        x = _values(x, s["x_scales"], 128)
        halves = 2 if s["act"] else 1
        per = s["weight_scales"].view(s["E"] * halves, -1, s["I"] // 128)
        per = per.repeat_interleave(128, 1)[:, :N].reshape(s["E"], -1, s["I"] // 128)
        w = _values(w, per, 128)
    y = torch.bmm(_padded(x, rows, held), w.float().transpose(1, 2).contiguous())
    if s["act"]:
        y = _silu(y[..., :N]) * y[..., N:]
    s["y"][rows[held]] = y[held].to(torch.bfloat16)
    return s["y"]


def _linear_backward(s):
    rows, held = _rows_of(s)
    g = _padded(s["grad_y"], rows, held)
    outs = []
    if "x" in s["want"]:
        gx = torch.bmm(g, s["weight"].float())
        s["grad_x"][rows[held]] = gx[held].to(torch.bfloat16)
        outs.append(s["grad_x"])
    if "w" in s["want"]:
        gw = torch.bmm(g.transpose(1, 2).contiguous(), _padded(s["x"], rows, held))
        s["grad_weight"].copy_(gw)
        outs.append(s["grad_weight"])
    return outs


def _norm(s):
    h = s["x"].float()
    outs = []
    if s["res"] is not None:
        r = (h + s["res"].float()).to(torch.bfloat16)
        h = r.float()
    inv = 1.0 / torch.sqrt(h.square().mean(dim=1) + 1e-6)
    y = h * inv[:, None] * s["weight"].float()
    if s["bf16"]:
        outs.append(y.to(torch.bfloat16))
    if s["fp8"]:
        outs += _to_e4m3(y)
    if s["res"] is not None:
        outs.append(r)
    return outs + [inv]


def _norm_backward(s):
    x, g = s["x"].float(), s["grad_y"].float()
    n = x * s["inv_rms"][:, None]
    gn = g * s["weight"].float()
    gx = (gn - n * (gn * n).mean(dim=1, keepdim=True)) * s["inv_rms"][:, None]
    if s["grad_residual"] is not None:
        gx = gx + s["grad_residual"].float()
    # one sum over the tokens for each channel: in 64 bits, for many tokens
    return gx.to(torch.bfloat16), (g * n).double().sum(dim=0).float()


def _row_held(s, R):
    """Which of the R rows an expert holds."""
    rows, held = _rows_of(s)
    out = torch.zeros(R, dtype=torch.bool, device="cuda")
    out[rows[held]] = True
    return out[:, None]


def _gate(s):
    N = s["N"]
    a = s["gate_up"].float()
    y = _silu(a[:, :N]) * a[:, N:]
    held = _row_held(s, a.shape[0])
    if s["fp8"]:
        codes, scales = _to_e4m3(y)
        s["out"][0].copy_(torch.where(held, codes.view(torch.uint8), s["out"][0]))
        s["out"][1].copy_(torch.where(held, scales, s["out"][1]))
        return s["out"][0].view(torch.float8_e4m3fn), s["out"][1]
    s["out"].copy_(torch.where(held, y.to(torch.bfloat16), s["out"]))
    return s["out"]


def _gate_backward(s):
    N = s["N"]
    a, g = s["gate_up"].float(), s["grad_y"].float()
    u = a[:, N:]
    sg = 1.0 / (1.0 + torch.exp(-a[:, :N]))
    si = a[:, :N] * sg
    d = torch.cat((g * u * (sg + si * (1.0 - sg)), g * si), dim=1).to(torch.bfloat16)
    s["out"].copy_(torch.where(_row_held(s, a.shape[0]), d, s["out"]))
    return s["out"]


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op in ("norm", "norm_backward"):
        T, H = case["T"], case["H"]
        if op == "norm":
            per = (2 + (4 if case["residual"] else 0) + (2 if case["bf16"] else 0)
                   + (1 + 4 / 128 if case["fp8"] else 0))
            return {"bytes": T * H * per + 4 * T + 2 * H, "flops": T * H * 6}
        per = 6 + (2 if case["residual"] else 0)
        return {"bytes": T * H * per + 4 * T + 6 * H, "flops": T * H * 12}
    rows, N = case["rows"], case["N"]
    if op == "gate":
        return {"bytes": rows * N * (4 + (1 + 4 / 128 if case["fp8"] else 2)),
                "flops": rows * N * 6}
    if op == "gate_backward":
        return {"bytes": rows * N * 10, "flops": rows * N * 12}
    E, I = case["E"], case["I"]
    W = 2 * N if op == "linear" and case["act"] else N
    active = min(E, rows)
    if op == "linear":
        one = 1 + 4 / 128 if case["fp8"] else 2
        return {"bytes": (active * W * I * (1 if case["fp8"] else 2) + rows * I * one
                          + rows * N * 2), "flops": 2 * rows * I * W}
    b = f = 0
    if "x" in case["want"]:
        b += active * W * I * 2 + rows * I * 2
        f += 2 * rows * I * W
    if "w" in case["want"]:
        b += E * W * I * (2 if case["gw"] == "bf16" else 4) + rows * I * 2
        f += 2 * rows * I * W
    return {"bytes": b + rows * W * 2, "flops": f}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return _exact_norm(s)
    if op == "norm_backward":
        return _exact_norm_backward(s)
    runs = []
    for e, n in enumerate(s["counts"].tolist()):
        b = int(s["offsets"][e]) if s["offsets"] is not None else e * s["C"]
        runs.append(slice(b, b + n))
    if op == "gate":
        return _exact_gate(s, runs)
    if op == "gate_backward":
        x = s["gate_up"].double().requires_grad_(True)
        y = torch.nn.functional.silu(x[:, :s["N"]]) * x[:, s["N"]:]
        g = torch.zeros_like(y)
        for r in runs:
            g[r] = s["grad_y"][r].double()
        y.backward(g)
        return x.grad
    if case["rows"] * case["I"] * case["N"] > 2e12:
        return None
    if op == "linear_backward":
        outs = []
        if "x" in case["want"]:
            gx = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
            for e, r in enumerate(runs):
                gx[r] = s["grad_y"][r].double() @ s["weight"][e].double()
            outs.append(gx)
        if "w" in case["want"]:
            gw = torch.zeros(s["weight"].shape, dtype=torch.float64, device="cuda")
            for e, r in enumerate(runs):
                gw[e] = s["grad_y"][r].double().t().contiguous() @ s["x"][r].double()
            outs.append(gw)
        return outs
    N, I = case["N"], case["I"]
    out = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    for e, r in enumerate(runs):
        x, w = s["x"][r], s["weight"][e]
        if case["fp8"]:
            x = (x.view(torch.float8_e4m3fn).double()
                 * s["x_scales"][r].double().repeat_interleave(128, 1))
            w = w.view(torch.float8_e4m3fn).double()
            NB = (N + 127) // 128
            ch = torch.arange(w.shape[0], device="cuda")
            block = ch // N * NB + ch % N // 128
            w *= s["weight_scales"][e].double()[block].repeat_interleave(128, 1)
        y = x.double() @ w.double().t().contiguous()
        if case["act"]:
            y = torch.nn.functional.silu(y[:, :N]) * y[:, N:]
        out[r] = y
    return out


def _exact_e4m3(v):
    """The scaled values ahead of their rounding, and the scales."""
    b = v.view(v.shape[0], v.shape[1] // 128, 128)
    top = b.abs().max(dim=2).values.clamp(min=1e-4)
    return (b / top[..., None] * 448).reshape(v.shape), top / 448


def _exact_norm(s):
    h = s["x"].double()
    total = None
    if s["res"] is not None:
        total = h + s["res"].double()
        h = total.to(torch.bfloat16).double()
    inv = (h.pow(2).sum(1) / s["H"] + 1e-6).pow(-0.5)
    y = (h.t() * inv).t() * s["weight"].double()
    outs = [y] if s["bf16"] else []
    if s["fp8"]:
        outs += _exact_e4m3(y)
    return outs + ([] if total is None else [total]) + [inv]


def _exact_norm_backward(s):
    """By automatic differentiation in 64 bits, with the inverse norm as a function of x."""
    x = s["x"].double().requires_grad_(True)
    w = s["weight"].double().requires_grad_(True)
    y = x * (x.pow(2).mean(1, keepdim=True) + 1e-6).pow(-0.5) * w
    y.backward(s["grad_y"].double())
    gx = x.grad
    return gx if s["grad_residual"] is None else gx + s["grad_residual"].double(), w.grad


def _exact_gate(s, runs):
    N = s["N"]
    y = torch.zeros((s["gate_up"].shape[0], N), dtype=torch.float64, device="cuda")
    for r in runs:
        a = s["gate_up"][r].double()
        y[r] = torch.nn.functional.silu(a[:, :N]) * a[:, N:]
    if not s["fp8"]:
        return y
    codes, scales = torch.zeros_like(y), torch.zeros_like(y[:, ::128])
    for r in runs:
        codes[r], scales[r] = _exact_e4m3(y[r])
    return codes, scales
