"""The operators around the FP8 GEMMs of a gated MLP block, as cases to time
and to compare.

Three operators (the norm, the gated feed-forward, the clipping of the
gradients), each in every direction that it has:

  norm_fwd   the residual's addition, the root-mean-square norm and the E4M3
             1x128 quantisation of its output (what the block's first
             projection reads)
  norm_bwd   its backward pass: the gradient of the residual stream and of
             the norm's weight
  ffn_fwd    the gated feed-forward: gate and up projections of E4M3
             operands, SiLU and the product, quantised 1x128 for the down
             projection; in training also the two projections in bf16
  ffn_bwd    the backward pass of the gate: the gradients of both
             projections, quantised per row for the data gradient and per
             column for the weight gradient, and the recomputed activation
             quantised per column for the down projection's weight gradient
  clip       the global norm of a list of gradients, and the gradients
             scaled to a largest norm

`run` computes a case in plain torch operations (own = False) or with the
framework's kernels (own = True), on the inputs that `prepare` made. Sizes are
the framework's own: hidden width 7168, MLP width 18432, expert width 2048.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
GROUP = 128
E4M3_MAX = 448.0
HIDDEN, MLP, EXPERT = 7168, 18432, 2048


# ---------------------------------------------------------------- cases ----

def listed():
    return [
        # one decoded token's residual stream, before the block
        {"name": "norm_fwd_1x7168", "op": "norm_fwd", "T": 1, "D": HIDDEN, "residual": True, "gamma": "bf16"},
        # a training batch of packed sequences, its length odd
        {"name": "norm_fwd_8191x7168", "op": "norm_fwd", "T": 8191, "D": HIDDEN, "residual": True, "gamma": "bf16"},
        # fine-tuning on one ragged sequence at a narrow width, a block's first norm (no residual)
        {"name": "norm_bwd_1031x2048", "op": "norm_bwd", "T": 1031, "D": EXPERT, "residual": False, "gamma": "f32"},
        # the training batch, with the gradient that arrives on the residual stream
        {"name": "norm_bwd_8192x7168", "op": "norm_bwd", "T": 8192, "D": HIDDEN, "residual": True, "gamma": "bf16"},
        # decoding one token through the dense MLP: the weights' stream
        {"name": "ffn_fwd_1x7168x18432", "op": "ffn_fwd", "M": 1, "K": HIDDEN, "I": MLP, "save": False},
        # a decoding batch through the shared expert: few weights, few rows
        {"name": "ffn_fwd_24x7168x2048", "op": "ffn_fwd", "M": 24, "K": HIDDEN, "I": EXPERT, "save": False},
        # a ragged prompt through the shared expert
        {"name": "ffn_fwd_333x7168x2048", "op": "ffn_fwd", "M": 333, "K": HIDDEN, "I": EXPERT, "save": False},
        # training, dense MLP: the projections are kept for the backward pass
        {"name": "ffn_fwd_4096x7168x18432", "op": "ffn_fwd", "M": 4096, "K": HIDDEN, "I": MLP, "save": True},
        # the shared expert in a small training batch
        {"name": "ffn_bwd_640x2048", "op": "ffn_bwd", "M": 640, "I": EXPERT},
        # the dense MLP's backward pass
        {"name": "ffn_bwd_4096x18432", "op": "ffn_bwd", "M": 4096, "I": MLP},
        # clipping a small adapter's gradients: many little bf16 and FP32 tensors of odd sizes
        {"name": "clip_120_small", "op": "clip", "n": 120, "total": 1500007, "types": "mixed", "scale": 1.0},
        # clipping the MLP layer's weight gradients (FP32, as the weight-gradient GEMM writes them)
        {"name": "clip_9_large", "op": "clip", "n": 9, "total": 400000013, "types": "f32", "scale": 1e-3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    w = max(lo, _log(rng, lo, hi) // GROUP * GROUP)
    return w + GROUP if w == 24 * GROUP else w


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "ffn_fwd", "ffn_bwd", "clip"])
    if op in ("norm_fwd", "norm_bwd"):
        D = _width(rng, 128, MLP)
        T = _log(rng, 1, min(16384, 8192 * HIDDEN // D))
        return {"op": op, "T": T, "D": D, "residual": rng.random() < 0.5, "gamma": rng.choice(["bf16", "f32"])}
    if op == "ffn_fwd":
        return {"op": op, "M": _log(rng, 1, 4096), "K": _width(rng, 256, HIDDEN), "I": _width(rng, 128, MLP),
                "save": rng.random() < 0.5}
    if op == "ffn_bwd":
        I = _width(rng, 128, MLP)
        return {"op": op, "M": GROUP * _log(rng, 1, min(128, 4096 * MLP // I // GROUP)), "I": I}
    n = _log(rng, 1, 300)
    return {"op": op, "n": n, "total": _log(rng, max(2000, 20 * n), 400000000),
            "types": rng.choice(["f32", "bf16", "mixed"]), "scale": rng.choice([1e-6, 1e-3, 1.0])}


def work(case):
    op = case["op"]
    if op in ("norm_fwd", "norm_bwd"):
        T, D, r = case["T"], case["D"], case["residual"]
        g = D * (2 if case["gamma"] == "bf16" else 4)
        if op == "norm_fwd":
            # x (and the residual) in, the sum out, codes, scales and rstd out
            return {"bytes": T * D * ((2 + 2 + 2 if r else 2) + 1) + T * (D // GROUP) * 4 + T * 4 + g, "flops": 8 * T * D}
        # dy, h (and the residual's gradient) in, dx out; rstd, gamma in; dgamma out
        return {"bytes": T * D * (2 + 2 + (2 if r else 0) + 2) + T * 4 + g + D * 4, "flops": 12 * T * D}
    if op == "ffn_fwd":
        M, K, I = case["M"], case["K"], case["I"]
        b = M * K + M * (K // GROUP) * 4 + 2 * I * K + (2 * I // GROUP) * (K // GROUP) * 4 + M * I + M * (I // GROUP) * 4
        if case["save"]:
            b += M * 2 * I * 2
        return {"bytes": b, "flops": 2 * M * K * 2 * I}
    if op == "ffn_bwd":
        M, I = case["M"], case["I"]
        # gate, up, dh in; the two gradients twice and the activation once out, with their scales
        return {"bytes": M * I * (4 + 2) + 5 * M * I + 5 * (M * I // GROUP) * 4, "flops": 30 * M * I}
    n_b = sum(k * s for k, s in zip(_sizes(case), _elt(case)))
    return {"bytes": 2 * n_b, "flops": 3 * sum(_sizes(case))}


def _sizes(case):
    """Element counts of the gradient tensors, one over its rank: a few large, many small, odd ones among them."""
    n, total = case["n"], case["total"]
    whole = sum(1.0 / (i + 1) for i in range(n))
    rest = [max(1, int(total / (i + 1) / whole)) for i in range(1, n)]
    return [max(1, total - sum(rest))] + rest


def _elt(case):
    return [{"f32": 4, "bf16": 2, "mixed": 4 if i % 3 else 2}[case["types"]] for i in range(case["n"])]


# --------------------------------------------------------------- inputs ----

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _quant_rows(y):
    """E4M3 codes and FP32 scales of y [rows, cols] in groups of 128 along a row."""
    v = y.reshape(y.shape[0], -1, GROUP)
    amax = v.abs().amax(-1)
    inv = E4M3_MAX / amax
    dead = (amax == 0) | torch.isinf(inv)
    inv = torch.where(dead, torch.ones_like(inv), inv)
    s = torch.where(dead, torch.ones_like(amax), amax / E4M3_MAX)
    q = (v * inv[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.reshape(y.shape), s.t()


def _quant_blocks(w):
    n, k = w.shape
    v = w.reshape(n // GROUP, GROUP, k // GROUP, GROUP)
    amax = v.abs().amax((1, 3))
    inv = E4M3_MAX / amax
    q = (v * inv[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.reshape(n, k), amax / E4M3_MAX


def _ld(n):
    return (max(n, 1) + 3) // 4 * 4


def _codes(*shape):
    return torch.empty(shape, dtype=torch.uint8, device=DEV)


def _f32(*shape):
    return torch.empty(shape, dtype=torch.float32, device=DEV)


def _bf16(*shape):
    return torch.empty(shape, dtype=torch.bfloat16, device=DEV)


def prepare(case, seed):
    op, g = case["op"], _gen(seed)
    s = {"case": case}
    if op in ("norm_fwd", "norm_bwd"):
        T, D = case["T"], case["D"]
        gamma = 1.0 + 0.2 * _randn(g, D)
        s["gamma"] = gamma.to(torch.bfloat16) if case["gamma"] == "bf16" else gamma
        # per-channel magnitudes are log-normal, as in the framework's dense workload
        chan = torch.exp(_randn(g, D))
        if op == "norm_fwd":
            s["x"] = (_randn(g, T, D) * chan).to(torch.bfloat16)
            s["residual"] = (_randn(g, T, D) * chan).to(torch.bfloat16) if case["residual"] else None
            s["buf"] = dict(q=_codes(T, D), scales=_f32(D // GROUP, _ld(T)), rstd=_f32(T))
            if case["residual"]:
                s["buf"]["h"] = _bf16(T, D)
        else:
            s["h"] = (_randn(g, T, D) * chan).to(torch.bfloat16)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
            s["dy"] = (_randn(g, T, D) * 1e-3).to(torch.bfloat16)
            s["dres"] = (_randn(g, T, D) * 1e-3).to(torch.bfloat16) if case["residual"] else None
            s["buf"] = dict(dx=_bf16(T, D), dgamma=_f32(D))
    elif op == "ffn_fwd":
        M, K, I = case["M"], case["K"], case["I"]
        x = (_randn(g, M, K) * torch.exp(0.5 * _randn(g, K))).to(torch.bfloat16).float()
        q, sc = _quant_rows(x)
        s["xq"] = q.view(torch.uint8)
        s["sx"] = _f32(K // GROUP, _ld(M))
        s["sx"][:, :M] = sc
        wq, s["sw"] = _quant_blocks((_randn(g, 2 * I, K) * 0.02).to(torch.bfloat16).float())
        s["wq"] = wq.view(torch.uint8)
        s["buf"] = dict(h=_codes(M, I), scales=_f32(I // GROUP, _ld(M)))
        if case["save"]:
            s["buf"]["gu"] = _bf16(M, 2 * I)
    elif op == "ffn_bwd":
        M, I = case["M"], case["I"]
        s["gu"] = (_randn(g, M, 2 * I) * 1.5).to(torch.bfloat16)
        s["dh"] = (_randn(g, M, I) * 1e-3).to(torch.bfloat16)
        s["buf"] = dict(q=_codes(M, 2 * I), scales=_f32(2 * I // GROUP, M), qT=_codes(2 * I, M),
                        scalesT=_f32(M // GROUP, 2 * I), hqT=_codes(I, M), hscalesT=_f32(M // GROUP, I))
    else:
        # the gradients are views of one bucket per type, one behind the other
        # with no padding, as are the clipped ones
        s["flat"], s["out"], at, to = {}, {}, {}, {}
        for e, dt in ((4, torch.float32), (2, torch.bfloat16)):
            sizes = [k for k, x in zip(_sizes(case), _elt(case)) if x == e]
            if sizes:
                s["flat"][e] = (_randn(g, sum(sizes)) * case["scale"]).to(dt)
                s["out"][e] = torch.empty_like(s["flat"][e])
                at[e], to[e] = iter(s["flat"][e].split(sizes)), iter(s["out"][e].split(sizes))
        s["grads"] = [next(at[e]) for e in _elt(case)]
        # a quarter of the expected norm, so that the gradients are scaled
        s["max_norm"] = 0.25 * case["scale"] * math.sqrt(sum(_sizes(case)))
        s["buf"] = dict(out=[next(to[e]) for e in _elt(case)], norm=_f32(2))
    return s


# ---------------------------------------------------------- plain forms ----

def _plain_norm_fwd(s):
    h = s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(torch.bfloat16)     # the stream that the next block reads
    f = h.float()
    rstd = 1.0 / torch.sqrt((f * f).mean(1) + EPS)
    q, sc = _quant_rows(f * rstd[:, None] * s["gamma"].float())
    out = {"q": q, "scales": sc, "rstd": rstd}
    if s["residual"] is not None:
        out["h"] = h
    return out


def _plain_norm_bwd(s):
    dy, f, rstd = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    xhat = f * rstd
    dgamma = (dy * xhat).sum(0)
    a = dy * s["gamma"].float()
    dx = rstd * (a - xhat * (a * xhat).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return {"dx": dx.to(torch.bfloat16), "dgamma": dgamma}


def _plain_ffn_fwd(s):
    M, K, I = (s["case"][k] for k in "MKI")
    x = s["xq"].view(torch.float8_e4m3fn).float().view(M, K // GROUP, GROUP) * s["sx"][:, :M].t()[:, :, None]
    w = s["wq"].view(torch.float8_e4m3fn).float().view(2 * I // GROUP, GROUP, K // GROUP, GROUP) * s["sw"][:, None, :, None]
    gu = x.view(M, K) @ w.view(2 * I, K).t()
    gate, up = gu[:, :I], gu[:, I:]
    q, sc = _quant_rows(gate * (1.0 / (1.0 + torch.exp(-gate))) * up)
    out = {"h": q, "scales": sc}
    if s["case"]["save"]:
        out["gu"] = gu.to(torch.bfloat16)
    return out


def _plain_ffn_bwd(s):
    I = s["case"]["I"]
    gate, up, dh = s["gu"][:, :I].float(), s["gu"][:, I:].float(), s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    act = gate * sig
    d = torch.cat([dh * up * sig * (1.0 + gate * (1.0 - sig)), dh * act], 1)
    q, sc = _quant_rows(d)
    qT, scT = _quant_rows(d.t().contiguous())
    hqT, hscT = _quant_rows((act * up).t().contiguous())
    return {"q": q, "scales": sc, "qT": qT, "scalesT": scT, "hqT": hqT, "hscalesT": hscT}


def _plain_clip(s):
    flats = {e: v.float() for e, v in s["flat"].items()}
    norm = torch.sqrt(torch.stack([(v * v).sum() for v in flats.values()]).sum())
    coef = (s["max_norm"] / (norm + EPS)).clamp(max=1.0)
    return {"norm": torch.stack([norm, coef]), "grads": {str(e): (v * coef).to(s["flat"][e].dtype) for e, v in flats.items()}}


# ------------------------------------------------------------ own kernels ----

def _own(s):
    import fp8_fine_grained_gb300 as fg
    op, f8 = s["case"]["op"], torch.float8_e4m3fn
    if op == "norm_fwd":
        q, sc, h, rstd = fg.fp8_rmsnorm(s["x"], s["gamma"], EPS, residual=s["residual"], **s["buf"])
        out = {"q": q.view(f8), "scales": sc[:, :s["case"]["T"]], "rstd": rstd}
        if s["residual"] is not None:
            out["h"] = h
        return out
    if op == "norm_bwd":
        dx, dgamma = fg.fp8_rmsnorm_bwd(s["dy"], s["h"], s["rstd"], s["gamma"], dres=s["dres"], **s["buf"])
        return {"dx": dx, "dgamma": dgamma}
    if op == "ffn_fwd":
        h, sc, gu = fg.fp8_gated_gemm(s["xq"], s["sx"], s["wq"], s["sw"], **s["buf"])
        out = {"h": h.view(f8), "scales": sc[:, :s["case"]["M"]]}
        if s["case"]["save"]:
            out["gu"] = gu
        return out
    if op == "ffn_bwd":
        q, sc, qT, scT, hqT, hscT = fg.fp8_gated_bwd(s["gu"], s["dh"], **s["buf"])
        return {"q": q.view(f8), "scales": sc, "qT": qT.view(f8), "scalesT": scT, "hqT": hqT.view(f8), "hscalesT": hscT}
    norm, _ = fg.grad_clip(s["grads"], s["max_norm"], EPS, **s["buf"])
    return {"norm": norm, "grads": {str(e): v for e, v in s["out"].items()}}


def run(state):
    if own:
        return _own(state)
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "ffn_fwd": _plain_ffn_fwd,
            "ffn_bwd": _plain_ffn_bwd, "clip": _plain_clip}[state["case"]["op"]](state)


# -------------------------------------------------------------- in 64 bits ----

def _round_e4m3(v):
    """v rounded to the nearest E4M3 value, ties to the even one, at most 448 in magnitude."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 1, min=-6) - 3)
    return torch.clamp(torch.round(v / step) * step, -E4M3_MAX, E4M3_MAX)


def _exact_quant(y):
    """Code values and scales (groups outer) of the groups of 128 along y's last dimension."""
    m = y.unfold(1, GROUP, GROUP).abs().amax(2)
    s = torch.where(m > 0, m / E4M3_MAX, torch.ones_like(m))
    return _round_e4m3(y / s.repeat_interleave(GROUP, 1)), s.t()


def _exact_sigmoid(v):
    return torch.where(v >= 0, 1 / (1 + torch.exp(-v)), torch.exp(v) / (1 + torch.exp(v)))


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm_fwd":
        h = s["x"].double()
        if case["residual"]:
            h = (h + s["residual"].double()).to(torch.bfloat16).double()
        rstd = (h.pow(2).sum(1) / case["D"] + EPS).pow(-0.5)
        q, sc = _exact_quant(torch.einsum("td,t,d->td", h, rstd, s["gamma"].double()))
        out = {"q": q, "scales": sc, "rstd": rstd}
        if case["residual"]:
            out["h"] = h
        return out
    if op == "norm_bwd":
        dy, h, r, w = (s[k].double() for k in ("dy", "h", "rstd", "gamma"))
        # y_j = w_j h_j r, r = (mean h^2 + eps)^-1/2, dr/dh_j = -r^3 h_j / D
        dot = (dy * w * h).sum(1)
        dx = r[:, None] * (dy * w) - (r.pow(3) * dot / case["D"])[:, None] * h
        if case["residual"]:
            dx = dx + s["dres"].double()
        return {"dx": dx, "dgamma": torch.einsum("td,td,t->d", dy, h, r)}
    if op == "ffn_fwd":
        M, I = case["M"], case["I"]
        x = s["xq"].view(torch.float8_e4m3fn).double() * s["sx"][:, :M].double().t().repeat_interleave(GROUP, 1)
        w = s["wq"].view(torch.float8_e4m3fn).double()
        w *= s["sw"].double().repeat_interleave(GROUP, 0).repeat_interleave(GROUP, 1)
        gate, up = x @ w[:I].t(), x @ w[I:].t()
        del w
        q, sc = _exact_quant(gate * _exact_sigmoid(gate) * up)
        out = {"h": q, "scales": sc}
        if case["save"]:
            out["gu"] = torch.cat([gate, up], 1)
        return out
    if op == "ffn_bwd":
        gate, up, dh = (v.double() for v in (s["gu"][:, :case["I"]], s["gu"][:, case["I"]:], s["dh"]))
        sig = _exact_sigmoid(gate)
        d = torch.cat([dh * up * (sig + gate * sig * _exact_sigmoid(-gate)), dh * gate * sig], 1)
        h = gate * sig * up
        del gate, up, dh, sig
        q, sc = _exact_quant(d)
        qT, scT = _exact_quant(d.t())
        del d
        hqT, hscT = _exact_quant(h.t())
        return {"q": q, "scales": sc, "qT": qT, "scalesT": scT, "hqT": hqT, "hscalesT": hscT}
    norm = torch.sqrt(sum(v.double().pow(2).sum() for v in s["flat"].values()))
    coef = torch.clamp(s["max_norm"] / (norm + EPS), max=1.0)
    return {"norm": torch.stack([norm, coef]), "grads": {str(e): v.double() * coef for e, v in s["flat"].items()}}
