"""A transformer's gated MLP block on the FP8 path: one training or serving
step out of the library's calls.

    h = x + residual;  n = rmsnorm(h) * gamma
    y = W2 (silu(Wg n) * (Wu n))

Forward: fp8_rmsnorm adds the residual, normalises and writes n as E4M3 codes;
fp8_gated_gemm multiplies them with the stacked weight W13 = [Wg; Wu], applies
the gate and writes its output as E4M3 codes; fprop is the down projection. y
and h leave in bf16: the next block's norm adds them (h is its residual).

Backward, from dy (the gradient of y) and dres (the gradient that reaches h
from the next block's norm): dy is quantised in both layouts from one read,
dgrad through W2 gives the gradient of the gated activation, fp8_gated_bwd
turns it into the quantised gradients of the two projections and the operands
of the weight gradients, two wgrads and a dgrad follow, and fp8_rmsnorm_bwd
ends the block. Kept between the two passes: h, rstd and the two projections
in bf16; the normalised activation and the gated one are recomputed, already
quantised for the weight gradients.

The weights' codes are made once per optimiser step (quantize). Every step of
the computation is a library kernel; rows (tokens) are arbitrary in the forward
pass and a multiple of 128 in the backward pass, whose weight gradients group
the tokens by 128.
"""
from collections import namedtuple

import torch

Weights = namedtuple("Weights", "gamma w13 s13 w2 s2 eps")
Saved = namedtuple("Saved", "h rstd gu")
Grads = namedtuple("Grads", "dx dw13 dw2 dgamma")


def quantize(gamma, w13, w2, eps=1e-6):
    """Weights of the block: gamma [D] (bf16 or float32), w13 bf16 [2I, D] (the
    gate projection's rows on top of the up projection's), w2 bf16 [D, I]."""
    import fp8_fine_grained_gb300 as fg
    if w13.shape[0] != 2 * w2.shape[1] or w13.shape[1] != w2.shape[0] or gamma.numel() != w13.shape[1]:
        raise ValueError("w13 must be [2I, D], w2 [D, I] and gamma [D], got %s, %s, %s"
                         % (tuple(w13.shape), tuple(w2.shape), tuple(gamma.shape)))
    return Weights(gamma, *fg.fp8_quant_128x128(w13), *fg.fp8_quant_128x128(w2), eps)


def forward(x, residual, w, save=False):
    """x bf16 [T, D] and residual (the same, or None). Returns (y bf16 [T, D],
    h bf16 [T, D], Saved or None): h is the residual stream for the next
    block, Saved what backward needs (save=True, T % 128 == 0)."""
    import fp8_fine_grained_gb300 as fg
    if save and x.shape[0] % 128:
        raise ValueError("save=True is for the backward pass, which takes tokens in multiples of 128; got %d"
                         % x.shape[0])
    nq, ns, h, rstd = fg.fp8_rmsnorm(x, w.gamma, w.eps, residual=residual)
    aq, sa, gu = fg.fp8_gated_gemm(nq, ns, w.w13, w.s13, save=save)
    y = fg.fprop(aq, sa, w.w2, w.s2)
    return y, h, Saved(h, rstd, gu) if save else None


def backward(dy, saved, w, dres=None):
    """dy bf16 [T, D], the gradient of y; dres bf16 [T, D] or None, the gradient
    of h from what follows. Returns Grads: dx bf16 [T, D] (the gradient of x
    and of the residual alike) and the FP32 gradients dw13 [2I, D], dw2 [D, I]
    and dgamma [D]."""
    import fp8_fine_grained_gb300 as fg
    if dy.shape[0] == 0:  # sums over no tokens (the GEMMs take no empty contraction)
        zeros = [torch.zeros(s, device=dy.device) for s in (w.w13.shape, w.w2.shape, w.gamma.shape)]
        return Grads(torch.empty_like(dy), *zeros)
    dyq, sdy, dyqT, sdyT = fg.fp8_quant_1x128_dual(dy)
    da = fg.dgrad(dyq, sdy, w.w2, w.s2)
    dq, ds, dqT, dsT, aqT, saT = fg.fp8_gated_bwd(saved.gu, da)
    nqT, nsT = fg.fp8_rmsnorm_t(saved.h, saved.rstd, w.gamma)
    dw13 = fg.wgrad(dqT, dsT, nqT, nsT)
    dw2 = fg.wgrad(dyqT, sdyT, aqT, saT)
    dn = fg.dgrad(dq, ds, w.w13, w.s13)
    dx, dgamma = fg.fp8_rmsnorm_bwd(dn, saved.h, saved.rstd, w.gamma, dres=dres)
    return Grads(dx, dw13, dw2, dgamma)


def clip(grads, max_norm):
    """Scale the block's weight gradients in place so that their global norm is
    at most max_norm; returns (norm, factor) as a float32 [2] on the device."""
    import fp8_fine_grained_gb300 as fg
    return fg.grad_clip([grads.dw13, grads.dw2, grads.dgamma], max_norm)[0]
