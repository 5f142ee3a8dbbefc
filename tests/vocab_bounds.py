"""Bounds of the gradients of the losses over a vocabulary, in float64 (u = 2^-24, half a step of fp32;
bf16's is 2^-8, fp16's 2^-11). They allow for G what it is held as:

z        |dz| <= scale sum_k |x w| (2 K + 2) u, each logit by itself
G        its exponential is off by dz + (4 |z| + 4 |lse| + 16) u + e_p, relative (the argument's product, the
         fused multiply-add, exp2 and four factors; e_p: the weights' sum), what the list takes off by
         (e_p + 8 u). What lies below the normal numbers may come out as 0: (a P + 4) 2^-126.
parts    in two parts of bf16 it then loses the rest's rounding, 2^-8 of 2^-8 |G|.
half     in fp16, 2^14 G / (a P): 2^-11 |G|, below fp16's normal numbers 2^-25 2^-14 a P. W keeps its
         bits but for 2^-24 where its largest value is 2^14 or more: 2^-38 of that. X with the factors a P and a
         power of two, which bring its largest value to 2^14 at least, loses 2^-11 of itself or 2^-25.
dX, dW   sum |dG| |w| + sum |G w| (2 n + 2) u over the n terms (two for an id or token in two parts), and
         the rounding to bf16: 2^-8 of the result.

tests/test_vocab_host.py shows on the CPU that G in one part of bf16 breaks them.
"""

import torch

U = 2.0 ** -24
HALF = 2.0 ** -8
HALF16 = 2.0 ** -11


def gradient_of_logits(x, w, ids, p, a, lse, scale, sign, e_p=0.0):
    """(G, error before its rounding) [M, N]: G = sign a (P exp(z - lse) - p at the ids), a = scale g."""
    N, K = w.shape
    z = scale * (x @ w.T)
    e_z = scale * (x.abs() @ w.abs().T) * ((2 * K + 2) * U)
    P = p.sum(1, keepdim=True)
    dense = P * torch.exp(z - lse[:, None])
    sparse = torch.zeros_like(z).scatter_add_(1, ids.clamp(0, N - 1), p)
    mag = a.abs()[:, None]
    rel = e_z + (4 * z.abs() + 4 * lse.abs()[:, None] + 16) * U + e_p
    err = mag * (dense * rel + sparse * (e_p + 8 * U)) * (1 + HALF) + (mag * P + 4) * 2.0 ** -126
    return sign * a[:, None] * (dense - sparse), err


def gradient_bounds(x, w, G, err, weight=None):
    """[(exact, bound)] of dX and dW for bf16 results: G in two parts, or, with the tokens' weights a P,
    in fp16."""
    ax, aw, aG = x.abs(), w.abs(), G.abs()
    if weight is None:
        e = HALF * HALF * aG + err
        slack, n = [e @ aw, e.T @ ax], 2
    else:
        weight = weight.abs()
        e = HALF16 * aG + err + 2.0 ** -39 * weight[:, None]
        # of H = G / weight, by the largest of weight |x|
        low = ((aG + e) / weight.clamp(min=1e-300)[:, None]).sum(0) * (2.0 ** -39 * float((weight * ax.amax(1)).max()))
        slack, n = [e @ aw + (aG + e).sum(1, keepdim=True) * (2.0 ** -38 * float(aw.max())),
                    e.T @ ax + (aG + e).T @ ax * (HALF16 + 8 * U) + low[:, None]], 1
    out = []
    for want, lim, mag, terms in ((G @ w, slack[0], aG @ aw, w.shape[0]), (G.T @ x, slack[1], aG.T @ ax, x.shape[0])):
        lim = lim + (mag + lim) * ((2 * n * terms + 2) * U)
        out.append((want, lim + HALF * (want.abs() + lim) + 1e-37))
    return out
