"""Bounds of the gradients of the losses over a vocabulary, in float64 (u = 2^-24, half a step of fp32;
bf16's is 2^-8). They allow for G what its parts allow:

z        |dz| <= scale sum_k |x w| (2 K + 2) u, each logit by itself
G        its exponential is off by dz + (4 |z| + 4 |lse| + 16) u + e_p, relative (the argument's product, the
         fused multiply-add, exp2 and four factors; e_p: the weights' sum), what the list takes off by
         (e_p + 8 u). In one part of bf16 it then loses 2^-8 |G|, in two the rest's rounding, 2^-8 of
         2^-8 |G|. What lies below the normal numbers may come out as 0: (a P + 4) 2^-126.
dX, dW   sum |dG| |w| + sum |G w| (2 n + 2) u over the n terms (two for an id or token in two parts), and
         the rounding to bf16: 2^-8 of the result.

tests/test_vocab_host.py shows on the CPU that a lost second part breaks them.
"""

import torch

U = 2.0 ** -24
HALF = 2.0 ** -8
PARTS = {1: HALF, 2: HALF * HALF}
TWICE = 128  # tokens that count, up to which G is held in two parts


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


def gradient_bounds(x, w, G, err, parts):
    """[(exact, bound)] of dX and dW for bf16 results; `parts` of G."""
    eG = PARTS[parts] * G.abs() + err
    out = []
    for want, lim, mag, n in ((G @ w, eG @ w.abs(), G.abs() @ w.abs(), w.shape[0]),
                              (G.T @ x, eG.T @ x.abs(), G.abs().T @ x.abs(), x.shape[0])):
        lim = lim + (mag + lim) * ((2 * parts * n + 2) * U)
        out.append((want, lim + HALF * (want.abs() + lim) + 1e-37))
    return out
