"""GPU tests of the losses over a vocabulary that hold more than their general bounds (those of
test_gpu_vocab.py; u = 2^-24, half a step of fp32)."""

import numpy as np
import pytest
import torch

from w8a8_gemm_rl_amd import binding as B

from gpu_helpers import DEV
import vocab_bounds as V
from vocab_bounds import U

pytestmark = pytest.mark.gpu


def _one_certain_id(M, N, K, scale, top, seed):
    """Tokens whose logit is scale * a at one id and 0 at all others, a a bf16 value up to `top`: every
    logit is exact (one product that is not zero). (X, W, target, a)."""
    r = np.random.default_rng(seed)
    a = torch.from_numpy((top ** r.uniform(0.3, 1.0, M)).astype(np.float32)).to(torch.bfloat16)
    slot = torch.from_numpy(r.integers(0, K, M))
    ids = torch.from_numpy(r.permutation(N)[:K])  # the id that hidden value k belongs to
    X = torch.zeros((M, K), dtype=torch.bfloat16)
    X[torch.arange(M), slot] = a
    W = torch.zeros((N, K), dtype=torch.bfloat16)
    W[ids, torch.arange(K)] = 1.0
    return X.to(DEV), W.to(DEV), ids[slot].to(DEV), a.double()


# one shape at least for each tile of the logits
CERTAIN = [(1, 5000, 64), (300, 1031, 520), (60, 20001, 1160), (1000, 3001, 264), (32, 100001, 520), (64, 66000, 72),
           (127, 40001, 584), (700, 40300, 128)]


@pytest.mark.parametrize("M,N,K", CERTAIN)
@pytest.mark.parametrize("scale,top", [(1.0, 30.0), (1.0, 3000.0), (0.7, 300.0), (1.0 / 3.0, 100.0), (30.0, 40.0)])
def test_logp_of_certain_ids_is_never_positive(M, N, K, scale, top):
    """logp = -log(1 + R), R = (N - 1) exp(-z): never above 0, and a divergence from one id of weight 1
    never below. Errors: the sum 1 + R is at most R off by its fp32 additions (what is added is
    rounded to what stands there at worst) and by at most (256 + 8) u (those of one tile), each term
    of R by (4 z log2 e + 8) u, relative; then fp32's rounding."""
    X, W, target, a = _one_certain_id(M, N, K, scale, top, M + N)
    scale = float(np.float32(scale))
    logp, lse = B.vocab_logp(X, W, target, scale=scale)
    loss, _ = B.vocab_distill(X, W, target[:, None], torch.zeros((M, 1), device=DEV), scale=scale)
    z = scale * a
    R = (N - 1) * torch.exp(-z)
    want = -torch.log1p(R)
    lim = torch.clamp(R, max=264 * U) + R / (1 + R) * (4 * z * 1.4427 + 8) * U + want.abs() * U
    # below the logits of a few ids the sum lies in more than one tile and the target adds little
    lim = lim + torch.where(R > 0.01, torch.full_like(R, 264 * U) + 4 * z * U, torch.zeros_like(R))
    got = logp.double().cpu()
    assert bool((got <= 0).all()), float(got.max())
    assert bool(((got - want).abs() <= lim).all()), float(((got - want).abs() - lim).max())
    assert torch.equal(loss, -logp)


def _gradients(M, N, K, live, L, seed, dtype="fp32", scale=1.0, need_dX=True, need_dW=True):
    """Both calls of a problem of which `live` tokens count, held to the bounds for as many parts of G as
    the header promises. Masked rows of X hold NaN, as do their lse and incoming gradients."""
    r = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=r).to(torch.bfloat16).to(DEV)
    w = (torch.randn((N, K), generator=r) * (2.0 / K ** 0.5)).to(torch.bfloat16).to(DEV)
    g = torch.randn(M, generator=r).to(DEV)
    on = torch.zeros(M, dtype=torch.bool)
    on[torch.randperm(M, generator=r)[:live]] = True
    on = on.to(DEV)
    n = max(L, 1)
    ids = torch.randint(0, N, (M, n), generator=r).to(DEV)
    ids[:, 0] = torch.randint(0, N, (M,), generator=r).to(DEV)
    ids[~on] = -1
    X = x.clone()
    X[~on] = float("nan")
    kw = dict(scale=scale)
    e_p = 0.0
    if L:
        teacher = (torch.randn((M, n), generator=r) * 2).to(torch.float32 if dtype == "fp32" else torch.bfloat16)
        teacher = teacher.to(DEV)
        kw.update(index=ids, teacher=teacher)
        _, lse = B.vocab_distill(X, w, **kw)
        y = float(scale) * teacher.double()
        p = torch.softmax(y, 1)
        # exp(y - top) / sum: arguments off by 3 u (|y| + |top|), the rest a few u, the sum L u
        e_p = 2 * (6 * float(y.abs().max()) + n + 10) * U
    else:
        kw.update(target=ids[:, 0].contiguous())
        _, lse = B.vocab_logp(X, w, **kw)
        p = torch.ones((M, 1), dtype=torch.float64, device=DEV)
    lse, gi = lse.clone(), g.clone()
    lse[~on] = float("nan")
    gi[~on] = float("nan")
    call = B.vocab_distill_grad if L else B.vocab_logp_grad
    got = call(X, w, lse=lse, **{"dloss" if L else "dlogp": gi}, need_dX=need_dX, need_dW=need_dW, **kw)
    i = on.nonzero()[:, 0]
    x64, w64 = x[i].double(), w.double()
    G, err = V.gradient_of_logits(x64, w64, ids[i], p[i], g[i].double() * scale, lse[i].double(), scale,
                                  1.0 if L else -1.0, e_p)
    for which, (out, (want, lim)) in enumerate(zip(got, V.gradient_bounds(x64, w64, G, err,
                                                                          2 if live <= V.TWICE else 1))):
        if out is None:
            continue
        if which == 0:
            assert not bool(out[~on].any())
            out = out[i]
        bad = ~((out.double() - want).abs() <= lim)
        assert not bool(bad.any()), ("dX", "dW")[which] + f": {int(bad.sum())}, {bad.nonzero()[:4].tolist()}"


# (tokens, ids, hidden, tokens that count): all of them on tiles of every kind, and both sides of 128
PARTS = [(1, 256, 64, 1), (2, 7, 16, 2), (31, 255, 56, 31), (33, 300, 128, 33), (64, 1000, 136, 64),
         (100, 700, 200, 100), (128, 256, 264, 128), (32, 100001, 520, 32), (64, 66000, 72, 64),
         (127, 40001, 584, 127), (60, 20001, 1160, 60), (128, 5003, 2056, 128),
         (129, 513, 72, 129), (129, 513, 72, 128), (300, 1031, 520, 129), (300, 1031, 520, 128), (300, 1031, 520, 1),
         (700, 40300, 72, 129), (700, 40300, 72, 128), (1000, 3001, 264, 65), (2000, 20001, 136, 33)]


@pytest.mark.parametrize("M,N,K,live", PARTS)
@pytest.mark.parametrize("L,dtype", [(0, "fp32"), (6, "fp32"), (6, "bf16")])
def test_gradients_to_the_parts_of_G(M, N, K, live, L, dtype):
    _gradients(M, N, K, live, L, seed=M + N + K + live, dtype=dtype, scale=0.75 if L else 1.0)
