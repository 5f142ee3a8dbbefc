"""GPU tests of the losses over a vocabulary that hold more than their general bounds (those of
test_gpu_vocab.py, whose u = 2^-24 and helpers are used here)."""

import numpy as np
import pytest
import torch

from w8a8_gemm_rl_amd import binding as B

from gpu_helpers import DEV
from test_gpu_vocab import U

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
