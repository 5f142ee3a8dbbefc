"""Host side of the losses over a vocabulary: what the binding refuses before any device is looked at,
and that the bounds of the GPU tests can fail (CPU)."""

import random

import pytest
import torch

from w8a8_gemm_rl_amd import binding as B

import vocab_bounds as V
import vocab_shapes as S


def test_hidden_states_and_head_are_matrices():
    """Contiguous tensors of other ranks, whose second size may well agree with the head's."""
    X, W = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((100, 64), dtype=torch.bfloat16)
    assert B._head_args(X, W) == (4, 100, 64, 64, 64)
    assert B._head_args(torch.zeros((4, 72), dtype=torch.bfloat16)[:, :64], W) == (4, 100, 64, 72, 64)
    for x, w in ((X.view(4, 64, 1), W), (X.new_zeros((4, 64, 64)), W), (X.new_zeros((2, 2, 64)), W), (X[0], W),
                 (X, W.new_zeros((100, 64, 64))), (X, W.view(-1)), (X.new_zeros(()), W)):
        with pytest.raises(ValueError):
            B._head_args(x, w)


@pytest.mark.parametrize("fn", ["qr_vocab_logp", "qr_vocab_logp_grad", "qr_vocab_distill", "qr_vocab_distill_grad"])
def test_refusals_of_scales(fn):
    """Scales whose product with log2 e is beyond fp32 are refused, all others pass (to the workspace's check)."""
    from test_oracle_vocab import _call

    for scale, status in ((3.0e38, -1), (1.8e38, -1), (2.0 ** 127, -3), (2.0 ** -149, -3)):
        assert _call(B, fn, scale=scale) == status, scale


def test_workspaces_up_to_the_limits():
    """Sizes and plans over the whole documented range: room for the copied rows of X at least (twice
    over where G may be in two parts), the list's tables, and the gradient's piece and sums of dX."""
    r = torch.Generator().manual_seed(3)
    shapes = [(1 << 22, (1 << 22) - 1, 1 << 16, 1024), (1 << 22, 1, 8, 1), (1, (1 << 22) - 1, 1 << 16, 1024),
              (1, 1, 8, 1), (128, 100, 8, 7), (129, 100, 8, 7)]
    for _ in range(3000):
        u = torch.rand(4, generator=r)
        shapes.append((int(2 ** (22 * u[0])), min(int(2 ** (22 * u[1])), (1 << 22) - 1),
                       max(8, int(2 ** (16 * u[2])) // 8 * 8), int(2 ** (10 * u[3]))))
    for M, N, K, L in shapes:
        piece = B.vocab_plan(M, N, K)[3]
        rows = 2 * M if M <= 128 else M
        assert 1 <= piece <= N and (piece == N or piece >= 4096)
        for fn, entries in (("qr_vocab_logp", 1), ("qr_vocab_distill", L)):
            size = B.workspace_size(fn, M, N, K, entries)
            assert size >= 2 * M * K + 8 * M * entries and size % 256 == 0
            size = B.workspace_size(fn + "_grad", M, N, K, entries)
            assert size >= rows * (2 * K + 2 * piece + 4 * K) + 4 * M * entries and size % 256 == 0


def _problem(M, N, K, L, seed):
    """(x, w, ids, p, a, lse) in float64, of values that bf16 holds."""
    r = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=r).bfloat16().double()
    w = (torch.randn((N, K), generator=r) * (2 / K ** 0.5)).bfloat16().double()
    ids = torch.stack([torch.randperm(N, generator=r)[:L] for _ in range(M)])
    p = torch.softmax(torch.randn((M, L), generator=r).double() * 2, 1)
    return x, w, ids, p, torch.randn(M, generator=r).double(), torch.logsumexp(x @ w.T, 1)


@pytest.mark.parametrize("M,N,K,L", [(1, 256, 64, 1), (31, 255, 56, 1), (64, 1000, 136, 5), (100, 700, 200, 1),
                                     (128, 256, 264, 5), (128, 2003, 72, 20), (300, 1031, 520, 1)])
def test_bounds_of_the_gradients_see_one_part_of_bf16(M, N, K, L):
    """Gradients from G in two parts of bf16 and from G, X and W in fp16 are within their bounds; from G
    in one part of bf16, as where the second were lost, they break both, in dX and in dW."""
    x, w, ids, p, a, lse = _problem(M, N, K, L, M + N)
    G, err = V.gradient_of_logits(x, w, ids, p, a, lse, 1.0, 1.0)
    weight = a.abs() * p.sum(1)
    hi = G.float().bfloat16()
    lo = (G.float() - hi.float()).bfloat16().double()
    half = lambda t, k: (t * 2.0 ** k).float().half().double()  # noqa: E731
    H, xf = half(G / weight[:, None], 14), x * weight[:, None]
    kx, kw = (14 - int(torch.floor(torch.log2(t.abs().max()))) for t in (xf, w))
    fp16 = ((H @ half(w, kw)) * weight[:, None] * 2.0 ** (-14 - kw), (H.T @ half(xf, kx)) * 2.0 ** (-14 - kx))
    two, one = ((t @ w, t.T @ x) for t in (hi.double() + lo, hi.double()))
    for got, kind, ok in ((two, None, True), (fp16, weight, True), (one, None, False), (one, weight, False)):
        for g, (want, lim) in zip(got, V.gradient_bounds(x, w, G, err, kind)):
            bad = int(((g.float().bfloat16().double() - want).abs() > lim).sum())
            assert (bad == 0) == ok, (kind is None, ok, bad, g.numel())


def test_gpu_tests_run_every_body():
    """What calls of a sweep of shapes and masks run on, the GPU tests' shapes run: tiles, the choice
    among them that is left to the GPU, and the hint, each with both gradients or one."""
    kinds = [(True, True), (True, False), (False, True)]
    run = {b for s in S.TILES + S.STREAMED + S.HALF for k in kinds for b in S.bodies(B.vocab_plan, *s, *k)}
    r = random.Random(5)
    met = set()
    for _ in range(20000):
        M, N = int(2 ** r.uniform(0, 13)), int(2 ** r.uniform(0, 18))
        K = max(8, int(2 ** r.uniform(3, 13)) // 8 * 8)
        live = r.choice([M, M, r.randint(0, M), min(M, r.randint(0, 300))])
        met |= {b for k in kinds for b in S.bodies(B.vocab_plan, M, N, K, live, *k)}
    assert met <= run, sorted(met - run)
    for what in ("sums", "G"):  # every tile, with the hint and without
        assert len({b[:4] for b in run if b[0].startswith(what)}) == 16
