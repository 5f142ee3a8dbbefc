"""Pins of the oracle's losses over a vocabulary, and the host-side checks of their entry points (CPU)."""

import ctypes

import numpy as np
import pytest
import torch

import oracle as O

RNG = np.random.default_rng


def _case(M, N, K, L, seed):
    r = RNG(seed)
    X, W = r.standard_normal((M, K)), r.standard_normal((N, K)) * 0.3
    target = r.integers(0, N, M)
    index = np.stack([r.permutation(N)[:L] for _ in range(M)])
    teacher = r.standard_normal((M, L)) * 2
    return X, W, target, index, teacher, r.standard_normal(M)


def test_logp_against_torch():
    X, W, target, _, _, g = _case(7, 23, 5, 3, 1)
    target[2], target[5] = -100, 23
    x, w = torch.tensor(X, requires_grad=True), torch.tensor(W, requires_grad=True)
    t = torch.tensor(np.where((target >= 0) & (target < 23), target, -100))
    ce = torch.nn.functional.cross_entropy(1.7 * (x @ w.T), t, reduction="none", ignore_index=-100)
    value, lse = O.vocab_loss(X, W, scale=1.7, target=target)
    assert np.allclose(value, -ce.detach().numpy(), rtol=1e-12, atol=1e-12)
    assert value[2] == 0 and lse[2] == 0 and value[5] == 0 and lse[5] == 0
    (-ce * torch.tensor(g)).sum().backward()
    dX, dW, _ = O.vocab_grad(X, W, g, scale=1.7, target=target)
    assert np.allclose(dX, x.grad.numpy(), rtol=1e-11, atol=1e-12)
    assert np.allclose(dW, w.grad.numpy(), rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("own_sum", [False, True])
def test_distill_against_torch(own_sum):
    X, W, _, index, teacher, g = _case(6, 31, 4, 5, 2)
    index[0, 3:], index[1], index[2, 1] = -1, -1, 31
    tl = np.log(np.exp(0.6 * teacher).sum(1)) + 0.3 if own_sum else None
    x, w = torch.tensor(X, requires_grad=True), torch.tensor(W, requires_grad=True)
    logq = torch.log_softmax(0.6 * (x @ w.T), dim=1)
    total = 0
    want = np.zeros(6)
    for t in range(6):
        js = [j for j in range(5) if 0 <= index[t, j] < 31]
        if not js:
            continue
        y = torch.tensor(0.6 * teacher[t, js])
        logp = y - (tl[t] if own_sum else torch.logsumexp(y, 0))
        loss = (logp.exp() * (logp - logq[t, torch.tensor(index[t, js])])).sum()
        want[t] = loss.item()
        total = total + g[t] * loss
    total.backward()
    lists = dict(index=index, teacher=teacher, teacher_lse=tl)
    value, lse = O.vocab_loss(X, W, scale=0.6, **lists)
    assert np.allclose(value, want, rtol=1e-11, atol=1e-12) and value[1] == 0 and lse[1] == 0
    dX, dW, _ = O.vocab_grad(X, W, g, scale=0.6, **lists)
    assert np.allclose(dX, x.grad.numpy(), rtol=1e-10, atol=1e-12)
    assert np.allclose(dW, w.grad.numpy(), rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("which", ["target", "index"])
def test_gradients_against_differences(which):
    X, W, target, index, teacher, g = _case(3, 11, 4, 3, 3)
    index[1, 2] = index[1, 0]  # one id twice
    lists = dict(target=target) if which == "target" else dict(index=index, teacher=teacher)
    f = lambda a, b: float(g @ O.vocab_loss(a, b, scale=1.3, **lists)[0])  # noqa: E731
    dX, dW, _ = O.vocab_grad(X, W, g, scale=1.3, **lists)
    h = 1e-5
    for A, D in ((X, dX), (W, dW)):
        for i in np.ndindex(A.shape):
            old = A[i]
            A[i] = old + h
            up = f(X, W)
            A[i] = old - h
            down = f(X, W)
            A[i] = old
            # central differences: h^2 times third derivatives of order one, and 1e-15 / h
            assert abs((up - down) / (2 * h) - D[i]) < 1e-8


def test_lists_by_hand():
    # two entries at 0 and log 3, one of them twice as an id; weights 1/4, 3/4
    ids, p, live = O.vocab_lists(index=[[4, 4, -1], [-1, 9, 9], [0, 1, 2]], N=9, scale=1.0,
                                 teacher=[[0.0, np.log(3.0), 5.0], [1.0, 1.0, 1.0], [-np.inf] * 3])
    assert np.allclose(p[0], [0.25, 0.75, 0.0]) and list(live) == [True, False, True]
    assert not p[1].any() and not p[2].any()
    # uniform logits: the loss is log N - entropy of p, the gradient of no token moves X
    X, W = np.zeros((3, 2)), np.ones((9, 2))
    value, lse = O.vocab_loss(X, W, index=ids, teacher=np.array([[0.0, np.log(3.0), 5.0]] * 3) * [[1], [1], [1]])
    assert np.isclose(value[0], np.log(9) + 0.25 * np.log(0.25) + 0.75 * np.log(0.75))
    assert np.isclose(lse[0], np.log(9)) and value[1] == 0 and lse[1] == 0


# ----------------------------------------------------------------------------
# Entry points: arguments refused on the host
# ----------------------------------------------------------------------------

FN = ("qr_vocab_logp", "qr_vocab_logp_grad", "qr_vocab_distill", "qr_vocab_distill_grad")
P = ctypes.c_void_p


def _call(B, fn, **kw):
    """The entry point with arguments that pass, but for those given (pointers are made up: a call
    that passes every check is not made here)."""
    d = dict(X=P(4096), ldx=64, W=P(8192), ldw=64, M=4, N=100, K=64, target=P(64), index=P(64), teacher=P(64),
             bf16=0, tl=None, L=3, scale=1.0, out=P(128), lse=P(256), g=P(512), dX=P(1 << 20), lddx=64,
             dW=P(1 << 21), lddw=64, ws=P(1 << 22), wsb=0)
    d.update(kw)
    a = [d[k] for k in ("X", "ldx", "W", "ldw", "M", "N", "K")]
    a += [d["target"]] if "logp" in fn else [d[k] for k in ("index", "teacher", "bf16", "tl", "L")]
    a += [d["scale"]]
    a += [d[k] for k in ("lse", "g", "dX", "lddx", "dW", "lddw")] if "grad" in fn else [d["out"], d["lse"]]
    return getattr(B.lib(), fn)(*a, d["ws"], d["wsb"], None)


@pytest.fixture(scope="module")
def B():
    from w8a8_gemm_rl_amd import binding
    binding.lib()
    return binding


@pytest.mark.parametrize("fn", FN)
def test_refusals(B, fn):
    c = lambda **kw: _call(B, fn, **kw)  # noqa: E731
    assert c() == -3 and "workspace" in B.lib().qr_last_error().decode()  # all else passes
    assert c(ws=None) == -3
    assert c(ws=P((1 << 22) + 128), wsb=1 << 40) == -3  # misaligned
    for bad in (dict(M=-1), dict(N=0), dict(N=-1), dict(K=0), dict(ldx=56), dict(ldw=56), dict(X=None),
                dict(W=None), dict(lse=None)):
        assert c(**bad) == -1, bad
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert c(scale=s) == -1
    for bad in (dict(K=60), dict(ldx=68), dict(ldw=65), dict(X=P(4104)), dict(W=P(8200)), dict(K=65544, ldx=65544, ldw=65544, lddx=65544, lddw=65544),
                dict(M=(1 << 22) + 1), dict(N=1 << 22), dict(ldw=(1 << 21) + 8), dict(ldx=(1 << 21) + 8),
                dict(lse=P(258))):
        assert c(**bad) == -2, bad
    if "grad" in fn:
        assert c(dX=None, dW=None) == -1 and c(g=None) == -1 and c(lddx=56) == -1 and c(lddw=8) == -1
        assert c(lddx=68) == -2 and c(dW=P((1 << 21) + 8)) == -2 and c(g=P(514)) == -2
    else:
        assert c(out=None) == -1 and c(out=P(130)) == -2
    if "logp" in fn:
        assert c(target=None) == -1 and c(target=P(68)) == -2
    else:
        assert c(index=None) == -1 and c(teacher=None) == -1 and c(bf16=2) == -1
        assert c(L=0) == -1 and c(L=1025) == -1 and c(teacher=P(66)) == -2 and c(tl=P(66)) == -2
        assert c(teacher=P(66), bf16=1) == -3
    if "grad" not in fn:  # no tokens: nothing to do
        assert c(M=0, X=None, target=None, index=None, teacher=None, out=None, lse=None, ws=None) == 0


def test_workspace_sizes(B):
    for fn in FN:
        L = 1 if "logp" in fn else 64
        size = lambda M, N, K: B.workspace_size(fn, M, N, K, L)  # noqa: E731
        assert size(0, 100, 64) == 0 and size(1, 1, 8) > 0
        for bad in ((-1, 10, 64), (4, 0, 64), (4, 10, 12), (4, 10, 0), (1 << 23, 10, 64)):
            with pytest.raises(B.QRError):
                size(*bad)
        # the logits of 8192 tokens of 131072 ids would take 4 GiB in fp32
        assert size(8192, 131072, 3584) < 1 << 30
    for fn in FN[2:]:
        with pytest.raises(B.QRError):
            B.workspace_size(fn, 4, 100, 64, 0)


def test_plans(B):
    """Every plan that a sweep of shapes meets is one that the GPU tests run."""
    from vocab_shapes import LARGE, SMALL

    run = {B.vocab_plan(*s)[:3] for s in SMALL + LARGE}
    # the gradient's pieces have plans of their own, of fewer ids
    r = RNG(7)
    met = set()
    for _ in range(20000):
        M, N, K = (int(round(2 ** r.uniform(0, hi))) for hi in (14, 18, 13))
        K = max(8, K // 8 * 8)
        ids, tokens, rows, piece = B.vocab_plan(M, N, K)
        assert piece <= N and (piece == N or piece % 256 == 0)
        met.add((ids, tokens, rows))
    assert {p[:2] for p in met} <= {p[:2] for p in run}
    assert {p[2] for p in met} <= {p[2] for p in run}
    for bad in ((0, 10, 64), (4, 0, 64), (4, 10, 12)):
        with pytest.raises(B.QRError):
            B.vocab_plan(*bad)
