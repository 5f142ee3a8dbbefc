"""GPU tests of the losses over a large vocabulary against the float64 oracle.

Bounds, derived here and used throughout (u = 2^-24, half a step of fp32; bf16's is 2^-8):

logits   products of two bf16 values are exact in fp32; K of them added in any order, each addition
         off by at most 2 u (the matrix cores may cut where fp32 rounds), and one product with the
         scale: |dz| <= scale sum|x w| (2 K + 2) u =: e_z[t, v]; e_z[t] is its maximum over v.
lse      exp2's argument is an fma of a product with the rounded scale * log2(e) (2 u |z| log2 e in
         all) and a maximum rounded alike; exp2 itself within 2^-22; at most 512 fp32 additions in a
         tile and few in float64 after: relative error of the sum <= (2 * 2 |z|max + 4 + 512 + 8) u, and a
         last rounding of lse: |dlse| <= e_z + (4 zmax + 600) u + |lse| u.
logp     |d| <= e_z (twice: logit and sum) + dlse + |logp| u.
weights  p = expf(c y - top) / sum or expf(c y - lse'): arguments off by at most 3 u max(|c y| + |top|),
         expf and the division a few u, the sum L u: relative 2 (3 ymax + L + 10) u =: e_p.
loss     sum_j |p_j| (e_z + dlse) + p_j (|log p_j| + |z_j - lse| + 1) e_p, and the last rounding.
G        the exponential's argument off by e_z + (4 |z| + 4 |lse|) u, factors a few u, lists' weights e_p,
         then rounded to bf16: |dG| <= 2^-8 |G| + (a p)(e_z + (4 zmax + 4 |lse| + 16) u) + |b| (e_p + 8 u)
         (1 + 2^-8), the subtraction's rounding within the 8 u of either; and where the exponential or
         G is below the normal numbers, 2^-126, it may come out as 0: (a + 1) 2^-126.
dX, dW   sum |dG| |w| + sum |G w| (2 n + 2) u (n terms), then rounded to bf16: 2^-8 of the result.
"""

import numpy as np
import pytest
import torch

import oracle as O
from w8a8_gemm_rl_amd import binding as B
from w8a8_gemm_rl_amd import inputs as I

from gpu_helpers import DEV
from vocab_shapes import LARGE, SMALL

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = 2.0 ** -8
TINY = 1e-37  # below bf16's and fp32's normal range results may be flushed or lose bits


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def _f64(t):
    return t.double().cpu().numpy()


def _padded(t, pad, fill):
    """The tensor inside rows `pad` elements longer that hold `fill`."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype)
    buf[:, : t.shape[1]] = t
    return buf.to(DEV)[:, : t.shape[1]]


def _inputs(M, N, K, L=0, seed=0, masked=(), pad=0, dtype="fp32", own_sum=False, scale=1.0):
    """Inputs of a call on the device and their float64 copies; masked tokens' rows of X hold NaN,
    as does the padding between rows."""
    r = np.random.default_rng(seed)
    X = _bf16(r.standard_normal((M, K)))
    W = _bf16(r.standard_normal((N, K)) * (2.0 / np.sqrt(K)))
    masked = np.zeros(M, bool) if len(masked) == 0 else np.asarray(masked)
    d = dict(X64=_f64(X), W64=_f64(W), scale=scale, masked=masked)
    X = X.clone()
    X[torch.from_numpy(masked)] = float("nan")
    d["X"], d["W"] = _padded(X, pad, float("nan")), _padded(W, pad, float("nan"))
    if L:
        index = np.stack([r.permutation(max(N, L))[:L] for _ in range(M)]).astype(np.int64)
        teacher = torch.from_numpy((r.standard_normal((M, L)) * 3).astype(np.float32))
        if dtype == "bf16":
            teacher = teacher.to(torch.bfloat16)
        index[masked] = r.choice([-1, N, N + 5, -7], (int(masked.sum()), L))
        lists = dict(index=index, teacher=_f64(teacher), teacher_lse=None)
        dev = dict(index=torch.from_numpy(index).to(DEV), teacher=teacher.to(DEV), teacher_lse=None)
        if own_sum:
            tl = np.log(np.exp(scale * lists["teacher"]).sum(1) * 1.25).astype(np.float32)
            tl[masked] = np.nan
            lists["teacher_lse"], dev["teacher_lse"] = tl.astype(np.float64), torch.from_numpy(tl).to(DEV)
    else:
        target = r.integers(0, N, M)
        target[masked] = r.choice([-1, N, -100, 1 << 40], int(masked.sum()))
        lists = dict(target=target)
        dev = dict(target=torch.from_numpy(target).to(DEV))
    d.update(lists=lists, dev=dev)
    return d


def _errors(d):
    """(z, lse, live, ids, p, e_z per token, largest |z| per token, e_p) of the bounds above."""
    z, lse = O.vocab_logits(d["X64"], d["W64"], d["scale"])
    K = d["X64"].shape[1]
    e_z = (d["scale"] * (np.abs(d["X64"]) @ np.abs(d["W64"]).T) * (2 * K + 2) * U).max(axis=1)
    ids, p, live = O.vocab_lists(scale=d["scale"], N=d["W64"].shape[0], **d["lists"])
    e_p = 0.0
    if "index" in d["lists"]:
        y = d["scale"] * np.abs(d["lists"]["teacher"])
        y = np.where(np.isfinite(y), y, 0.0).max() * 2
        if d["lists"]["teacher_lse"] is not None:
            y += np.nanmax(np.abs(d["lists"]["teacher_lse"]))
        e_p = 2 * (3 * y + ids.shape[1] + 10) * U
    return z, lse, live, ids, p, e_z, np.abs(z).max(axis=1), e_p


def _forward(d, **kw):
    if "index" in d["dev"]:
        return B.vocab_distill(d["X"], d["W"], scale=d["scale"], **d["dev"], **kw)
    return B.vocab_logp(d["X"], d["W"], scale=d["scale"], **d["dev"], **kw)


def _backward(d, lse, g, **kw):
    call = B.vocab_distill_grad if "index" in d["dev"] else B.vocab_logp_grad
    return call(d["X"], d["W"], lse=lse, **{"dloss" if "index" in d["dev"] else "dlogp": g}, scale=d["scale"],
                **d["dev"], **kw)


def _check_forward(d, got, err=None):
    z, lse, live, ids, p, e_z, zmax, e_p = err or _errors(d)
    value, own = (t.cpu().numpy().astype(np.float64) for t in got)
    want, wlse = O.vocab_loss(d["X64"], d["W64"], scale=d["scale"], **d["lists"])
    b_lse = e_z + (4 * zmax + 600) * U + np.abs(lse) * U
    assert np.all(np.abs(own - wlse) <= b_lse)
    if "index" in d["lists"]:
        zi = np.take_along_axis(z, ids.clip(0, z.shape[1] - 1), axis=1) - lse[:, None]
        lp = np.abs(np.log(np.where(p > 0, p, 1.0)))
        b = (p * (e_z + b_lse)[:, None] + p * (lp + np.abs(zi) + 1) * (e_p + 8 * U)).sum(axis=1)
    else:
        b = e_z + b_lse
    assert np.all(np.abs(value - want) <= b + np.abs(want) * U + 1e-30)
    assert not value[~live].any() and not own[~live].any()


def _check_backward(d, lse, g, dX, dW, err=None):
    """`lse` is what the call was given."""
    z, _, live, ids, p, e_z, zmax, e_p = err or _errors(d)
    l64 = np.where(live, lse.cpu().numpy().astype(np.float64), 0.0)
    g64 = np.where(live, g.cpu().numpy().astype(np.float64), 0.0)
    X64 = np.where(live[:, None], d["X64"], 0.0)
    wX, wW, G = O.vocab_grad(X64, d["W64"], g64, scale=d["scale"], lse=l64, **d["lists"])
    a = np.abs(g64) * d["scale"]
    dense = a[:, None] * p.sum(axis=1, keepdims=True) * np.exp(np.where(live[:, None], z - l64[:, None], 0.0))
    sparse = np.zeros_like(G)
    for t in range(G.shape[0]):
        np.add.at(sparse[t], ids[t].clip(0, G.shape[1] - 1), p[t] * a[t])
    rel = e_z + (4 * zmax + 4 * np.abs(l64) + 16) * U + e_p
    eG = HALF * np.abs(G) + (dense * rel[:, None] + sparse * (e_p + 8 * U)) * (1 + HALF)
    eG += ((a * p.sum(axis=1) + 1) * 2.0 ** -126)[:, None]
    n_v, n_t = G.shape[1], G.shape[0]
    for got, want, bound, mag, n in (
            (dX, wX, eG @ np.abs(d["W64"]), np.abs(G) @ np.abs(d["W64"]), n_v),
            (dW, wW, eG.T @ np.abs(X64), np.abs(G).T @ np.abs(X64), n_t)):
        if got is None:
            continue
        o = _f64(got)
        lim = bound + (mag + bound) * (2 * n + 2) * U
        lim = lim + HALF * (np.abs(want) + lim) + TINY
        bad = ~(np.abs(o - want) <= lim)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())
    if dX is not None:
        assert not _f64(dX)[~live].any()


def _both(d, need_dX=True, need_dW=True, seed=5):
    err = _errors(d)
    value, lse = _forward(d)
    _check_forward(d, (value, lse), err)
    M = d["X"].shape[0]
    g = np.random.default_rng(seed).standard_normal(M).astype(np.float32)
    lse, g = lse.clone(), torch.from_numpy(g)
    g[torch.from_numpy(d["masked"])] = float("nan")
    lse[torch.from_numpy(d["masked"]).to(DEV)] = float("nan")
    g = g.to(DEV)
    dX, dW = _backward(d, lse, g, need_dX=need_dX, need_dW=need_dW)
    assert (dX is None) == (not need_dX) and (dW is None) == (not need_dW)
    _check_backward(d, lse, g, dX, dW, err)
    return value, lse, g, dX, dW


@pytest.mark.parametrize("M,N,K", SMALL)
def test_logp_sizes(M, N, K):
    _both(_inputs(M, N, K, seed=M + N + K, pad=8 * (M % 3)))


@pytest.mark.parametrize("M,N,K", SMALL)
@pytest.mark.parametrize("L,dtype,own_sum", [(1, "fp32", False), (5, "bf16", True), (70, "fp32", False)])
def test_distill_sizes(M, N, K, L, dtype, own_sum):
    _both(_inputs(M, N, K, L=L, seed=M + N + K + L, dtype=dtype, own_sum=own_sum, scale=0.7, pad=8 * (N % 2)))


def _check_large(X, W, got, lse, grads, g, ids, p, live, sign, e_p):
    """The bounds of the module's head, in float64 on the device. ids [M, L], p [M, L], `got` the
    losses' values; zeros where not live."""
    M, K = X.shape
    N = W.shape[0]
    x, w = X.double() * live[:, None], W.double()
    z = x @ w.T
    l64 = torch.logsumexp(z, 1)
    e = (x.abs() @ w.abs().T).amax(1) * (2 * K + 2) * U + (4 * z.abs().amax(1) + 5 * l64.abs() + 616) * U
    assert torch.all(((lse.double() - l64).abs() <= e)[live]) and not bool(lse[~live].any())
    zi = torch.gather(z, 1, ids.clamp(0, N - 1)) - l64[:, None]
    lp = torch.where(p > 0, p, 1.0).log()
    want = (p * (lp - zi)).sum(1) if sign > 0 else zi[:, 0]
    lim = (p * (2 * e[:, None] + (lp.abs() + zi.abs() + 1) * (e_p + 8 * U))).sum(1) + want.abs() * U
    assert torch.all(((got.double() - want).abs() <= lim)[live]) and not bool(got[~live].any())
    a = (g.double() * live * sign)[:, None]
    q = p.sum(1, keepdim=True) * torch.exp(z - lse.double()[:, None])
    t = torch.zeros_like(q).scatter_add_(1, ids.clamp(0, N - 1), p)
    G, mag = (q - t) * a, (q + t) * a.abs()
    eG = HALF * G.abs() + mag * (e[:, None] + e_p + 24 * U) * (1 + HALF) + (a.abs() + 1) * 2.0 ** -126
    for out, want, bound, big, n in ((grads[0], G @ w, eG @ w.abs(), G.abs() @ w.abs(), N),
                                     (grads[1], G.T @ x, eG.T @ x.abs(), G.abs().T @ x.abs(), M)):
        lim = bound + (big + bound) * (2 * n + 2) * U
        assert torch.all((out.double() - want).abs() <= lim + HALF * (want.abs() + lim) + TINY)
    assert not bool(grads[0][~live].any())


def _large(M, N, K, keep):
    r = torch.Generator().manual_seed(M + N + K)
    X = torch.randn((M, K), generator=r).to(torch.bfloat16).to(DEV)
    W = (torch.randn((N, K), generator=r) * (1.5 / K ** 0.5)).to(torch.bfloat16).to(DEV)
    live = (torch.rand(M, generator=r) < keep).to(DEV)
    live[M // 2] = True
    g = torch.randn(M, generator=r).to(DEV)
    target = torch.randint(0, N, (M,), generator=r).to(DEV)
    target[~live] = -1
    logp, lse = B.vocab_logp(X, W, target)
    grads = B.vocab_logp_grad(X, W, target, lse, g)
    _check_large(X, W, logp, lse, grads, g, target[:, None], live[:, None].double(), live, -1.0, 0.0)
    L = 12
    index = torch.randint(0, N, (M, L), generator=r).to(DEV)
    index[:, 3] = N - 1 - torch.arange(M, device=DEV) % 3
    index[torch.rand((M, L), generator=r).to(DEV) < 0.2] = N
    index[:, 0] = 0
    index[~live] = -1
    teacher = (torch.randn((M, L), generator=r) * 2).to(DEV)
    loss, lse = B.vocab_distill(X, W, index, teacher)
    grads = B.vocab_distill_grad(X, W, index, teacher, lse, g)
    ok = (index >= 0) & (index < N)
    p = torch.softmax(teacher.double().masked_fill(~ok, -1e9), 1) * ok
    e_p = 2 * (6 * float(teacher.abs().max()) + L + 10) * U
    _check_large(X, W, loss, lse, grads, g, index, p, live, 1.0, e_p)


@pytest.mark.parametrize("M,N,K", LARGE)
def test_large_sizes(M, N, K):
    _large(M, N, K, 0.9)


@pytest.mark.parametrize("M,N,K,keep", [(200, 100003, 264, 0.9), (200, 100003, 264, 0.3), (700, 40300, 264, 0.1),
                                        (700, 20001, 72, 0.25),
                                        (2000, 3001, 136, 0.05), (2000, 20001, 72, 0.0)])
def test_few_of_many_tokens_count(M, N, K, keep):
    """Plans for tiles of 256 tokens where one or two tiles of 128 hold all that count, G in two parts
    among many masked tokens, none at all."""
    assert M > 1000 or B.vocab_plan(M, N, K)[1] == 256
    _large(M, N, K, keep)


@pytest.mark.parametrize("L", [0, 6])
@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("mask", ["all", "first", "last", "half", "but one"])
def test_masked_tokens_hold_anything(M, L, mask):
    m = np.zeros(M, bool)
    if mask == "all":
        m[:] = True
    elif mask == "first":
        m[0] = True
    elif mask == "last":
        m[-1] = True
    elif mask == "half":
        m[np.random.default_rng(M).permutation(M)[: M // 2]] = True
    else:
        m[:] = True
        m[M // 2] = False
    d = _inputs(M, 413, 88, L=L, seed=M, masked=m, pad=16)
    _, _, _, dX, dW = _both(d)
    if m.all():
        assert not bool(dX.any()) and not bool(dW.any())


def test_lists_of_every_kind():
    """Short lists, one id twice (and everywhere), ids next to each other and across tiles' borders,
    teacher logits at -inf and at the type's lowest value, a list with no weight at all."""
    M, N, K, L = 12, 1100, 64, 40
    d = _inputs(M, N, K, L=L, seed=11)
    ix, te = d["lists"]["index"], d["lists"]["teacher"]
    ix[0, 3:] = -1
    ix[1] = np.arange(L) + 236          # across id 256
    ix[2] = 1099 - np.arange(L)         # falling, to the last id
    ix[3, 5:9] = ix[3, 0]
    ix[4] = 17                          # one id 40 times
    te[5, 3:20] = -np.inf
    te[6] = -np.inf
    te[7] = np.float64(np.finfo(np.float32).min)
    te[8, 1:] = np.float64(np.finfo(np.float32).min)
    ix[9, ::2] = N + np.arange(L // 2)
    ix[10, : L - 1] = -3
    te[11] = 80.0 + np.arange(L)
    d["dev"]["index"] = torch.from_numpy(ix).to(DEV)
    d["dev"]["teacher"] = torch.from_numpy(te.astype(np.float32)).to(DEV)
    # the bound's largest |c y|: rows whose lowest values have weight 0 or are all alike are exact
    keep = te.copy()
    te_err = np.where(np.abs(te) > 1e30, 0.0, te)
    d["lists"]["teacher"] = te_err
    e_p = _errors(d)[7]
    d["lists"]["teacher"] = keep
    err = _errors(d)[:7] + (e_p,)
    value, lse = _forward(d)
    _check_forward(d, (value, lse), err)
    g = torch.linspace(-1.0, 2.0, M, device=DEV)
    dX, dW = _backward(d, lse, g)
    _check_backward(d, lse, g, dX, dW, err)
    assert float(value[6]) == 0.0 and not bool(dX[6].any()) and float(lse[6]) != 0.0


def test_longest_lists_and_the_longest_refused():
    _both(_inputs(3, 5000, 64, L=1024, seed=3))
    _both(_inputs(2, 1024, 64, L=1024, seed=4, own_sum=True))
    d = _inputs(2, 2000, 64, L=1025, seed=3)
    with pytest.raises(B.QRError):
        _forward(d)


@pytest.mark.parametrize("scale", [0.01, 30.0])
def test_scales(scale):
    """Nearly flat and nearly certain distributions."""
    _both(_inputs(70, 600, 72, seed=8, scale=scale))
    _both(_inputs(70, 600, 72, L=9, seed=9, scale=scale, own_sum=True))


def test_exact_values():
    """A head of zeros: every probability is 1 / 256, so G is exact in bf16, and with small whole
    numbers in X and powers of two as incoming gradients dW has no rounding but its last."""
    M, N, K = 320, 256, 72
    r = np.random.default_rng(2)
    X = _bf16(r.integers(-3, 4, (M, K)))
    target = torch.from_numpy(r.integers(0, N, M))
    g = torch.from_numpy(2.0 ** r.integers(-3, 3, M)).float()
    W = torch.zeros((N, K), dtype=torch.bfloat16, device=DEV)
    logp, lse = B.vocab_logp(X.to(DEV), W, target.to(DEV))
    assert torch.all((logp.cpu().double() + np.log(256)).abs() <= 600 * U + 6 * U)
    dX, dW = B.vocab_logp_grad(X.to(DEV), W, target.to(DEV), lse, g.to(DEV))
    G = torch.nn.functional.one_hot(target, N).double() - 1.0 / N
    want = (g.double()[:, None] * G).T @ X.double()
    assert torch.equal(dW.cpu(), want.float().to(torch.bfloat16)) and not bool(dX.any())


def test_gradient_against_differences():
    """The calls' own losses at shifted weights: steps h along a direction D, (f(+h) - f(-h)) / 2 h
    against <dW, D>. Each f is a sum of M values off by at most e (the forward bound): M e / h, plus
    h^2 / 6 of the third derivative (at most 8 |scale dz|^3 a token), plus what bf16 takes from dW."""
    M, N, K = 24, 300, 64
    d = _inputs(M, N, K, L=4, seed=21, scale=1.0)
    r = np.random.default_rng(3)
    W64 = np.round(d["W64"] * 64) / 64  # steps of 1/8 stay exact in bf16
    D = np.zeros((N, K))
    D[r.integers(0, N, 40), r.integers(0, K, 40)] = 1.0
    h = 0.125
    def f(s):
        d["W64"] = W64 + s * D
        d["W"] = _bf16(d["W64"]).to(DEV)
        assert np.array_equal(_f64(d["W"]), d["W64"])
        value, lse = _forward(d)
        _check_forward(d, (value, lse))
        return value, lse
    up, down = f(h)[0], f(-h)[0]
    value, lse = f(0.0)
    g = torch.ones(M, device=DEV)
    _, dW = _backward(d, lse, g)
    dz = np.abs(d["X64"] @ D.T).max()
    z, l64, _, _, _, e_z, zmax, e_p = _errors(d)
    e = (4 * e_z + (8 * zmax + 1300) * U + 40 * (e_p + 8 * U)).max()
    lhs = float((up.double() - down.double()).sum()) / (2 * h)
    rhs = float((_f64(dW) * D).sum())
    slack = 2 * HALF * float((np.abs(_f64(dW)) * D).sum()) + HALF * float(
        (np.abs(O.vocab_grad(d["X64"], d["W64"], np.ones(M), **d["lists"])[2]).T @ np.abs(d["X64"]) * D).sum())
    assert abs(lhs - rhs) <= M * e / h + h * h / 6 * 8 * M * dz ** 3 + slack


@pytest.mark.parametrize("which", ["dX", "dW"])
@pytest.mark.parametrize("M", [20, 280])
def test_one_gradient_only(which, M):
    for L in (0, 3):
        _both(_inputs(M, 520, 72, L=L, seed=M), need_dX=which == "dX", need_dW=which == "dW")


def test_pieces_of_the_vocabulary():
    """Enough tokens that the gradient's workspace holds 4352 ids at a time: three pieces, the last
    of 296 ids, lists across their borders, half of the tokens masked."""
    M, N, K, L = 30000, 9000, 64, 7
    r = torch.Generator().manual_seed(4)
    X = torch.randn((M, K), generator=r).to(torch.bfloat16).to(DEV)
    W = (torch.randn((N, K), generator=r) * 0.25).to(torch.bfloat16).to(DEV)
    index = torch.randint(0, N, (M, L), generator=r)
    index[:, 1] = 4351 + torch.arange(M) % 3
    index[torch.rand(M, generator=r) < 0.5] = -1
    index = index.to(DEV)
    teacher = torch.randn((M, L), generator=r).to(DEV)
    loss, lse = B.vocab_distill(X, W, index, teacher)
    g = torch.randn(M, generator=r).to(DEV)
    dX, dW = B.vocab_distill_grad(X, W, index, teacher, lse, g)
    live = index[:, 0] >= 0
    x, w = X.double() * live[:, None], W.double()
    z = x @ w.T
    l64 = torch.logsumexp(z, 1)
    e = (x.abs() @ w.abs().T).amax(1) * (2 * K + 2) * U + (4 * z.abs().amax(1) + 4 * l64.abs() + 616) * U
    assert torch.all(((lse.double() - l64).abs() <= e)[live]) and not bool(lse[~live].any())
    p = torch.softmax(teacher.double(), 1)
    want = (p * (p.log() - torch.gather(z, 1, index.clamp(0)) + l64[:, None])).sum(1)
    e_p = 2 * (3 * 2 * 6 + L + 10) * U
    assert torch.all(((loss.double() - want).abs() <= 3 * e + 40 * (e_p + 8 * U))[live])
    a = (g.double() * live)[:, None]
    q = torch.exp(z - lse.double()[:, None])
    t = torch.zeros_like(q).scatter_add_(1, index.clamp(0), p)
    G, mag = (q - t) * a, (q + t) * a.abs()
    eG = HALF * G.abs() + mag * (e[:, None] + e_p + 8 * U)
    for got, want, bound, big, n in ((dX, G @ w, eG @ w.abs(), G.abs() @ w.abs(), N),
                                     (dW, G.T @ x, eG.T @ x.abs(), G.abs().T @ x.abs(), M)):
        lim = bound + (big + bound) * (2 * n + 2) * U
        assert torch.all((got.double() - want).abs() <= lim + HALF * (want.abs() + lim) + TINY)
    assert not bool(dX[~live].any())


def test_offsets_past_32_bits():
    """A head of 2.5 G elements, rows in a wider buffer: the last ids' logits and gradients."""
    N, K, ld, M = 600_000, 4096, 4160, 5
    W = torch.zeros((N, ld), dtype=torch.bfloat16, device=DEV)[:, :K]
    r = torch.Generator().manual_seed(1)
    X = torch.randn((M, K), generator=r).to(torch.bfloat16).to(DEV)
    rows = torch.tensor([0, 1, 255, 256, 300_000, 524_287, 524_288, N - 2, N - 1], device=DEV)
    vals = (torch.randn((len(rows), K), generator=r) * 0.05).to(torch.bfloat16).to(DEV)
    W[rows] = vals
    target = torch.tensor([0, 524_288, N - 1, N - 2, 300_000], device=DEV)
    logp, lse = B.vocab_logp(X, W, target)
    z = X.double() @ vals.double().T
    l64 = torch.log(torch.exp(z).sum(1) + (N - len(rows)))
    pick = torch.stack([z[i, (rows == target[i]).nonzero()[0, 0]] for i in range(M)])
    e = (X.double().abs() @ vals.double().abs().T).amax(1) * (2 * K + 2) * U + (4 * z.abs().amax(1) + 616 + 20) * U
    assert torch.all((lse.double() - l64).abs() <= e) and torch.all((logp.double() - pick + l64).abs() <= 2 * e)
    g = torch.tensor([1.0, -2.0, 0.5, 1.0, 3.0], device=DEV)
    dX, dW = B.vocab_logp_grad(X, W, target, lse, g)
    G = -torch.exp(z - lse.double()[:, None])
    G[torch.arange(M, device=DEV), [int((rows == t).nonzero()[0, 0]) for t in target]] += 1.0
    G *= g.double()[:, None]
    eG = HALF * G.abs() + 2 * g.double().abs()[:, None] * e[:, None]
    want, lim = G @ vals.double(), eG @ vals.double().abs()
    lim = lim + G.abs() @ vals.double().abs() * (2 * N + 2) * U
    assert torch.all((dX.double() - want).abs() <= lim + HALF * (want.abs() + lim))
    want, lim = G.T @ X.double(), eG.T @ X.double().abs()
    assert torch.all((dW[rows].double() - want).abs() <= lim + HALF * (want.abs() + lim) + 1e-6 * lim)
    rest = dW[400_000]
    want = -(g.double() * torch.exp(-lse.double())) @ X.double()
    mag = (g.double().abs() * torch.exp(-lse.double())) @ X.double().abs()
    assert torch.all((rest.double() - want).abs() <= mag * (HALF + 2 * float(e.max()) + 20 * U) + HALF * want.abs())


def test_more_tiles_than_one_launch_takes():
    """2^20 tokens of 2^18 + 77 ids: 2^22 tiles and more, several launches of the logits, lists at their
    borders. X and W repeat a few rows, so float64 needs each pair once."""
    M, N, K, nx, nw = 1 << 20, (1 << 18) + 77, 8, 16, 61
    r = torch.Generator().manual_seed(9)
    xs = torch.randn((nx, K), generator=r).to(torch.bfloat16).to(DEV)
    wr = torch.randn((nw, K), generator=r).to(torch.bfloat16).to(DEV)
    X, W = xs[torch.arange(M, device=DEV) % nx], wr[torch.arange(N, device=DEV) % nw]
    per = (1 << 21) // (M // 256) * 256  # ids of a launch
    edges = torch.tensor([0, per - 1, per, 2 * per - 1, 2 * per, N - 1, N, -1], device=DEV)
    target = edges[(torch.arange(M, device=DEV) // nx) % len(edges)]
    logp, lse = B.vocab_logp(X, W, target)
    z = xs.double() @ wr.double().T
    count = torch.bincount(torch.arange(N, device=DEV) % nw, minlength=nw).double()
    l64 = torch.log((torch.exp(z) * count).sum(1))
    live = (target >= 0) & (target < N)
    zmax = z.abs().amax(1)
    e = (xs.double().abs() @ wr.double().abs().T).amax(1) * (2 * K + 2) * U + (4 * zmax + 616 + l64.abs()) * U
    which = torch.arange(M, device=DEV) % nx
    assert torch.all(((lse.double() - l64[which]).abs() <= e[which])[live]) and not bool(lse[~live].any())
    want = z[which, target.clamp(0, N - 1) % nw] - l64[which]
    assert torch.all(((logp.double() - want).abs() <= 2 * e[which] + want.abs() * U)[live])
    assert not bool(logp[~live].any())


def test_gradient_past_32_bits_of_tokens():
    """700000 tokens: a piece's G (4096 ids each) is 5.7 GB, its last rows lie past 2^31 elements; some
    live tokens at the end, the others masked or of no gradient."""
    M, N, K = 700_000, 5000, 16
    r = torch.Generator().manual_seed(2)
    X = torch.randn((M, K), generator=r).to(torch.bfloat16).to(DEV)
    W = (torch.randn((N, K), generator=r) * 0.5).to(torch.bfloat16).to(DEV)
    target = torch.randint(0, N, (M,), generator=r).to(DEV)
    g = torch.zeros(M, device=DEV)
    rows = torch.tensor([0, 5, 349_999, 524_288, M - 3, M - 2, M - 1], device=DEV)
    g[rows] = torch.randn(len(rows), generator=r).to(DEV)
    logp, lse = B.vocab_logp(X, W, target)
    dX, dW = B.vocab_logp_grad(X, W, target, lse, g)
    x, w = X[rows].double(), W.double()
    z = x @ w.T
    G = -torch.exp(z - lse[rows].double()[:, None])
    G[torch.arange(len(rows), device=DEV), target[rows]] += 1.0
    G *= g[rows].double()[:, None]
    e = (x.abs() @ w.abs().T).amax(1) * (2 * K + 2) * U + (8 * z.abs().amax(1) + 616) * U
    eG = HALF * G.abs() + (G.abs() + g[rows].double().abs()[:, None] * torch.exp(z - lse[rows].double()[:, None])) \
        * (e[:, None] + 16 * U) * 2
    lim = eG @ w.abs() + (G.abs() @ w.abs()) * (2 * N + 2) * U
    want = G @ w
    assert torch.all((dX[rows].double() - want).abs() <= lim + HALF * (want.abs() + lim) + TINY)
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[rows] = False
    assert not bool(dX[keep].any())
    # dW: M terms of which all but seven are zero (no rounding)
    lim = eG.T @ x.abs() + (G.abs().T @ x.abs()) * 20 * U
    want = G.T @ x
    assert torch.all((dW.double() - want).abs() <= lim + HALF * (want.abs() + lim) + TINY)


def test_given_outputs_and_strides():
    """Outputs of the caller: rows between which others lie are left as they were."""
    d = _inputs(150, 400, 72, seed=6)
    value, lse, g, dX, dW = _both(d)
    out = [torch.full((n + 1, 96), 7.0, dtype=torch.bfloat16, device=DEV) for n in (150, 400)]
    dX2, dW2 = _backward(d, lse, g, dX=out[0][:150, 8:80], dW=out[1][:400, 8:80])
    assert torch.equal(dX2, dX) and torch.equal(dW2, dW)
    for o in out:
        assert bool((o[:, :8] == 7).all()) and bool((o[:, 80:] == 7).all()) and bool((o[-1] == 7).all())
    v = torch.full((150,), 3.0, device=DEV)
    l2 = torch.full((150,), 3.0, device=DEV)
    assert _forward(d, logp=v, lse=l2)[0] is v and torch.equal(v, value) and torch.equal(l2, lse)


def test_no_tokens():
    X = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    W = torch.ones((300, 64), dtype=torch.bfloat16, device=DEV)
    t = torch.empty(0, dtype=torch.int64, device=DEV)
    f = torch.empty(0, device=DEV)
    logp, lse = B.vocab_logp(X, W, t)
    assert logp.numel() == 0 and lse.numel() == 0
    dX, dW = B.vocab_logp_grad(X, W, t, f, f, dW=torch.full_like(W, 3.0))
    assert dX.shape == (0, 64) and not bool(dW.any())


def test_same_bits_every_time_and_on_another_stream():
    for L in (0, 20):
        d = _inputs(270, 3000, 264, L=L, seed=L, masked=np.arange(270) % 5 == 0)
        value, lse, g, dX, dW = _both(d)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            v2, l2 = _forward(d)
            x2, w2 = _backward(d, lse, g)
        v3, l3 = _forward(d)  # at the same time, each call with a workspace of its own
        x3, w3 = _backward(d, lse, g)
        torch.cuda.synchronize()
        for a, b, c in ((value, v2, v3), (dX, x2, x3), (dW, w2, w3)):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_captured_chain_from_hidden_states_and_back():
    """logp -> ACR / TIS loss -> gradient as a trainer runs them, captured in one graph, replayed on
    new contents with eager work in between; two graphs captured side by side."""
    M, N, K = 200, 1500, 136
    batches = []
    for seed in (1, 2, 3):
        d = _inputs(M, N, K, seed=seed, masked=np.arange(M) % 4 == seed % 4)
        r = np.random.default_rng(seed)
        d["prox"] = torch.from_numpy(-np.abs(r.standard_normal(M)).astype(np.float32) - 7).to(DEV)
        d["beh"] = (d["prox"] + torch.from_numpy(r.standard_normal(M).astype(np.float32) * 0.1).to(DEV)).contiguous()
        d["adv"] = torch.from_numpy(r.standard_normal(M).astype(np.float32)).to(DEV)
        batches.append(d)

    def chain(X, W, target, prox, beh, adv):
        logp, lse = B.vocab_logp(X, W, target, scale=1.1)
        mask = (target >= 0).logical_and(target < N).to(torch.uint8)
        loss, grad, sums = B.acr_tis_loss(logp, prox, beh, adv, mask, I.ACR_EPS, I.ACR_C)
        dX, dW = B.vocab_logp_grad(X, W, target, lse, grad, scale=1.1)
        return logp, loss, sums, dX, dW

    def args(d):
        return [d["X"], d["W"], d["dev"]["target"], d["prox"], d["beh"], d["adv"]]

    want = [[t.clone() for t in chain(*args(d))] for d in batches]
    torch.cuda.synchronize()
    static = [[t.clone() for t in args(batches[0])] for _ in range(2)]
    graphs, outs = [], []
    for st in static:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            chain(*st)
        torch.cuda.current_stream().wait_stream(s)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(chain(*st))
        graphs.append(gr)
    for k in range(6):
        for i, gr in enumerate(graphs):
            for dst, src in zip(static[i], args(batches[(k + i) % 3])):
                dst.copy_(src)
            gr.replay()
        eager = chain(*args(batches[k % 3]))
        torch.cuda.synchronize()
        for i in range(2):
            for a, b in zip(outs[i], want[(k + i) % 3]):
                assert torch.equal(a, b), (k, i)
        for a, b in zip(eager, want[k % 3]):
            assert torch.equal(a, b)
    # and what the chain computes: the loss's gradient through the oracle
    d = batches[0]
    d["scale"] = 1.1
    logp, lse = B.vocab_logp(d["X"], d["W"], d["dev"]["target"], scale=1.1)
    _check_forward(d, (logp, lse))
    mask = (~d["masked"]).astype(np.uint8)
    _, g, _ = B.acr_tis_loss(logp, d["prox"], d["beh"], d["adv"], torch.from_numpy(mask).to(DEV), I.ACR_EPS, I.ACR_C)
    _check_backward(d, lse, g, want[0][3], want[0][4])


def test_captured_calls_follow_the_masks():
    """One graph of the calls, replayed with all, some, few and none of the tokens counting: what the
    kernels choose for those that count is chosen anew each time."""
    M, N, K, L = 700, 20001, 136, 5
    r = torch.Generator().manual_seed(12)
    X = torch.randn((M, K), generator=r).to(torch.bfloat16).to(DEV)
    W = (torch.randn((N, K), generator=r) * 0.1).to(torch.bfloat16).to(DEV)
    g = torch.randn(M, generator=r).to(DEV)
    teacher = torch.randn((M, L), generator=r).to(DEV)
    ids = torch.randint(0, N, (M, L), generator=r)
    masks = [torch.rand(M, generator=r) < keep for keep in (1.0, 0.5, 0.2, 0.1, 0.0)]
    lists = [torch.where(m[:, None], ids, torch.tensor(-1)).to(DEV) for m in masks]

    def calls(index, target):
        logp, lse = B.vocab_logp(X, W, target)
        grads = B.vocab_logp_grad(X, W, target, lse, g)
        loss, dlse = B.vocab_distill(X, W, index, teacher)
        return (logp, lse, loss, dlse) + tuple(grads) + tuple(B.vocab_distill_grad(X, W, index, teacher, dlse, g))

    want = [[t.clone() for t in calls(i, i[:, 0].contiguous())] for i in lists]
    index, target = lists[0].clone(), lists[0][:, 0].contiguous()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls(index, target)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = calls(index, target)
    for k in (0, 3, 1, 4, 2, 0, 4, 3):
        index.copy_(lists[k])
        target.copy_(lists[k][:, 0])
        graph.replay()
        eager = calls(lists[k], lists[k][:, 0].contiguous())
        torch.cuda.synchronize()
        for i, (a, b, c) in enumerate(zip(out, want[k], eager)):
            assert torch.equal(a, b) and torch.equal(c, b), (k, i)
    assert not bool(want[4][4].any()) and not bool(want[4][5].any())


def test_refused_calls():
    d = _inputs(4, 100, 64, L=3, seed=1)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    f = torch.zeros(4, device=DEV)
    X, W, ix, te = d["X"], d["W"], d["dev"]["index"], d["dev"]["teacher"]
    bad = [
        lambda: B.vocab_logp(X.float(), W, t), lambda: B.vocab_logp(X, W.half(), t),
        lambda: B.vocab_logp(X, W[:, :56], t), lambda: B.vocab_logp(X, W, t.int()),
        lambda: B.vocab_logp(X, W, t[:3]), lambda: B.vocab_logp(X, W, t.cpu()),
        lambda: B.vocab_logp(X[:, ::2], W[:, ::2], t), lambda: B.vocab_logp(X, W, t, lse=f.double()),
        lambda: B.vocab_logp_grad(X, W, t, f, f[:2]), lambda: B.vocab_logp_grad(X, W, t, f.half(), f),
        lambda: B.vocab_logp_grad(X, W, t, f, f, need_dX=False, need_dW=False),
        lambda: B.vocab_logp_grad(X, W, t, f, f, dX=X.float()),
        lambda: B.vocab_distill(X, W, ix[:, :2], te), lambda: B.vocab_distill(X, W, ix.int(), te),
        lambda: B.vocab_distill(X, W, ix, te.half()), lambda: B.vocab_distill(X, W, ix, te, teacher_lse=f[:1]),
        lambda: B.vocab_distill_grad(X, W, ix, te, f, f[:1]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(i)
    lib = [
        lambda: B.vocab_logp(X[:, :60], W[:, :60], t), lambda: B.vocab_logp(X, W, t, scale=0.0),
        lambda: B.vocab_logp(X, W, t, scale=float("nan")), lambda: B.vocab_logp(X, W[:0], t),
        lambda: B.vocab_logp(X, W, t, ws=torch.empty(8, dtype=torch.uint8, device=DEV)),
        lambda: B.vocab_logp(X[:, 4:60], W[:, 4:60], t),
        lambda: B.vocab_logp(X[:1].expand(4, 64), W, t),  # rows that are one row
    ]
    for i, call in enumerate(lib):
        with pytest.raises(B.QRError):
            call()
            raise AssertionError(i)
