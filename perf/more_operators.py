"""Losses over a large vocabulary, as cases to measure: from hidden states and the head's
weights to per-token losses and back, without the logits ever being held whole.

Four operators of a trainer beside the per-token policy loss:

  logp          log-probability of one id per token (the negative cross entropy) and the log of
                the softmax's sum, from hidden states X [M, K] and the head W [N, K]
  logp_grad     its gradient: dX and dW from d loss / d logp
  distill       divergence from a teacher of whom the top logits are known: per token a list of
                ids with the teacher's logits
  distill_grad  its gradient

`run` computes them in plain torch operations in 32 bits, in pieces of the vocabulary, or, with
`own` set, by the framework's kernels. `exact` computes them in 64 bits.

With logits z = scale X W^T: lse = log sum exp z; logp = z[target] - lse; a target outside
[0, N) masks the token (0, no gradient). A list's entries have p = softmax of the teacher's
scaled logits over the list, or exp(scale * logit - teacher_lse) with the teacher's own sum;
loss = sum p (log p - (z[id] - lse)); ids outside [0, N) are no entries, and a token without
entries is masked.
"""

import torch

own = False

DEV = "cuda"
HIDDEN_7B = 3584
HIDDEN_32B = 5120


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------

def listed():
    h, H = HIDDEN_7B, HIDDEN_32B
    return [
        # one sampled token scored by the full-precision actor: latency
        dict(name="logp_1", op="logp", M=1, N=32768, K=h, masked=0.0, scale=1.0, pad=0),
        # a short response, odd vocabulary, hidden states inside wider rows
        dict(name="logp_257_odd", op="logp", M=257, N=100003, K=h, masked=0.0, scale=1.0, pad=64),
        # a training micro-batch of the wide model
        dict(name="logp_4096_wide", op="logp", M=4096, N=131072, K=H, masked=0.0, scale=1.0, pad=0),
        # the update from one short response
        dict(name="logp_grad_33", op="logp_grad", M=33, N=32768, K=h, masked=0.0, scale=1.0, pad=0, dw=True),
        # a padded batch, half of it prompts and padding, sampled at temperature 0.8
        dict(name="logp_grad_2048_padded", op="logp_grad", M=2048, N=131072, K=h, masked=0.5, scale=1.25,
             pad=0, dw=True),
        # a training micro-batch
        dict(name="logp_grad_4096", op="logp_grad", M=4096, N=131072, K=h, masked=0.0, scale=1.0, pad=0,
             dw=True),
        # a few tokens against a teacher's twenty best ids, as a server returns them
        dict(name="distill_48_top20", op="distill", M=48, N=32768, K=h, L=20, teacher="fp32", full=True,
             masked=0.0, scale=1.0, pad=0),
        # a micro-batch against 64 ids, teacher logits in bf16, some lists shorter
        dict(name="distill_4096_top64", op="distill", M=4096, N=131072, K=h, L=64, teacher="bf16", full=False,
             masked=0.1, scale=1.0, pad=0),
        # an odd number of tokens through a frozen head: the hidden states' gradient only
        dict(name="distill_grad_301_frozen", op="distill_grad", M=301, N=100003, K=h, L=20, teacher="fp32",
             full=True, masked=0.0, scale=1.0, pad=0, dw=False),
        # a micro-batch of the wide model at temperature 2
        dict(name="distill_grad_2048_wide", op="distill_grad", M=2048, N=131072, K=H, L=64, teacher="bf16",
             full=False, masked=0.1, scale=0.5, pad=0, dw=True),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread over the logarithm."""
    v = lo * (hi / lo) ** rng.random()
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["logp", "logp_grad", "logp_grad", "distill", "distill_grad", "distill_grad"])
    c = dict(op=op, M=_log(rng, 1, 4096), N=_log(rng, 700, 131072), K=_log(rng, 64, HIDDEN_32B, 8),
             masked=rng.choice([0.0, 0.0, 0.1, 0.5, 0.9]), scale=rng.choice([1.0, 1.0, 1.25, 0.5]),
             pad=8 * rng.choice([0, 0, 1, 9]))
    if op.startswith("distill"):
        c.update(L=_log(rng, 1, 128), teacher=rng.choice(["fp32", "bf16"]), full=rng.random() < 0.5)
    if op.endswith("grad"):
        c.update(dw=rng.random() < 0.75)
        # no more work than the largest listed gradient
        while c["M"] * c["N"] * c["K"] > 4096 * 131072 * HIDDEN_7B:
            c["M"] //= 2
    return c


def _valid(c):
    """Tokens that are not masked: an exact count, whichever the seed takes."""
    return c["M"] - int(c["M"] * c["masked"])


def work(case):
    c = case
    M, N, K, V = c["M"], c["N"], c["K"], _valid(case)
    lists = M * (c["L"] * (8 + (4 if c["teacher"] == "fp32" else 2)) + 4 * c["full"]) if "L" in c else 8 * M
    if not c["op"].endswith("grad"):
        return {"bytes": 2 * (V + N) * K + lists + 8 * M, "flops": 2 * V * N * K}
    out = 2 * M * K + (2 * N * K if c["dw"] else 0)
    return {"bytes": 2 * (V + N) * K + lists + 8 * M + out, "flops": (6 if c["dw"] else 4) * V * N * K}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------

def _head(N, K, g):
    """Weights N(0, 0.02^2) in bf16, as a head's are."""
    W = torch.empty((N, K), dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 26) // K)
    for r in range(0, N, step):
        n = min(step, N - r)
        W[r:r + n] = torch.randn((n, K), device=DEV, generator=g) * 0.02
    return W


def _hidden(M, K, W, ids, g, pad):
    """Hidden states N(0, 1), turned towards the head's row of `ids` so that its logit rises by
    up to 12: tokens from undecided to certain. Rows `pad` elements longer in memory."""
    x = torch.randn((M, K), device=DEV, generator=g)
    lift = 12.0 * torch.rand((M, 1), device=DEV, generator=g)
    w = W[ids].float()
    x += lift * w / w.square().sum(dim=1, keepdim=True)
    buf = torch.zeros((M, K + pad), dtype=torch.bfloat16, device=DEV)
    buf[:, :K] = x
    return buf[:, :K]


def _lse32(X, W, scale):
    out = torch.full((X.shape[0],), -float("inf"), device=DEV)
    x = X.float() * scale
    for n in range(0, W.shape[0], 16384):
        out = torch.logaddexp(out, torch.logsumexp(x @ W[n:n + 16384].float().t(), dim=1))
    return out


def prepare(case, seed):
    c = case
    M, N, K = c["M"], c["N"], c["K"]
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    W = _head(N, K, g)
    # ids: small ones (common words) are frequent
    u = torch.rand(M, device=DEV, generator=g)
    ids = (N * u ** 3).long().clamp(max=N - 1)
    out = torch.randperm(M, device=DEV, generator=g)[: M - _valid(c)]
    st = dict(case=c, W=W, X=_hidden(M, K, W, ids, g, c["pad"]))
    if "L" in c:
        # distinct ids, the first of them the likely one; the teacher's logits fall along the list
        L = c["L"]
        step = 1 + (torch.rand((M, 1), device=DEV, generator=g) * max(N // L - 1, 1) * 0.999).long()
        index = (ids[:, None] + step * torch.arange(L, device=DEV)) % N
        s = torch.randn((M, L), device=DEV, generator=g) * 2.0
        s = s.sort(dim=1, descending=True).values + 8.0
        s[:, 0] += 4.0 * torch.rand(M, device=DEV, generator=g)
        short = torch.rand((M, 1), device=DEV, generator=g)
        if not c["full"]:  # lists of unequal length, padded with -1
            n = L - (short * 0.3 * L).long()
            index[torch.arange(L, device=DEV) >= n] = -1
        index[out] = -1
        st["index"] = index
        st["teacher"] = s if c["teacher"] == "fp32" else s.to(torch.bfloat16)
        st["teacher_lse"] = None
        if c["full"]:  # the list holds most of the teacher's probability, not all of it
            rest = torch.rand(M, device=DEV, generator=g) * 0.3
            st["teacher_lse"] = torch.logsumexp(s * c["scale"], dim=1) + rest
    else:
        target = ids.clone()
        target[out] = -100
        st["target"] = target
    if c["op"].endswith("grad"):
        st["lse"] = _lse32(st["X"], W, c["scale"])
        st["g"] = torch.randn(M, device=DEV, generator=g) / _valid(c)
    return st


# ----------------------------------------------------------------------------
# Plain forms
# ----------------------------------------------------------------------------

PIECE = 16384


def _lists(st, c):
    """(ids [M, L], probabilities [M, L], tokens that count [M]) of either operator."""
    N = c["N"]
    if "L" not in c:
        ids = st["target"][:, None]
        ok = (ids >= 0) & (ids < N)
        return ids, ok.float(), ok.any(dim=1)
    ids = st["index"]
    ok = (ids >= 0) & (ids < N)
    s = st["teacher"].float() * c["scale"]
    if st["teacher_lse"] is not None:
        p = torch.where(ok, torch.exp(s - st["teacher_lse"][:, None]), torch.zeros_like(s))
        return ids, p, ok.any(dim=1)
    s = torch.where(ok, s, torch.full_like(s, -float("inf")))
    top = s.amax(dim=1, keepdim=True)
    e = torch.exp(s - torch.where(ok.any(dim=1, keepdim=True), top, torch.zeros_like(top)))
    total = e.sum(dim=1, keepdim=True)
    return ids, e / torch.where(total > 0, total, torch.ones_like(total)), ok.any(dim=1)


def _plain_forward(st, c):
    ids, p, ok = _lists(st, c)
    M, N = c["M"], c["N"]
    rows = ok.nonzero()[:, 0]
    x = st["X"][rows].float()
    m = torch.full((rows.numel(),), -float("inf"), device=DEV)
    s = torch.zeros_like(m)
    z = torch.zeros((rows.numel(), ids.shape[1]), device=DEV)
    i = ids[rows]
    for n in range(0, N, PIECE):
        l = (x @ st["W"][n:n + PIECE].float().t()) * c["scale"]
        top = torch.maximum(m, l.amax(dim=1))
        s = s * torch.exp(m - top) + torch.exp(l - top[:, None]).sum(dim=1)
        m = top
        here = (i >= n) & (i < n + l.shape[1])
        z = torch.where(here, l.gather(1, (i - n).clamp(0, l.shape[1] - 1)), z)
    lse = m + torch.log(s)
    q = p[rows]
    full = torch.zeros(M, device=DEV)
    if "L" in c:
        t = torch.where(q > 0, q * (torch.log(q.clamp(min=1e-38)) - (z - lse[:, None])), torch.zeros_like(q))
        loss = full.index_copy(0, rows, t.sum(dim=1))
    else:
        loss = full.index_copy(0, rows, z[:, 0] - lse)
    return loss, full.index_copy(0, rows, lse)


def _plain_grad(st, c):
    ids, p, ok = _lists(st, c)
    M, N = c["M"], c["N"]
    rows = ok.nonzero()[:, 0]
    x = st["X"][rows].float()
    a = st["g"][rows] * c["scale"] * (1.0 if "L" in c else -1.0)
    i, q, lse = ids[rows], p[rows], st["lse"][rows]
    P = q.sum(dim=1)
    dx = torch.zeros_like(x)
    dW = torch.empty((N, c["K"]), dtype=torch.bfloat16, device=DEV) if c["dw"] else None
    for n in range(0, N, PIECE):
        w = st["W"][n:n + PIECE].float()
        G = torch.exp((x @ w.t()) * c["scale"] - lse[:, None]) * P[:, None]
        here = (i >= n) & (i < n + w.shape[0])
        G.scatter_add_(1, (i - n).clamp(0, w.shape[0] - 1), torch.where(here, -q, torch.zeros_like(q)))
        G *= a[:, None]
        dx += G @ w
        if dW is not None:
            dW[n:n + PIECE] = G.t() @ x
    dX = torch.zeros((M, c["K"]), dtype=torch.bfloat16, device=DEV)
    dX[rows] = dx.to(torch.bfloat16)
    return (dX, dW) if c["dw"] else dX


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------

def run(state):
    st, c = state, state["case"]
    if own:
        from w8a8_gemm_rl_amd import binding as B

        if c["op"] == "logp":
            return B.vocab_logp(st["X"], st["W"], st["target"], scale=c["scale"])
        if c["op"] == "distill":
            return B.vocab_distill(st["X"], st["W"], st["index"], st["teacher"], scale=c["scale"],
                                   teacher_lse=st["teacher_lse"])
        if c["op"] == "logp_grad":
            dX, dW = B.vocab_logp_grad(st["X"], st["W"], st["target"], st["lse"], st["g"], scale=c["scale"],
                                       need_dW=c["dw"])
        else:
            dX, dW = B.vocab_distill_grad(st["X"], st["W"], st["index"], st["teacher"], st["lse"], st["g"],
                                          scale=c["scale"], teacher_lse=st["teacher_lse"],
                                          need_dW=c["dw"])
        return (dX, dW) if c["dw"] else dX
    return _plain_grad(st, c) if c["op"].endswith("grad") else _plain_forward(st, c)


# ----------------------------------------------------------------------------
# 64 bits
# ----------------------------------------------------------------------------

def exact(case, seed):
    """From the definitions in float64, a block of tokens at a time, the whole vocabulary at
    once; gradients as the softmax minus the targets, built densely."""
    c, st = case, prepare(case, seed)
    M, N, K = c["M"], c["N"], c["K"]
    W, X = st["W"].double(), st["X"].double()
    f64 = dict(dtype=torch.float64, device=DEV)
    value, total = torch.zeros(M, **f64), torch.zeros(M, **f64)
    grad = c["op"].endswith("grad")
    dX = torch.zeros((M, K), **f64)
    dW = torch.zeros((N, K), **f64) if grad and c["dw"] else None
    for t0 in range(0, M, 1024):
        t = slice(t0, min(t0 + 1024, M))
        ids = st["index"][t] if "L" in c else st["target"][t].view(-1, 1)
        entry = torch.logical_and(ids.ge(0), ids.lt(N))
        live = entry.any(1)
        if "L" not in c:
            logq = torch.zeros(ids.shape, **f64)
        else:
            y = st["teacher"][t].double().mul(c["scale"]).masked_fill(~entry, -float("inf"))
            norm = torch.logsumexp(y, 1) if st["teacher_lse"] is None else st["teacher_lse"][t].double()
            logq = y - norm.where(live, torch.zeros_like(norm)).unsqueeze(1)
        prob = logq.exp().masked_fill(~entry, 0.0)
        z = torch.matmul(X[t], W.T).mul_(c["scale"])
        if not grad:
            lse = torch.logsumexp(z, 1)
            zi = torch.gather(z, 1, ids.clamp(0, N - 1)) - lse.unsqueeze(1)
            if "L" in c:
                term = prob * (logq.masked_fill(prob == 0, 0.0) - zi)
            else:
                term = zi.masked_fill(~entry, 0.0)
            value[t] = term.sum(1).masked_fill(~live, 0.0)
            total[t] = lse.masked_fill(~live, 0.0)
            continue
        sign = 1.0 if "L" in c else -1.0  # of the softmax's part
        target = torch.zeros_like(z).scatter_add_(1, ids.clamp(0, N - 1), prob)
        z.sub_(st["lse"][t].double().unsqueeze(1)).exp_().mul_(prob.sum(1, keepdim=True)).sub_(target)
        del target
        z.mul_((st["g"][t].double() * c["scale"] * sign).masked_fill(~live, 0.0).unsqueeze(1))
        dX[t] = torch.matmul(z, W)
        if dW is not None:
            dW.addmm_(z.T, X[t])
        del z
    if not grad:
        return value, total
    return (dX, dW) if c["dw"] else dX
