"""float64 torch forms of the two ends of a training step -- the output layer with its
cross-entropy, the scaled embedding lookup -- on any device, and how far a right kernel may be
from them: every bound counts roundings (half a step: bf16 2^-8, fp32 2^-24) term by term."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def has_target(targets, v):
    return (targets >= 0) & (targets < v)


def ce_fwd(x, E, targets, N):
    """loss (1), lse (M), row_loss (M), shard_loss (N)."""
    x, E = x.double(), E.double()
    M, v = x.shape[0], E.shape[0]
    logits = x @ E.T
    lse = torch.logsumexp(logits, 1)
    own = has_target(targets, v)
    rows = torch.zeros_like(lse)
    t = targets[own].long()
    rows[own] = lse[own] - logits[own, t]
    shards = torch.stack([rows[own][t // (v // N) == i].sum() for i in range(N)])
    return rows.sum().reshape(1) / M, lse, rows, shards


def ce_grad_logits(x, E, targets, lse, scale):
    """(p, q): softmax from lse, and the gradient by the logits."""
    x, E = x.double(), E.double()
    p = torch.exp(x @ E.T - lse.double()[:, None])
    own = has_target(targets, E.shape[0])
    hot = torch.zeros_like(p)
    r = torch.nonzero(own).squeeze(1)
    hot[r, targets[r].long()] = 1.0
    return p, (p - hot) * own[:, None] * scale


def ce_bwd(x, E, targets, lse, scale):
    """dx (M, h), dE (v, h)."""
    _, q = ce_grad_logits(x, E, targets, lse, scale)
    return q @ E.double(), q.T @ x.double()


def logit_error(x, E):
    """Of an fp32 dot product of h exact products, whatever its order: h roundings of partial sums
    (2^-23 each: an adder may cut instead of round), of at most sum |x||E|; per row, the largest."""
    h = x.shape[1]
    return (x.double().abs() @ E.double().abs().T).amax(1) * h * 2.0 ** -23


def ce_fwd_bounds(x, E, targets, N):
    """Of lse and row_loss (M each), shard_loss (N), loss (1).
    lse = ln 2 (m + log2 S): the logits' error; m, and each exponent l log2(e) - m, of one or two
    roundings of numbers not above max|l| log2(e) (2^-23 max|l| together); each power 2^-22; S of 16
    terms, 16 chunks, the slots and 32 warps, 2^-24 relative each, exponents of the joins as above;
    the logarithm and its product 2^-23 |lse| and 2^-22."""
    v, M = E.shape[0], x.shape[0]
    logits = x.double() @ E.double().T
    top = logits.abs().amax(1)
    e = logit_error(x, E)
    slots = -(-v // 64)
    lse = torch.logsumexp(logits, 1).abs()
    b = e + 2.0 ** -21 * top + 2.0 ** -23 * lse + 2.0 ** -24 * (64 + slots) + 2.0 ** -20
    rows = torch.where(has_target(targets, v), b + e + 2.0 ** -24 * (lse + top), torch.zeros_like(b))
    r = ce_fwd(x, E, targets, N)
    # fp32 sums over the rows: at most M roundings of at most the sum of |loss|
    total = (M + 2) * 2.0 ** -24 * r[2].abs().sum() + rows.sum()
    return b, rows, total.expand(N), total / M + 2.0 ** -23 * r[0].abs()


def ce_bwd_bounds(x, E, targets, lse, scale):
    """Of dx and dE. p = 2^(l log2(e) - lse log2(e)): relative error of the logit, of exponents of
    2^-22 of max(|l|, |lse|) and of the power, 2^-22; q = (p - hot) scale rounded to the element type
    (two more fp32 roundings); the products' fp32 sums as logit_error; the result's rounding."""
    M, v = x.shape[0], E.shape[0]
    p, q = ce_grad_logits(x, E, targets, lse, scale)
    own = has_target(targets, v)
    top = torch.maximum((x.double() @ E.double().T).abs().amax(1), lse.double().abs())
    rel = logit_error(x, E) + 2.0 ** -22 * top + 2.0 ** -22
    half = HALF[x.dtype] if x.dtype == torch.bfloat16 else 0.0
    dq = (p * rel[:, None] * abs(scale) * 1.01 * own[:, None] + q.abs() * (half + 2.0 ** -22) +
          2.0 ** -125 * abs(scale))
    xd, Ed = x.double().abs(), E.double().abs()
    dx, dE = ce_bwd(x, E, targets, lse, scale)
    aq = q.abs() + dq
    out = HALF[x.dtype] * 1.01
    bx = dq @ Ed + (aq @ Ed) * (v + 64) * 2.0 ** -23
    bE = dq.T @ xd + (aq.T @ xd) * (M + 64) * 2.0 ** -23
    return bx + (dx.abs() + bx) * out, bE + (dE.abs() + bE) * out


def embed_fwd(ids, E, scale):
    out = torch.zeros(ids.numel(), E.shape[1], dtype=torch.float64, device=E.device)
    own = has_target(ids, E.shape[0])
    out[own] = E.double()[ids[own].long()] * scale
    return out


def embed_bwd(ids, dx, v, scale, dE=None):
    """(gradient, sum of |dx| per element, tokens per row)."""
    own = has_target(ids, v)
    at = ids[own].long()
    z = lambda: torch.zeros(v, dx.shape[1], dtype=torch.float64, device=dx.device)
    g = z().index_add_(0, at, dx[own].double()) * scale
    a = z().index_add_(0, at, dx[own].double().abs())
    n = torch.bincount(at, minlength=v)
    if dE is not None:
        g = torch.where((n > 0)[:, None], g + dE.double(), dE.double())
    return g, a, n


def embed_bwd_bound(g, a, n, scale, dtype):
    """n + 2 roundings of partial sums in fp32 (sums, the factor, the sum with what was there),
    the result's rounding."""
    b = (n[:, None] + 2.0) * 2.0 ** -24 * (a * abs(scale) + g.abs()) * 1.01
    return b + (g.abs() + b) * HALF[dtype] * 1.01
