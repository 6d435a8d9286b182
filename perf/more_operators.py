"""Cases of the operators at the two ends of a language model's training step: the output
layer with its cross-entropy taken in pieces of the vocabulary, so that the logits are never
kept (tp_vocab_linear_ce_fwd, tp_vocab_linear_ce_bwd), and the scaled embedding lookup with
its gradient by sorted tokens (tp_vocab_embed_scaled_fwd, tp_vocab_embed_scaled_bwd).

`own` False computes the operators with elementary torch operations, True with the library's
entry points. E is (vocab, h), shared by both ends; ids and targets are int32, and those
outside [0, vocab) (here -1) take part in nothing, but the mean over the M rows counts them.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIGMA = 0.02  # of the embedding's values, as everywhere in the benchmark


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the small GPT's loss (its 4 x 32 tokens, vocabulary, width and two shards): latency
        dict(name="ce-fwd-gpt", op="ce-fwd", dtype="f32", M=128, v=256, h=128, N=2, skip=0.0),
        # the loss of a training batch: the cross-entropy benchmark's rows, vocabulary and shards
        # at the GQA block's width
        dict(name="ce-fwd-batch", op="ce-fwd", dtype="bf16", M=8192, v=50304, h=2048, N=8, skip=0.02),
        # the log-likelihood of a few tokens under a vocabulary that is not padded
        dict(name="ce-fwd-few", op="ce-fwd", dtype="bf16", M=37, v=50257, h=4096, N=1, skip=0.0),
        # the gradients of the small GPT's loss
        dict(name="ce-bwd-gpt", op="ce-bwd", dtype="f32", M=128, v=256, h=128, N=2, skip=0.0),
        # the gradients of a ragged micro-batch, unpadded vocabulary, a tenth of the rows padding
        dict(name="ce-bwd-ragged", op="ce-bwd", dtype="bf16", M=1003, v=50257, h=1032, N=1, skip=0.1),
        # the gradients of the training batch above
        dict(name="ce-bwd-batch", op="ce-bwd", dtype="bf16", M=8192, v=50304, h=2048, N=8, skip=0.02),
        # the same at the GELU benchmark's width: the largest
        dict(name="ce-bwd-large", op="ce-bwd", dtype="bf16", M=8192, v=50304, h=4096, N=8, skip=0.02),
        # the input rows of a decode step
        dict(name="embed-fwd-decode", op="embed-fwd", dtype="bf16", M=64, v=50304, h=8192, N=4, skip=0.0),
        # the input rows of a training batch
        dict(name="embed-fwd-batch", op="embed-fwd", dtype="bf16", M=8192, v=50304, h=4096, N=8, skip=0.02),
        # the embedding's gradient of that batch: many rows without a token, some with hundreds
        dict(name="embed-bwd-batch", op="embed-bwd", dtype="bf16", M=8192, v=50304, h=2048, N=8, skip=0.02),
        # that of many long sequences: the most frequent token comes four thousand times
        dict(name="embed-bwd-long", op="embed-bwd", dtype="bf16", M=65536, v=50257, h=4096, N=1, skip=0.01),
        # both ends of the small GPT with the shared embedding: lookup, loss, gradients, and the
        # lookup's gradient added to the output layer's
        dict(name="tied-step-gpt", op="step", dtype="f32", M=128, v=256, h=128, N=2, skip=0.0),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["ce-fwd", "ce-fwd", "ce-bwd", "ce-bwd", "ce-bwd", "embed-fwd", "embed-bwd",
                     "embed-bwd", "step"])
    N = rng.choice([1, 1, 2, 3, 4, 8, 16])
    case = dict(op=op, N=N, skip=rng.choice([0.0, 0.0, 0.02, 0.3]))
    if op.startswith("embed"):
        case.update(dtype=rng.choice(["bf16", "bf16", "f32"]), M=_log(rng, 1, 30000),
                    v=N * _log(rng, 1, 50304 // N))
        h = _log(rng, 1, 4096)
        return dict(case, h=h if rng.random() < 0.4 else -(-h // 8) * 8)
    if op == "step" or rng.random() < 0.25:
        return dict(case, dtype="f32", M=_log(rng, 1, 512), v=N * _log(rng, 1, 2048 // N),
                    h=_log(rng, 1, 256))
    return dict(case, dtype="bf16", M=_log(rng, 1, 8192), v=N * _log(rng, 1, 50304 // N),
                h=8 * _log(rng, 1, 2048 // 8))


def _tokens(gen, M, v, skip):
    """Token ids whose frequency falls with the id as 1 / (id + 1), the share `skip` of them -1."""
    u = torch.rand(M, generator=gen, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(v + 1.0)) - 1.0).long().clamp(0, v - 1)
    drop = torch.rand(M, generator=gen, device="cuda") < skip
    return torch.where(drop, torch.full_like(ids, -1), ids).to(torch.int32)


def prepare(case, seed):
    M, v, h = case["M"], case["v"], case["h"]
    dt = DTYPES[case["dtype"]]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.float32)
    st = dict(case, ids=_tokens(gen, M, v, case["skip"]), factor=math.sqrt(h), scale=1.0 / M)
    if case["op"] != "embed-bwd":
        st["E"] = (rnd(v, h) * SIGMA).to(dt)
    if case["op"] in ("ce-fwd", "ce-bwd", "step"):
        st["targets"] = _tokens(gen, M, v, case["skip"])
    if case["op"] in ("ce-fwd", "ce-bwd"):
        # a normalised row that points, more or less, to its target: losses from none to log v
        at = st["targets"].long().clamp(min=0)
        pull = torch.rand(M, 1, generator=gen, device="cuda") * min(1.0, 16.0 / (SIGMA * h))
        st["x"] = (rnd(M, h) + pull * st["E"].float()[at] / SIGMA).to(dt)
    if case["op"] == "ce-bwd":  # the forward pass keeps one number of each row
        st["lse"] = torch.logsumexp(st["x"].float() @ st["E"].float().T, dim=1)
    if case["op"] == "embed-bwd":
        st["dx"] = (rnd(M, h) * SIGMA).to(dt)
    if own:
        _buffers(st, case, dt)
    return st


def _buffers(st, case, dt):
    """What a user's program allocates once: outputs and workspaces."""
    from attention_gemms_gb300 import tpmlp as L
    op, M, v, h, N = case["op"], case["M"], case["v"], case["h"], case["N"]
    e = lambda *s, t=dt: torch.empty(s, dtype=t, device="cuda")
    f32 = torch.float32
    st["dt"] = L.DType.BF16 if dt == torch.bfloat16 else L.DType.F32
    size = 0
    if op in ("ce-fwd", "step"):
        st.update(lse=e(M, t=f32), row_loss=e(M, t=f32), shard_loss=e(N, t=f32), loss=e(1, t=f32))
        size = max(size, L.tp_vocab_linear_ce_workspace_size(1, M, v, h, N, st["dt"]))
    if op in ("ce-bwd", "step"):
        st.update(dx=e(M, h), dE=e(v, h))
        size = max(size, L.tp_vocab_linear_ce_workspace_size(0, M, v, h, N, st["dt"]))
    if op in ("embed-fwd", "step"):
        st.update(x=e(M, h))
    if op == "embed-bwd":
        st.update(dE=e(v, h))
    if op in ("embed-bwd", "step"):
        size = max(size, L.tp_vocab_embed_scaled_workspace_size(M, v, h, st["dt"]))
    st["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ the operators

def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    from attention_gemms_gb300 import tpmlp as L
    op, M, v, h, N, dt, ws = (st[k] for k in ("op", "M", "v", "h", "N", "dt", "ws"))
    if op in ("embed-fwd", "step"):
        L.tp_vocab_embed_scaled_fwd(st["ids"], st["E"], st["x"], M, v, h, N, st["factor"], dt)
    if op in ("ce-fwd", "step"):
        L.tp_vocab_linear_ce_fwd(st["x"], st["E"], st["targets"], st["lse"], st["row_loss"],
                                 st["shard_loss"], st["loss"], M, v, h, N, dt, ws, ws.numel())
    if op in ("ce-bwd", "step"):
        L.tp_vocab_linear_ce_bwd(st["x"], st["E"], st["targets"], st["lse"], st["dx"], st["dE"], M,
                                 v, h, N, st["scale"], dt, ws, ws.numel())
    if op in ("embed-bwd", "step"):
        L.tp_vocab_embed_scaled_bwd(st["ids"], st["dx"], st["dE"], M, v, h, N, st["factor"],
                                    op == "step", dt, ws, ws.numel())
    if op == "embed-fwd":
        return st["x"]
    if op == "embed-bwd":
        return st["dE"]
    if op == "ce-fwd":
        return st["loss"], st["lse"], st["row_loss"], st["shard_loss"]
    if op == "ce-bwd":
        return st["dx"], st["dE"]
    return st["loss"], st["shard_loss"], st["dx"], st["dE"]


def _lookup(ids, E, factor):
    rows = E.float()[ids.long().clamp(min=0)] * factor
    return torch.where((ids >= 0)[:, None], rows, torch.zeros_like(rows))


def _loss(x, E, targets, N):
    """(loss, lse, loss of each row, loss of each vocabulary shard) and the logits, in 32 bits."""
    v = E.shape[0]
    logits = x.float() @ E.float().T
    m = logits.amax(1, keepdim=True)
    lse = (m + torch.log(torch.exp(logits - m).sum(1, keepdim=True))).squeeze(1)
    at = logits.gather(1, targets.long().clamp(min=0)[:, None]).squeeze(1)
    rows = torch.where(targets >= 0, lse - at, torch.zeros_like(lse))
    shard = torch.div(targets.long(), v // N, rounding_mode="floor")
    shards = torch.stack([torch.where(shard == i, rows, torch.zeros_like(rows)).sum()
                          for i in range(N)])
    return (shards.sum() / x.shape[0]).reshape(1), lse, rows, shards, logits


def _loss_grads(x, E, targets, lse, scale, logits=None):
    """(dx, dE) in 32 bits."""
    xf, Ef = x.float(), E.float()
    if logits is None:
        logits = xf @ Ef.T
    p = torch.exp(logits - lse[:, None])
    hit = torch.nonzero(targets >= 0).squeeze(1)
    p[hit, targets[hit].long()] -= 1.0
    p *= torch.where(targets >= 0, scale, 0.0)[:, None]
    return p @ Ef, p.T @ xf


def _lookup_grad(ids, dx, v, factor):
    """dE in 32 bits."""
    keep = torch.nonzero(ids >= 0).squeeze(1)
    dE = torch.zeros(v, dx.shape[1], device="cuda")
    dE.index_add_(0, ids[keep].long(), dx[keep].float())
    return dE * factor


def _plain(st):
    op, v, N, dt = st["op"], st["v"], st["N"], DTYPES[st["dtype"]]
    if op == "embed-fwd":
        return _lookup(st["ids"], st["E"], st["factor"]).to(dt)
    if op == "embed-bwd":
        return _lookup_grad(st["ids"], st["dx"], v, st["factor"]).to(dt)
    if op == "ce-fwd":
        return _loss(st["x"], st["E"], st["targets"], N)[:4]
    if op == "ce-bwd":
        dx, dE = _loss_grads(st["x"], st["E"], st["targets"], st["lse"], st["scale"])
        return dx.to(dt), dE.to(dt)
    x = _lookup(st["ids"], st["E"], st["factor"])
    loss, lse, _, shards, logits = _loss(x, st["E"], st["targets"], N)
    dx, dE = _loss_grads(x, st["E"], st["targets"], lse, st["scale"], logits)
    dE = dE + _lookup_grad(st["ids"], dx, v, st["factor"])
    return loss, shards, dx.to(dt), dE.to(dt)


# ------------------------------------------------------------------ least work and exact values

def _distinct(M, v, skip):
    """How many different ids _tokens is expected to give."""
    n, top = M * (1.0 - skip), math.log(v + 1.0)
    return sum(1.0 - (1.0 - math.log((i + 2.0) / (i + 1.0)) / top * (1.0 - 1e-12)) ** n
               for i in range(v))


def work(case):
    M, v, h, N = case["M"], case["v"], case["h"], case["N"]
    e = 2 if case["dtype"] == "bf16" else 4
    seen = round(_distinct(M, v, case["skip"])) if case["op"] == "embed-fwd" else 0
    ends = (M + v) * h * e  # x and E, or their gradients
    product = 2 * M * v * h
    fwd = dict(bytes=ends + 4 * M + 4 * (2 * M + N + 1), flops=product)
    # the logits again, and the two gradients' products
    bwd = dict(bytes=2 * ends + 8 * M, flops=3 * product)
    # the rows of E that occur are read; every row of its gradient is written
    lookup = dict(bytes=(seen + M) * h * e + 4 * M, flops=M * h)
    scatter = dict(bytes=ends + 4 * M, flops=M * h)
    parts = {"ce-fwd": [fwd], "ce-bwd": [bwd], "embed-fwd": [lookup], "embed-bwd": [scatter],
             "step": [dict(bytes=(2 * M + 2 * v) * h * e + 8 * M, flops=4 * product)]}[case["op"]]
    return {k: sum(p[k] for p in parts) for k in ("bytes", "flops")}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op, M, v, h, N = case["op"], case["M"], case["v"], case["h"], case["N"]
    if not op.startswith("embed") and 6.0 * M * v * h > 1.2e13:
        return None
    ids = st["ids"].long()
    live = ids >= 0
    f64 = dict(dtype=torch.float64, device="cuda")
    if op == "embed-bwd":
        dE = torch.zeros(v, h, **f64)
        # the tokens in the order of their ids, each id's rows added up by differences of a running sum
        order = torch.argsort(ids, stable=True)[int((~live).sum()):]
        for c in range(0, h, 256):
            run_ = torch.cumsum(st["dx"][order, c:c + 256].double(), 0)
            run_ = torch.cat([torch.zeros(1, run_.shape[1], **f64), run_])
            end = torch.searchsorted(ids[order], torch.arange(v, device="cuda"), right=True)
            start = torch.searchsorted(ids[order], torch.arange(v, device="cuda"))
            dE[:, c:c + 256] = (run_[end] - run_[start]) * st["factor"]
        return dE
    E = st["E"].double()
    if op == "embed-fwd":
        x = torch.zeros(M, h, **f64)
        x[live] = E.index_select(0, ids[live]) * st["factor"]
        return x
    if op == "step":
        x = torch.zeros(M, h, **f64)
        x[live] = E.index_select(0, ids[live]) * st["factor"]
    else:
        x = st["x"].double()
    t = st["targets"].long()
    own_rows = t >= 0
    logits = torch.matmul(x, E.transpose(0, 1))
    lse = st["lse"].double() if op == "ce-bwd" else torch.logsumexp(logits, 1)
    if op != "ce-bwd":
        rows = torch.zeros(M, **f64)
        rows[own_rows] = lse[own_rows] - logits[own_rows, t[own_rows]]
        shards = torch.zeros(N, **f64).index_add_(0, t[own_rows] // (v // N), rows[own_rows])
        loss = rows.sum().reshape(1) / M
        if op == "ce-fwd":
            return loss, lse, rows, shards
    # (softmax - one_hot) / M on the rows with a target, as two terms of each gradient
    weight = own_rows.double() / M
    q = logits.sub_(lse[:, None]).exp_().mul_(weight[:, None])
    at = E.new_zeros(M, h)
    at[own_rows] = E[t[own_rows]]
    dx = q @ E - weight[:, None] * at
    dE = q.transpose(0, 1) @ x
    dE.index_add_(0, t[own_rows], x[own_rows] * (-1.0 / M))
    if op == "ce-bwd":
        return dx, dE
    dE.index_add_(0, ids[live], dx[live] * st["factor"])
    return loss, shards, dx, dE
