"""The two ends of a training step together and as a program uses them: a tied language model without
layers between them, trained; steps replayed from a CUDA graph; several streams; expired waits."""
import threading

import pytest
import torch

from attention_gemms_gb300 import tpmlp as T
from tests import ends_ref as R
from tests.test_gpu_ends import (BF, DT, F32, ce_case, gen, guarded, poison, rnd, run_bwd, run_fwd,
                                 tokens, within)

pytestmark = pytest.mark.gpu


class Tied:
    """x = LN(scale E[ids]), loss = CE(x E^T, targets): the buffers and the calls of a step's forward
    and backward pass, every gradient of E included."""

    def __init__(self, M, v, h, N, dt, seed):
        g = gen(seed)
        self.M, self.v, self.h, self.N, self.dt, self.scale = M, v, h, N, dt, h ** 0.5
        self.E = rnd(g, v, h, sigma=0.05, dt=dt)
        self.gamma = 1.0 + 0.1 * torch.randn(h, generator=g, device="cuda")
        self.beta = 0.1 * torch.randn(h, generator=g, device="cuda")
        self.ids, self.targets = tokens(g, M, v, "zipf"), tokens(g, M, v)
        e = lambda *s, t=dt: torch.full(s, float("nan"), dtype=t, device="cuda")
        self.x0, self.x, self.dx, self.dx0, self.dE = e(M, h), e(M, h), e(M, h), e(M, h), e(v, h)
        self.mean, self.rstd, self.lse, self.rows = (e(M, t=F32) for _ in range(4))
        self.shards, self.loss, self.dg, self.db = e(N, t=F32), e(1, t=F32), e(h, t=F32), e(h, t=F32)
        d = DT[dt]
        self.n = max(T.tp_vocab_linear_ce_workspace_size(1, M, v, h, N, d),
                     T.tp_vocab_linear_ce_workspace_size(0, M, v, h, N, d),
                     T.tp_vocab_embed_scaled_workspace_size(M, v, h, d),
                     T.tp_workspace_size(T.Op.LAYERNORM_BWD, M, h, 0, 1, d, T.Act.NONE, T.Reduce.SPLITK))
        self.ws = poison(self.n)

    def step(self, stream=None):
        M, v, h, N, d, ws, n = self.M, self.v, self.h, self.N, DT[self.dt], self.ws, self.n
        T.tp_vocab_embed_scaled_fwd(self.ids, self.E, self.x0, M, v, h, N, self.scale, d, stream)
        T.tp_layernorm_fwd(self.x0, self.gamma, self.beta, self.x, self.mean, self.rstd, M, h, 1e-5,
                           d, stream)
        T.tp_vocab_linear_ce_fwd(self.x, self.E, self.targets, self.lse, self.rows, self.shards,
                                 self.loss, M, v, h, N, d, ws, n, stream)
        T.tp_vocab_linear_ce_bwd(self.x, self.E, self.targets, self.lse, self.dx, self.dE, M, v, h, N,
                                 1.0 / M, d, ws, n, stream)
        T.tp_layernorm_bwd(self.x0, self.gamma, self.mean, self.rstd, self.dx, None, self.dx0, self.dg,
                           self.db, M, h, d, ws, n, stream)
        T.tp_vocab_embed_scaled_bwd(self.ids, self.dx0, self.dE, M, v, h, N, self.scale, True, d, ws, n,
                                    stream)

    def outputs(self):
        return [t.clone() for t in (self.loss, self.shards, self.dE, self.dg, self.db)]

    def reference(self):
        """The same in float64 by autograd: loss, dE, dgamma, dbeta."""
        E = self.E.double().requires_grad_()
        gamma, beta = (t.double().requires_grad_() for t in (self.gamma, self.beta))
        x0 = E[self.ids.long()] * self.scale
        x = torch.nn.functional.layer_norm(x0, (self.h,), gamma, beta, 1e-5)
        own = R.has_target(self.targets, self.v)
        rows = torch.logsumexp(x @ E.T, 1)[own] - (x[own] * E[self.targets[own].long()]).sum(1)
        loss = rows.sum() / self.M
        loss.backward()
        return loss.detach(), E.grad, gamma.grad, beta.grad


@pytest.mark.parametrize("M,v,h,N", [(128, 256, 128, 2), (300, 1003, 72, 1), (2000, 5000, 256, 8)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_tied_ends_against_autograd(M, v, h, N, dt):
    s = Tied(M, v, h, N, dt, 3)
    s.step()
    torch.cuda.synchronize()
    assert T.tp_check_status() == 0
    loss, dE, dg, db = s.reference()
    # bf16: each of x0, x, q, dx, dx0 and dE rounds once on the way, 2^-8 of its own size at the most
    # each; relative to the largest entry, six such roundings; fp32: sums of up to M + v + h terms
    tol = 6 * 2.0 ** -8 if dt == BF else 4e-5
    assert abs(s.loss.item() - loss.item()) <= tol * loss.item()
    for got, want in ((s.dE, dE), (s.dg, dg), (s.db, db)):
        assert (got.double() - want).abs().max() <= tol * want.abs().max()


def test_tied_gradient_by_differences():
    """The loss's change along its own gradient, in fp32."""
    s = Tied(200, 300, 64, 3, F32, 4)
    s.step()
    torch.cuda.synchronize()
    g, E0 = s.dE.clone(), s.E.clone()
    norm2 = float((g.double() ** 2).sum())
    f = []
    eps = 0.02 / norm2 ** 0.5
    for sign in (1, -1):
        s.E.copy_(E0 + sign * eps * g)
        s.step()
        torch.cuda.synchronize()
        f.append(s.loss.item())
    # central difference: error eps^2 |third derivative| / 6 of 4e-4 parts, the losses' 1e-6 / eps
    assert abs((f[0] - f[1]) / (2 * eps) - norm2) <= 2e-2 * norm2


@pytest.mark.parametrize("dt", [BF, F32])
def test_steps_replay_from_a_graph(dt):
    """One captured step, replayed with other tokens, against eager calls, bit for bit; AdamW moves E
    between the replays in fp32."""
    s = Tied(500, 700, 128, 2, dt, 5)
    s.step()
    torch.cuda.synchronize()
    m, v2, grad = (torch.zeros(s.v * s.h, device="cuda") for _ in range(3))
    count = torch.zeros(1, dtype=torch.int32, device="cuda")

    def whole():
        s.step()
        if dt == F32:
            T.tp_train_step_advance(count, None, None, 0)
            T.tp_adamw_step_device(s.E, s.dE, m, v2, s.v * s.h, count, 1e-3, 0.9, 0.999, 1e-8, 0.01)

    E0 = s.E.clone()

    def play(run):
        s.E.copy_(E0)
        for t in (m, v2, count):
            t.zero_()
        got = []
        for k in range(3):
            g = gen(100 + k)
            s.ids.copy_(tokens(g, s.M, s.v, ("zipf", "same", "none")[k]))
            s.targets.copy_(tokens(g, s.M, s.v))
            run()
            torch.cuda.synchronize()
            got += s.outputs() + [s.E.clone()]
        return got

    want = play(whole)
    graph = torch.cuda.CUDAGraph()
    s.E.copy_(E0)
    with torch.cuda.graph(graph):
        whole()
    got = play(graph.replay)
    assert T.tp_check_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_graphs_with_one_workspace():
    """Graphs of two models that share a workspace, replayed in turn on one stream."""
    a, b = Tied(300, 500, 64, 1, BF, 6), Tied(90, 2000, 128, 4, BF, 7)
    for s in (a, b):
        s.step()
    torch.cuda.synchronize()
    want = [a.outputs(), b.outputs()]
    n = max(a.n, b.n)
    a.ws = b.ws = poison(n)
    graphs = []
    for s in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.step()
    for _ in range(3):
        for t in (a.dE, b.dE, a.loss, b.loss):
            t.fill_(float("nan"))
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        assert all(torch.equal(x, y) for x, y in zip(s.outputs(), w))


def test_calls_from_threads_on_their_own_streams():
    cases = [Tied(300, 1500, 128, 3, BF, 10), Tied(64, 3000, 64, 1, BF, 11),
             Tied(257, 400, 72, 2, F32, 12), Tied(1000, 900, 256, 4, BF, 13)]
    for s in cases:
        s.step()
    torch.cuda.synchronize()
    want = [s.outputs() for s in cases]
    errors = []

    def work(s):
        try:
            stream = torch.cuda.Stream()
            for _ in range(10):
                s.step(stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and T.tp_check_status() == 0
    for s, w in zip(cases, want):
        assert all(torch.equal(x, y) for x, y in zip(s.outputs(), w))


@pytest.mark.parametrize("M,v,h", [(40, 900, 128), (200, 300, 64), (1200, 5000, 320), (600, 9000, 2048)])
def test_expired_waits_are_reported(M, v, h):
    """Every tile form of the cross-entropy's products gives up in time, and the next call is right."""
    x, E, t = ce_case(M, v, h, BF)
    good = run_fwd(x, E, t, 1)
    gx, gE = run_bwd(x, E, t, good[1].clone(), 1.0 / M)
    d, lse = T.DType.BF16, good[1].clone()
    n = max(T.tp_vocab_linear_ce_workspace_size(f, M, v, h, 1, d) for f in (0, 1))
    ws, out = poison(n), [guarded(k) for k in (M, M, 1, 1)]
    dx, dE = guarded(M * h, BF), guarded(v * h, BF)
    T.tp_set_wait_timeout_ns(2_000_000)
    T.tp_debug_inject_wait_fault(1)
    try:
        T.tp_vocab_linear_ce_fwd(x, E, t, *out, M, v, h, 1, d, ws, n)
        assert T.tp_check_status() == T.Status.TIMEOUT
        T.tp_vocab_linear_ce_bwd(x, E, t, lse, dx, dE, M, v, h, 1, 1.0 / M, d, ws, n)
        assert T.tp_check_status() == T.Status.TIMEOUT
    finally:
        T.tp_debug_inject_wait_fault(0)
        T.tp_set_wait_timeout_ns(0)
    again = run_fwd(x, E, t, 1)
    assert all(torch.equal(a, b) for a, b in zip(again, good))
    hx, hE = run_bwd(x, E, t, lse, 1.0 / M)
    assert torch.equal(hx, gx) and torch.equal(hE, gE)


def test_results_do_not_depend_on_what_ran_before():
    """The same call after others, in workspaces of other contents: the same bits."""
    x, E, t = ce_case(130, 2000, 64, BF)
    a = run_fwd(x, E, t, 2)
    n = T.tp_vocab_linear_ce_workspace_size(1, 130, 2000, 64, 2, T.DType.BF16)
    for fill in (0, 1, 127):
        ws = torch.full((n + 256,), fill, dtype=torch.uint8, device="cuda")
        ws[n:] = 255
        b = run_fwd(x, E, t, 2, ws=ws)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    g = gen(2)
    ids, dx = tokens(g, 3000, 700), rnd(g, 3000, 64)
    k = T.tp_vocab_embed_scaled_workspace_size(3000, 700, 64, T.DType.BF16)
    outs = []
    for fill in (0, 1, 255):
        ws, dE = torch.full((k,), fill, dtype=torch.uint8, device="cuda"), guarded(700 * 64, BF)
        T.tp_vocab_embed_scaled_bwd(ids, dx, dE, 3000, 700, 64, 1, 1.0, 0, T.DType.BF16, ws, k)
        outs.append(dE)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("offset", [1, 2, 3])
def test_words_that_are_not_16_byte_aligned(offset):
    """ids, targets and per-row outputs begin anywhere on 4 bytes."""
    g = gen(offset)
    M, v, h = 1000, 600, 64
    x, E = rnd(g, M, h), rnd(g, v, h, sigma=0.1)
    pad = lambda t: torch.cat([torch.zeros(offset, dtype=t.dtype, device="cuda"), t])[offset:]
    t = pad(tokens(g, M, v))
    assert t.data_ptr() % 16 == 4 * offset
    n = T.tp_vocab_linear_ce_workspace_size(1, M, v, h, 1, T.DType.BF16)
    out = [torch.full((k + 8,), -1.0, device="cuda")[offset:offset + k] for k in (M, M, 1, 1)]
    T.tp_vocab_linear_ce_fwd(x, E, t, *out, M, v, h, 1, T.DType.BF16, poison(n), n)
    want = run_fwd(x, E, t.clone(), 1)
    assert torch.equal(out[0], want[1]) and torch.equal(out[1], want[2]) and torch.equal(out[3], want[0])
    dx = rnd(g, M, h)
    ids = pad(tokens(g, M, v, "zipf"))
    k = T.tp_vocab_embed_scaled_workspace_size(M, v, h, T.DType.BF16)
    dE, dE2 = guarded(v * h, BF), guarded(v * h, BF)
    T.tp_vocab_embed_scaled_bwd(ids, dx, dE, M, v, h, 1, 2.0, 0, T.DType.BF16, poison(k), k)
    T.tp_vocab_embed_scaled_bwd(ids.clone(), dx, dE2, M, v, h, 1, 2.0, 0, T.DType.BF16, poison(k), k)
    assert torch.equal(dE, dE2)
    y = guarded(M * h, BF)
    T.tp_vocab_embed_scaled_fwd(ids, E, y, M, v, h, 1, 2.0, T.DType.BF16)
    ref = R.embed_fwd(ids, E, 2.0)
    within(y[:M * h].view(M, h), ref, ref.abs() * 2.0 ** -8 * 1.01)


@pytest.mark.parametrize("M", [1300, 5000, 16400])
def test_many_calls_without_a_pause(M):
    """Kernels of more and of fewer CTAs than the SMs hold, one behind the other: every call ends, and
    the last is right."""
    v, h = 3000, 64
    x, E, t = ce_case(M, v, h, BF)
    d, n = T.DType.BF16, 0
    big = 300_001  # a sort of more CTAs than there are SMs
    for f in (0, 1):
        n = max(n, T.tp_vocab_linear_ce_workspace_size(f, M, v, h, 1, d))
    n = max(n, T.tp_vocab_embed_scaled_workspace_size(M, big, 8, d))
    ws = poison(n)
    out = [torch.empty(k, device="cuda") for k in (M, M, 1, 1)]
    dx, dE = torch.empty(M, h, dtype=BF, device="cuda"), torch.empty(v, h, dtype=BF, device="cuda")
    dB, g = torch.empty(big, 8, dtype=BF, device="cuda"), rnd(gen(1), M, 8)
    for _ in range(10):
        T.tp_vocab_linear_ce_fwd(x, E, t, *out, M, v, h, 1, d, ws, n)
    for _ in range(5):
        T.tp_vocab_linear_ce_fwd(x, E, t, *out, M, v, h, 1, d, ws, n)
        T.tp_vocab_linear_ce_bwd(x, E, t, out[0], dx, dE, M, v, h, 1, 1.0 / M, d, ws, n)
        T.tp_vocab_embed_scaled_bwd(t, g, dB, M, big, 8, 1, 1.0, 0, d, ws, n)
    torch.cuda.synchronize()
    assert T.tp_check_status() == 0
    want = run_fwd(x, E, t, 1)
    assert torch.equal(out[0], want[1]) and torch.equal(out[3], want[0])
    wx, wE = run_bwd(x, E, t, want[1].clone(), 1.0 / M)
    assert torch.equal(dx, wx) and torch.equal(dE, wE)


def test_few_rows_of_a_large_gradient_without_a_pause_and_replayed():
    """dE's own kernel of few rows between the GEMMs: back to back, and captured with new inputs."""
    M, v, h = 40, 40_000, 512
    d = T.DType.BF16
    x, E, t = ce_case(M, v, h, BF)
    lse = run_fwd(x, E, t, 1)[1].clone()
    n = T.tp_vocab_linear_ce_workspace_size(0, M, v, h, 1, d)
    ws = poison(n)
    dx, dE = torch.empty(M, h, dtype=BF, device="cuda"), torch.empty(v, h, dtype=BF, device="cuda")

    def step():
        T.tp_vocab_linear_ce_bwd(x, E, t, lse, dx, dE, M, v, h, 1, 1.0 / M, d, ws, n)

    for _ in range(50):
        step()
    torch.cuda.synchronize()
    assert T.tp_check_status() == 0
    wx, wE = run_bwd(x, E, t, lse, 1.0 / M)
    assert torch.equal(dx, wx) and torch.equal(dE, wE)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x2, _, t2 = ce_case(M, v, h, BF, seed=2)
    x.copy_(x2)
    t.copy_(t2)
    lse.copy_(run_fwd(x, E, t, 1)[1])
    dx.fill_(float("nan"))
    dE.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    wx, wE = run_bwd(x, E, t, lse, 1.0 / M)
    assert torch.equal(dx, wx) and torch.equal(dE, wE)
