"""A language model's step with the library's operators from end to end: embedding, dropout, norm
and head, forward and backward, and the sharded optimizer step of its unit."""

import pytest
import torch

import model_ends_cases as E
from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

BF = torch.bfloat16
VOCAB, DIM, ROWS, P = 700, 136, 260, 0.2


def weights(seed):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return [(0.05 * r(VOCAB, DIM)).cuda(), (1 + 0.1 * r(DIM)).cuda(), (0.05 * r(VOCAB, DIM)).cuda()]


class Step:
    """Forward and backward of embedding -> dropout -> norm -> head on one rank's tokens; the
    gradients go into a row of the unit. The buffers are made once."""

    def __init__(self, lib, shapes, tied):
        new = lambda *s, t=BF: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
        self.lib, self.tied = lib, tied
        self.row = new(sum(torch.Size(s).numel() for s in shapes))
        self.grads = [g.view(s) for g, s in zip(self.row.split([torch.Size(s).numel() for s in shapes]), shapes)]
        self.h0, self.h1, self.h2, self.d1, self.d2 = (new(ROWS, DIM) for _ in range(5))
        self.rstd, self.loss = new(ROWS, t=torch.float32), new(1, t=torch.float32)
        self.counter = torch.zeros(1, dtype=torch.int64, device="cuda")
        byte = lambda n: new(n, t=torch.uint8)  # noqa: E731
        head = torch.empty(VOCAB, DIM, dtype=BF, device="meta")
        self.work = [byte(lib.linear_cross_entropy_workspace(self.h2, head)),
                     byte(lib.rms_norm_backward_workspace(ROWS, DIM)), byte(lib.embedding_backward_workspace(ROWS, VOCAB, DIM))]

    def __call__(self, params, tokens, targets, offset):
        lib, (embed, norm, head) = self.lib, (params + params[:1])[:3]
        de, dn, dh = (self.grads + self.grads[:1])[:3]
        drop = dict(seed=99, offset=offset, counter=self.counter)
        lib.embedding(tokens, embed, self.h0, scale=DIM ** 0.5)
        lib.dropout(self.h0, self.h1, P, **drop)
        lib.rms_norm(self.h1, norm, self.h2, rstd=self.rstd)
        lib.linear_cross_entropy(self.h2, head, targets, self.loss, self.work[0], dhidden=self.d2, dweight=dh)
        lib.rms_norm_backward(self.d2, self.h1, norm, self.rstd, self.d1, dn, self.work[1])
        lib.dropout(self.d1, self.d1, P, **drop)
        lib.embedding_backward(tokens, self.d1, de, self.work[2], scale=DIM ** 0.5, accumulate=self.tied)


def batch(seed):
    gen = torch.Generator().manual_seed(seed)
    tokens = torch.randint(0, VOCAB, (ROWS,), generator=gen).square() // VOCAB
    targets = torch.where(torch.rand(ROWS, generator=gen) < 0.2, -100, torch.randint(0, VOCAB, (ROWS,), generator=gen))
    tokens[5] = -1
    return tokens.cuda(), targets.cuda()


def loss_64(params, tokens, targets, offset):
    """The same in 64 bits, from the bf16 parameters, without any rounding between."""
    embed, norm, head = (params + params[:1])[:3]
    ok = (tokens >= 0)[:, None]
    h = torch.where(ok, embed[tokens.clamp_min(0)] * DIM ** 0.5, torch.zeros((), dtype=torch.float64, device="cuda"))
    below = round(P * 65536)
    keep = torch.from_numpy((E.dropout_bits(ROWS, DIM, 99, offset) >= below)).cuda()
    h = h * keep * (65536 / (65536 - below))
    h = h / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6) * norm
    z = h @ head.T
    counted = targets >= 0
    return (torch.logsumexp(z, 1) - z.gather(1, targets.clamp_min(0)[:, None])[:, 0])[counted].mean()


@pytest.mark.parametrize("tied", [False, True])
def test_gradients(lib, tied):
    """Every parameter's gradient against autograd in 64 bits."""
    params = [p.to(BF) for p in weights(1)][:2 if tied else 3]
    tokens, targets = batch(2)
    step = Step(lib, [p.shape for p in params], tied)
    step(params, tokens, targets, 40)
    torch.cuda.synchronize()
    leaves = [p.double().requires_grad_() for p in params]
    want = loss_64(leaves, tokens, targets, 40)
    want.backward()
    assert abs(float(step.loss) - want.item()) <= 0.01 * want.item()
    for g, p in zip(step.grads, leaves):
        # bf16 activations and gradients on the way, a handful of roundings each, in the 2-norm
        assert float((g.double() - p.grad).norm()) <= 6 * E.BF16 * float(p.grad.norm())


def test_captured_step(lib):
    """The step in a graph: each replay, with other tokens, parameters and dropout, is the eager one's bits."""
    params = [p.to(BF) for p in weights(3)]
    step = Step(lib, [p.shape for p in params], False)
    tokens, targets = batch(4)
    step(params, tokens, targets, 7)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(params, tokens, targets, 7)
    for i in range(4):
        for a, b in zip((tokens, targets), batch(10 + i)):
            a.copy_(b)
        params[2].mul_(1.1)
        step.counter.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        got = step.row.clone(), step.loss.clone()
        step.row.zero_()
        step(params, tokens, targets, 7)
        torch.cuda.synchronize()
        assert E.same_bits(got[0], step.row) and E.same_bits(got[1], step.loss)


def test_two_streams(lib):
    """Two ranks' steps at once, each on a stream and with buffers of its own."""
    params = [p.to(BF) for p in weights(5)]
    alone, both = [], [Step(lib, [p.shape for p in params], False) for _ in range(2)]
    for i, s in enumerate(both):
        s(params, *batch(20 + i), 50 + i)
        torch.cuda.synchronize()
        alone.append((s.row.clone(), s.loss.clone()))
        s.row.zero_()
    data, streams = [batch(20 + i) for i in range(2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for i, (s, st) in enumerate(zip(both, streams)):
            with torch.cuda.stream(st):
                s(params, *data[i], 50 + i)
    torch.cuda.synchronize()
    for s, (row, loss) in zip(both, alone):
        assert E.same_bits(s.row, row) and E.same_bits(s.loss, loss)


def test_sharded_training_step(lib):
    """The ranks' gradient rows through the sharded AdamW step, against the same steps made of
    64-bit gradients: the parameters' change has the right direction and size."""
    F = 2
    masters = weights(7)
    shapes = [p.shape for p in masters]
    units = [lib.Unit(shapes, F, r) for r in range(F)]
    step = Step(lib, shapes, False)
    shards = []
    for u in units:
        p = torch.empty(u.S, device="cuda")
        lib.flatten_pad(u, masters, p)
        shards.append((p, torch.zeros_like(p), torch.zeros_like(p), p.to(BF)))
    params = [torch.empty(s, dtype=BF, device="cuda") for s in shapes]
    lib.cast_unflatten(units[0], [s[3] for s in shards], params)
    rows, want = [], 0.0
    leaves = [p.double().requires_grad_() for p in params]
    for r in range(F):
        tokens, targets = batch(30 + r)
        step(params, tokens, targets, 60 + r)
        rows.append(step.row.clone())
        loss_64(leaves, tokens, targets, 60 + r).backward()
    for u, (p, m, v, w) in zip(units, shards):
        lib.reduce_adamw_shard(u, rows, p, m, v, w, lib.AdamWHparams(lr=1e-3, weight_decay=0.0), 1)
    torch.cuda.synchronize()
    flat = torch.cat([q.grad.reshape(-1) for q in leaves]) / F
    got = torch.cat([m[:u.shard_valid] for u, (_, m, _, _) in zip(units, shards)]).double() * 10    # 1 - beta1
    assert float((got - flat).norm()) <= 6 * E.BF16 * float(flat.norm())
