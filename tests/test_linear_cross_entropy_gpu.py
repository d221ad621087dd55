"""The head's loss and its gradients against the formulas in 64 bits."""

import pytest
import torch

import model_ends_cases as E
from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

BF = torch.bfloat16
NAN, INF = float("nan"), float("inf")


def inputs(rows, vocab, dim, extra=0, shift=0, skip=0.0, seed=0, sure=6.0):
    gen = torch.Generator().manual_seed(seed)
    w = E.rows_of(vocab, dim, dim + extra, shift, BF, 0.05, seed + 1)
    t = torch.randint(0, vocab, (rows,), generator=gen)
    x = E.rows_of(rows, dim, dim + extra, shift, BF, 1.0, seed + 2)
    right = w.double().cpu()[t]
    more = sure * torch.rand(rows, 1, generator=gen) * right / right.square().sum(1, keepdim=True).clamp_min(1e-3)
    x.copy_((x.double().cpu() + more).to(BF))
    if skip:
        gone = torch.rand(rows, generator=gen) < skip
        t[gone] = torch.tensor([-100, -1, vocab, 2 ** 40])[torch.randint(0, 4, (int(gone.sum()),), generator=gen)]
    return x, w, t.cuda()


def call(lib, x, w, t, dx=None, dw=None, losses=None, piece=0, **kw):
    need = lib.linear_cross_entropy_workspace(x, w, dhidden=dx is not None, dweight=dw is not None, piece=piece)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out = torch.full((1,), NAN, device="cuda")
    lib.linear_cross_entropy(x, w, t, out, ws, losses=losses, dhidden=dx, dweight=dw, piece=piece, **kw)
    torch.cuda.synchronize()
    return out


def check(lib, x, w, t, extra=0, shift=0, piece=0, mean=True, scale=1.0, grads="both"):
    rows, dim = x.shape
    vocab = w.shape[0]
    dx = E.Guarded(rows, dim, dim + extra, shift, BF) if grads in ("both", "dhidden") else None
    dw = E.Guarded(vocab, dim, dim + extra, shift, BF) if grads in ("both", "dweight") else None
    each = E.Guarded(1, rows, rows, 0, torch.float32)
    out = call(lib, x, w, t, dx and dx.t, dw and dw.t, each.t[0], piece, reduction="mean" if mean else "sum", grad_scale=scale)
    want = E.loss(x, w, t, scale, mean)
    assert E.near(each.t[0], *want["losses"], E.F32)
    assert E.near(out, *want["loss"], E.F32)
    for g, name in ((dx, "dhidden"), (dw, "dweight")):
        if g is not None:
            assert E.near(g.t, *want[name], E.BF16), name
            assert g.intact()
    assert each.intact()
    return out, each.t[0], dx and dx.t, dw and dw.t


SIZES = [(1, 1, 1, 0, 0), (1, 2, 3, 0, 0), (3, 5, 7, 0, 0), (2, 300, 8, 0, 0), (16, 64, 64, 0, 0), (17, 65, 64, 0, 0),
         (64, 64, 64, 0, 0), (65, 129, 65, 0, 0), (33, 1000, 96, 8, 8), (130, 257, 130, 3, 1), (256, 256, 256, 0, 0),
         (257, 513, 260, 0, 0), (300, 2000, 1027, 73, 1), (512, 777, 64, 0, 0), (100, 4099, 200, 0, 0),
         (40, 130, 4104, 0, 0), (1, 5003, 512, 0, 0), (600, 1290, 520, 0, 0)]


@pytest.mark.parametrize("rows,vocab,dim,extra,shift", SIZES)
@pytest.mark.parametrize("skip", [0.0, 0.4])
def test_loss(lib, rows, vocab, dim, extra, shift, skip):
    x, w, t = inputs(rows, vocab, dim, extra, shift, skip)
    check(lib, x, w, t, extra, shift)


# enough for every tile: many rows and tokens, long rows, few rows and a long vocabulary, unaligned ones
@pytest.mark.parametrize("rows,vocab,dim,extra,shift,piece", [
    (4100, 4200, 136, 0, 0, 0), (2100, 2100, 4104, 0, 0, 0), (2100, 2100, 4104, 8, 0, 1100), (1500, 5003, 1027, 9, 1, 0),
    (5000, 300, 2056, 0, 0, 0), (300, 9001, 2050, 0, 0, 0), (64, 20000, 320, 0, 0, 0), (1300, 3000, 600, 0, 0, 0),
    (9000, 520, 72, 0, 0, 4000), (513, 30000, 520, 0, 8, 0)])
def test_larger(lib, rows, vocab, dim, extra, shift, piece):
    x, w, t = inputs(rows, vocab, dim, extra, shift, 0.1, seed=rows)
    check(lib, x, w, t, extra, shift, piece=piece)


def test_every_row_once(lib):
    """Values that no product rounds, so that every element has to be right: each row's softmax is
    one or zero, the gradients' sums are small whole numbers."""
    for rows, vocab, dim in ((700, 600, 512), (5000, 5100, 264), (2600, 640, 4096)):
        x, w = torch.zeros(rows, dim, dtype=BF, device="cuda"), torch.zeros(vocab, dim, dtype=BF, device="cuda")
        r, v = torch.arange(rows, device="cuda"), torch.arange(vocab, device="cuda")
        w[v, v % dim] = 256.0                       # logits of 0 and 65536
        x[r, (7 * r) % min(dim, vocab)] = 256.0
        best = (7 * r) % min(dim, vocab)
        t = torch.where(r % 3 == 0, -100, (best + 1 + r) % min(dim, vocab))
        if vocab > dim:                             # several of the vocabulary alike: the first only
            w[dim:] = 0.0
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        losses = torch.empty(rows, device="cuda")
        call(lib, x, w, t, dx, dw, losses, reduction="sum")
        miss = (t >= 0) & (t != best)
        assert torch.equal(losses, miss * 65536.0)
        want = torch.zeros(rows, dim, device="cuda")
        want[r[miss], best[miss]] = 256.0
        want[r[miss], t[miss]] = -256.0
        assert torch.equal(dx.float(), want)
        sums = torch.zeros(vocab, dim, device="cuda")
        sums.index_put_((best[miss], best[miss]), torch.tensor(256.0, device="cuda"), accumulate=True)
        sums.index_put_((t[miss], best[miss]), torch.tensor(-256.0, device="cuda"), accumulate=True)
        assert torch.equal(dw, sums.to(BF))


@pytest.mark.parametrize("grads", ["none", "dhidden", "dweight"])
@pytest.mark.parametrize("rows,vocab,dim", [(1, 700, 64), (19, 300, 100), (70, 129, 65), (300, 600, 264)])
def test_what_is_asked_for(lib, rows, vocab, dim, grads):
    """The same bits whichever outputs are wanted."""
    x, w, t = inputs(rows, vocab, dim, skip=0.2)
    full = check(lib, x, w, t, mean=False, scale=0.3)
    part = check(lib, x, w, t, mean=False, scale=0.3, grads=grads)
    for a, b in zip(full, part):
        assert b is None or E.same_bits(a, b)


@pytest.mark.parametrize("mean", [True, False])
@pytest.mark.parametrize("piece", [1, 64, 100, 256, 299, 300, 1000])
def test_pieces(lib, piece, mean):
    rows, vocab, dim = 300, 333, 136
    x, w, t = inputs(rows, vocab, dim, skip=0.3, seed=5)
    check(lib, x, w, t, piece=piece, mean=mean, scale=2.5)
    check(lib, x, w, t[torch.argsort((t < 0) | (t >= vocab), stable=True)], piece=piece, mean=mean)   # rows that count first


@pytest.mark.parametrize("piece", [0, 64])
def test_no_row_counts(lib, piece):
    x, w, t = inputs(130, 200, 72)
    x.fill_(NAN)
    for targets in (torch.full_like(t, -100), torch.full_like(t, 200)):
        for mean in ("mean", "sum"):
            dx, dw = torch.full_like(x, 7.0), torch.full_like(w, 7.0)
            losses = torch.full((130,), 7.0, device="cuda")
            out = call(lib, x, w, targets, dx, dw, losses, piece, reduction=mean)
            assert float(out) == 0 and not bool(torch.count_nonzero(dx)) and not bool(torch.count_nonzero(dw))
            assert not bool(torch.count_nonzero(losses))


def test_no_rows(lib):
    w = torch.randn(100, 64, device="cuda").to(BF)
    x, t = torch.empty(0, 64, dtype=BF, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    dx, dw = torch.empty_like(x), torch.full_like(w, 7.0)
    assert float(call(lib, x, w, t, dx, dw)) == 0
    assert not bool(torch.count_nonzero(dw))
    assert float(call(lib, x, w, t)) == 0


@pytest.mark.parametrize("piece", [0, 64])
def test_what_rows_that_do_not_count_hold(lib, piece):
    """NaN and infinities in rows without a target, in the gaps between rows and past the last
    column change nothing."""
    rows, vocab, dim = 150, 290, 100
    x, w, t = inputs(rows, vocab, dim, 28, 4, skip=0.3, seed=7)       # the gaps hold NaN
    gone = (t < 0) | (t >= vocab)
    x[gone] = torch.tensor([NAN, INF] * 50, device="cuda").to(BF)
    a = check(lib, x.clone().masked_fill_(gone[:, None], 0.0), w.clone(), t, piece=piece)
    dx, dw = torch.empty(rows, dim, dtype=BF, device="cuda"), torch.empty(vocab, dim, dtype=BF, device="cuda")
    losses = torch.empty(rows, device="cuda")
    out = call(lib, x, w, t, dx, dw, losses, piece)
    for p, q in zip(a, (out, losses, dx, dw)):
        assert E.same_bits(p, q)


def test_rows_that_are_not_numbers(lib):
    """A NaN stays in its row of losses and dhidden; logits far apart overflow nothing."""
    x, w, t = inputs(70, 200, 64, seed=9)
    ref_dx, ref = torch.empty_like(x), torch.empty(70, device="cuda")
    call(lib, x, w, t, ref_dx, None, ref)
    y = x.clone()
    y[3, 5] = NAN
    dx, losses = torch.empty_like(x), torch.empty(70, device="cuda")
    out = call(lib, y, w, t, dx, None, losses)
    assert bool(out.isnan()) and bool(losses[3].isnan()) and bool(dx[3].isnan().all())
    keep = torch.arange(70, device="cuda") != 3
    assert E.same_bits(losses[keep], ref[keep]) and E.same_bits(dx[keep], ref_dx[keep])
    # logits of +-1e4: the loss is their difference, softmax one or zero
    x = torch.zeros(4, 64, device="cuda").to(BF)
    w = torch.zeros(100, 64, device="cuda").to(BF)
    x[:, 0] = 100.0
    w[7, 0], w[9, 0] = 100.0, -100.0
    t = torch.tensor([7, 9, 0, 7], device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    losses = torch.empty(4, device="cuda")
    call(lib, x, w, t, dx, dw, losses, reduction="sum")
    assert losses.tolist() == [0.0, 20000.0, 10000.0, 0.0]
    assert dx[:, 0].tolist() == [0.0, 200.0, 100.0, 0.0] and not bool(torch.count_nonzero(dx[:, 1:]))
    assert dw[:, 0].float().nonzero()[:, 0].tolist() == [0, 7, 9] and float(dw[7, 0]) == 200.0


def test_sure_rows(lib):
    """The loss of a row that is sure of its target keeps its relative accuracy."""
    dim, vocab = 64, 500
    x = torch.randn(40, dim, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    w = (0.05 * torch.randn(vocab, dim, generator=torch.Generator().manual_seed(2))).to(BF).cuda()
    t = torch.arange(40, device="cuda") * 7
    w[t] = (x.double() * torch.linspace(0.05, 0.8, 40, device="cuda")[:, None] / 2).to(BF)
    out = check(lib, x, w, t)
    want = E.loss(x, w, t)["losses"][0]
    assert float(want.min()) < 1e-6 and bool(((out[1].double() - want).abs() <= 1e-4 * want).all())


def test_gradients_against_differences(lib):
    """The gradients are those of the library's own loss."""
    rows, vocab, dim = 12, 30, 16
    x, w, t = inputs(rows, vocab, dim, seed=11)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    call(lib, x, w, t, dx, dw, reduction="sum")
    for seed in range(4):
        gen = torch.Generator().manual_seed(seed)
        for a, g in ((x, dx), (w, dw)):
            # steps that bf16 holds: a power of two above the values' own step
            v = torch.randn(a.shape, generator=gen).sign().cuda() * 0.0625
            plus, minus = (a.float() + v).to(BF), (a.float() - v).to(BF)
            moved = (plus.double() - minus.double()) / 2
            f = (lambda b: call(lib, b, w, t, reduction="sum")) if a is x else (lambda b: call(lib, x, b, t, reduction="sum"))
            d = (f(plus).double() - f(minus).double()) / 2
            want = (g.double() * moved).sum()
            # the third derivative of a row's loss along the step is at most 2 (largest change of a
            # logit)^3, over 6; bf16 gradients; fp32 losses
            other = w if a is x else x
            reach = (moved.abs() @ other.double().abs().T.contiguous()).amax()
            tol = rows * reach ** 3 / 3 + 2 * E.BF16 * (g.double().abs() * moved.abs()).sum() + rows * 1e-5
            assert abs(float(d - want)) <= float(tol)


def test_captured_and_on_a_stream(lib):
    rows, vocab, dim = 200, 600, 128
    x, w, t = inputs(rows, vocab, dim, skip=0.2, seed=13)
    other = inputs(rows, vocab, dim, skip=0.5, seed=14)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    loss, losses = torch.empty(1, device="cuda"), torch.empty(rows, device="cuda")
    ws = torch.empty(lib.linear_cross_entropy_workspace(x, w, piece=128), dtype=torch.uint8, device="cuda")
    run = lambda **kw: lib.linear_cross_entropy(x, w, t, loss, ws, losses=losses, dhidden=dx, dweight=dw, piece=128, **kw)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    kept = [x.clone(), w.clone(), t.clone()]
    for i in range(4):
        for dst, src in zip((x, w, t), other if i % 2 else kept):
            dst.copy_(src)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        got = [a.clone() for a in (loss, losses, dx, dw)]
        want = E.loss(x, w, t)
        assert E.near(loss, *want["loss"], E.F32) and E.near(dw, *want["dweight"], E.BF16)
        run()
        torch.cuda.synchronize()
        for a, b in zip(got, (loss, losses, dx, dw)):
            assert E.same_bits(a, b)
    side = torch.cuda.Stream()
    for a in (loss, losses, dx, dw):
        a.zero_()
    torch.cuda.synchronize()
    run(stream=side)
    side.synchronize()
    for a, b in zip(got, (loss, losses, dx, dw)):
        assert E.same_bits(a, b)


def test_offsets_past_32_bits(lib):
    """Rows of every matrix 2^31 bytes and more from the first."""
    rows, vocab, dim, pitch = 40, 30000, 64, 40000
    far = torch.empty(vocab * pitch, dtype=BF, device="cuda").view(vocab, pitch)
    out = torch.empty(vocab * pitch, dtype=BF, device="cuda").view(vocab, pitch)
    x, w, t = inputs(rows, vocab, dim, seed=15)
    t[0] = vocab - 1
    far[:, :dim] = w
    wide = torch.empty(rows, 1 << 26, dtype=BF, device="cuda")
    wide[:, :dim] = x
    dx, dw = torch.empty_like(wide)[:, :dim], out[:, :dim]
    ref_x, ref_w = torch.empty_like(x), torch.empty_like(w)
    a = call(lib, wide[:, :dim], far[:, :dim], t, dx, dw)
    b = call(lib, x, w, t, ref_x, ref_w)
    assert E.same_bits(a, b) and E.same_bits(dx, ref_x) and E.same_bits(dw, ref_w)


def test_wide_pitches(lib):
    """Rows of weight further apart than a tile's 32-bit offsets reach."""
    rows, vocab, dim, pitch = 70, 150, 72, (1 << 20) + 64
    x, w, t = inputs(rows, vocab, dim, seed=17)
    far = torch.empty(vocab, pitch, dtype=BF, device="cuda")
    far[:, :dim] = w
    dx, dw, ref_x, ref_w = (torch.empty_like(a) for a in (x, w, x, w))
    a, b = call(lib, x, far[:, :dim], t, dx, dw), call(lib, x, w, t, ref_x, ref_w)
    assert E.same_bits(a, b) and E.same_bits(dx, ref_x) and E.same_bits(dw, ref_w)
    few = far[:40, :dim]                            # rows of hidden too
    a, b = call(lib, few, w, t[:40], dx[:40]), call(lib, few.contiguous(), w, t[:40], ref_x[:40])
    assert E.same_bits(a, b) and E.same_bits(dx[:40], ref_x[:40])


def test_refuses(lib):
    x, w, t = inputs(10, 20, 16)
    loss, ws = torch.empty(1, device="cuda"), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for bad in (lambda: lib.linear_cross_entropy(x.float(), w, t, loss, ws), lambda: lib.linear_cross_entropy(x, w, t.int(), loss, ws),
                lambda: lib.linear_cross_entropy(x, w, t, loss.double(), ws), lambda: lib.linear_cross_entropy(x, w, t, loss, ws.int()),
                lambda: lib.linear_cross_entropy(x, w, t, loss, ws, dhidden=x.float())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: lib.linear_cross_entropy(x[0], w, t, loss, ws), lambda: lib.linear_cross_entropy(x, w[:, :8], t, loss, ws),
                lambda: lib.linear_cross_entropy(x, w, t[:5], loss, ws), lambda: lib.linear_cross_entropy(x, w, t, loss[:0], ws),
                lambda: lib.linear_cross_entropy(x, w, t, loss, ws, losses=loss), lambda: lib.linear_cross_entropy(x, w, t, loss, ws, dweight=x),
                lambda: lib.linear_cross_entropy(x, w, t, loss, ws.cpu()), lambda: lib.linear_cross_entropy(x.T, w, t, loss, ws),
                lambda: lib.linear_cross_entropy(x, w, t, loss, ws, reduction="none")):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lib.linear_cross_entropy(x, w, t, loss, ws[:256]), lambda: lib.linear_cross_entropy(x, w, t, loss, ws, dhidden=x),
                lambda: lib.linear_cross_entropy(x, w, t, loss, ws[16:]), lambda: lib.linear_cross_entropy(x, w, t, loss, ws, piece=-1),
                lambda: lib.linear_cross_entropy(x, w, t, loss, ws, grad_scale=NAN)):
        with pytest.raises(lib.FsdpError):
            bad()
