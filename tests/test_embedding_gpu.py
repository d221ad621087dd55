"""The embedding, forward and backward, against the formulas in 64 bits."""

import pytest
import torch

import model_ends_cases as E
from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

BF, F = torch.bfloat16, torch.float32
# tokens, vocab, dim, pitch - dim, elements off the allocation's start
SIZES = [(1, 1, 1, 0, 0), (1, 7, 5, 0, 0), (3, 300, 8, 0, 0), (65, 100, 64, 3, 1), (130, 513, 100, 0, 0),
         (1, 1000, 4096, 0, 0), (257, 70, 1027, 73, 1), (1000, 40, 33, 0, 3), (700, 5003, 520, 8, 0),
         (2050, 1500, 2056, 0, 0), (40, 131, 9000, 1, 1), (5000, 2, 24, 0, 0), (9, 140000, 16, 0, 0)]


def tokens_of(n, vocab, kind, seed=0):
    gen = torch.Generator().manual_seed(seed)
    t = torch.randint(0, vocab, (n,), generator=gen)
    if kind == "few":                                   # a handful of tokens, in long lists
        t = t.remainder(min(3, vocab)) * max(1, (vocab - 1) // 3)
    if kind == "outside":                               # a third is no row of the vocabulary
        bad = torch.tensor([-1, -100, vocab, vocab + 5, -2 ** 62, 2 ** 62])
        t = torch.where(torch.rand(n, generator=gen) < 0.34, bad[torch.randint(0, 6, (n,), generator=gen)], t)
    return t.cuda()


def back(lib, tokens, dy, dw, **kw):
    ws = torch.full((lib.embedding_backward_workspace(tokens.numel(), *dw.shape),), 255, dtype=torch.uint8, device="cuda")
    lib.embedding_backward(tokens, dy, dw, ws, **kw)


@pytest.mark.parametrize("kind", ["any", "outside"])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n,vocab,dim,extra,shift", SIZES)
def test_forward(lib, n, vocab, dim, extra, shift, dtype, kind):
    w = E.rows_of(vocab, dim, dim + extra, shift, dtype, 1.0, 1)
    t = tokens_of(n, vocab, kind)
    for scale in (1.0, 37.3):
        out = E.Guarded(n, dim, dim + extra, shift, dtype)
        lib.embedding(t, w, out.t, scale=scale)
        torch.cuda.synchronize()
        ok = (t >= 0) & (t < vocab)
        want = torch.where(ok[:, None], w[t.clamp(0, vocab - 1)].double() * scale, torch.zeros((), dtype=torch.float64, device="cuda"))
        # the scale's rounding to fp32 and the product's
        assert E.near(out.t, want, want.abs() * 2 * E.F32, E.HALF[dtype])
        if scale == 1.0:
            assert torch.equal(out.t.double(), want)
        assert out.intact()


def test_forward_special_values(lib):
    """Values that are not numbers stay where they are; tokens of any shape."""
    for dtype in (BF, F):
        w = torch.randn(6, 40).to(dtype).cuda()
        w[1, 3], w[2, 39], w[3, 0] = float("nan"), float("inf"), -0.0
        t = torch.tensor([[1, 2], [3, 7]], device="cuda")
        out = torch.empty(4, 40, dtype=dtype, device="cuda")
        lib.embedding(t, w, out)
        torch.cuda.synchronize()
        want = torch.cat([w[1:4], torch.zeros(1, 40, dtype=dtype, device="cuda")])
        assert torch.equal(out.isnan(), want.isnan()) and E.same_bits(out.nan_to_num(7.0), want.nan_to_num(7.0))
        if dtype == BF:
            assert E.bits(out)[0, 3] == 0x7FC0
    lib.embedding(torch.empty(0, dtype=torch.int64, device="cuda"), w, out[:0])


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("kind", ["any", "few", "outside"])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n,vocab,dim,extra,shift", SIZES)
def test_backward(lib, n, vocab, dim, extra, shift, dtype, kind, add):
    dy = E.rows_of(n, dim, dim + extra, shift, dtype, 1e-2, 2)
    t = tokens_of(n, vocab, kind, 3)
    dw = E.Guarded(vocab, dim, dim + extra, shift, dtype)
    old = E.rows_of(vocab, dim, dim + extra, shift, dtype, 0.1, 4) if add else None
    if add:
        dw.t.copy_(old)
    padding = int(t[0]) if n > 2 and vocab > 2 else -1
    back(lib, t, dy, dw.t, scale=3.7, accumulate=add, padding_idx=padding)
    torch.cuda.synchronize()
    want, off, count = E.embedding_backward(t, dy, vocab, 3.7, old, padding)
    assert E.near(dw.t, want, off, E.HALF[dtype])
    absent = count == 0
    if add:
        assert E.same_bits(dw.t[absent], old[absent])
    else:
        assert not bool(torch.count_nonzero(dw.t[absent]))
    assert dw.intact()
    again = torch.empty(vocab, dim, dtype=dtype, device="cuda")
    if add:
        again.copy_(old)
    back(lib, t, dy, again, scale=3.7, accumulate=add, padding_idx=padding)
    torch.cuda.synchronize()
    assert E.same_bits(again, dw.t)


@pytest.mark.parametrize("dtype", [BF, F])
def test_backward_of_frequent_tokens(lib, dtype):
    """Lists of every length around the ones that are split, and all of 20000 tokens the same."""
    lengths = [1, 2, 3, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 130, 255, 256, 257, 511, 513, 1000, 0, 1025, 5]
    t = torch.cat([torch.full((k,), i) for i, k in enumerate(lengths)])
    t = t[torch.randperm(len(t), generator=torch.Generator().manual_seed(1))].cuda()
    for tokens, vocab in ((t, len(lengths)), (torch.full((20000,), 5, device="cuda"), 9)):
        for dim in (24, 1032):
            dy = E.rows_of(len(tokens), dim, dim, 0, dtype, 1.0, 5)
            for add in (False, True):
                dw = torch.full((vocab, dim), 0.5, dtype=dtype, device="cuda")
                old = dw.clone() if add else None
                back(lib, tokens, dy, dw, accumulate=add)
                torch.cuda.synchronize()
                want, off, _ = E.embedding_backward(tokens, dy, vocab, 1.0, old)
                assert E.near(dw, want, off, E.HALF[dtype]), (vocab, dim, add)


@pytest.mark.parametrize("dtype,n,vocab,dim", [(BF, 3000, 12000, 2056), (F, 2500, 30001, 1028), (BF, 9000, 7000, 4096), (F, 40, 9000, 1500),
                                               (BF, 100, 40000, 2048), (BF, 2048, 5000, 1024), (BF, 2049, 5000, 1024)])
def test_backward_large(lib, dtype, n, vocab, dim):
    """Outputs that go past L2, whose zeros are written by every launch; frequent tokens at both
    ends of the vocabulary."""
    gen = torch.Generator().manual_seed(n)
    t = torch.randint(0, vocab, (n,), generator=gen)
    t[::3] = torch.tensor([0, 1, vocab - 1, vocab - 2, vocab // 2])[torch.randint(0, 5, (len(t[::3]),), generator=gen)]
    t = t.cuda()
    dy = E.rows_of(n, dim, dim, 0, dtype, 1e-2, 3)
    for add in (False, True):
        dw = torch.full((vocab, dim), 0.25 if add else float("nan"), dtype=dtype, device="cuda")
        back(lib, t, dy, dw, scale=2.0, accumulate=add)
        torch.cuda.synchronize()
        want, off, _ = E.embedding_backward(t, dy, vocab, 2.0, torch.full_like(dw, 0.25) if add else None)
        assert E.near(dw, want, off, E.HALF[dtype])
        del want, off


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("n,dim,extra", [(9000, 2056, 0), (3000, 8200, 8), (40000, 520, 0), (1200, 20001, 0)])
def test_forward_large(lib, dtype, n, dim, extra):
    w = E.rows_of(500, dim, dim, 0, dtype, 1.0, 1)
    t = tokens_of(n, 500, "outside")
    out = E.Guarded(n, dim, dim + extra, 0, dtype)
    lib.embedding(t, w, out.t)
    torch.cuda.synchronize()
    ok = (t >= 0) & (t < 500)
    assert torch.equal(out.t, torch.where(ok[:, None], w[t.clamp(0, 499)], torch.zeros((), dtype=dtype, device="cuda")))
    assert out.intact()


def test_backward_order(lib):
    """Equal tokens are summed so that the same inputs give the same bits, and values that are not
    numbers reach only their own row."""
    n, vocab, dim = 4096, 64, 256
    t = tokens_of(n, vocab, "any", 8)
    dy = torch.randn(n, dim, device="cuda").to(BF)
    ref = torch.empty(vocab, dim, dtype=BF, device="cuda")
    back(lib, t, dy, ref)
    for _ in range(5):
        got = torch.empty_like(ref)
        back(lib, t, dy, got)
        torch.cuda.synchronize()
        assert E.same_bits(got, ref)
    i = int(torch.nonzero(t == 7)[0])
    dy[i, 3] = float("inf")
    dy[i, 4] = float("nan")
    back(lib, t, dy, got)
    torch.cuda.synchronize()
    same = got.clone()
    same[7, 3:5] = ref[7, 3:5]
    assert E.same_bits(same, ref) and bool(got[7, 3].isinf()) and bool(got[7, 4].isnan())


def test_no_tokens(lib):
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    dw = torch.full((300, 40), 7.0, device="cuda")
    back(lib, none, torch.empty(0, 40, device="cuda"), dw, accumulate=True)
    torch.cuda.synchronize()
    assert bool((dw == 7).all())
    back(lib, none, torch.empty(0, 40, device="cuda"), dw)
    torch.cuda.synchronize()
    assert not bool(torch.count_nonzero(dw))


def test_offsets_past_32_bits(lib):
    """Rows far apart: 3 * 2^31 bytes from the first to the last."""
    vocab, dim, pitch = 40000, 24, 80000
    buf = torch.zeros(vocab * pitch, dtype=BF, device="cuda")
    w = buf.view(vocab, pitch)[:, :dim]
    rows = torch.tensor([0, 1, 13000, 27000, 39998, 39999], device="cuda")
    vals = torch.randn(6, dim, device="cuda").to(BF)
    w[rows] = vals
    out = torch.empty(6, dim, dtype=BF, device="cuda")
    lib.embedding(rows, w, out)
    torch.cuda.synchronize()
    assert torch.equal(out, vals)
    back(lib, rows, vals, w, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(w[rows], (vals.float() * 2).to(BF))
    lib.embedding(torch.arange(vocab, device="cuda"), vals[:1], w)          # an output past 32 bits
    torch.cuda.synchronize()
    assert torch.equal(w[0], vals[0]) and not bool(torch.count_nonzero(w[1:]))


def test_refuses_other_types(lib):
    w = torch.zeros(4, 8, device="cuda")
    t = torch.zeros(2, dtype=torch.int64, device="cuda")
    out = torch.zeros(2, 8, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for call in (lambda: lib.embedding(t.int(), w, out), lambda: lib.embedding(t, w, out.bfloat16()),
                 lambda: lib.embedding_backward(t, out.bfloat16(), w, ws), lambda: lib.embedding_backward(t, out, w, ws.int())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: lib.embedding(t, w, out[:1]), lambda: lib.embedding(t, w.T, out), lambda: lib.embedding(t[:1].expand(2), w, out),
                 lambda: lib.embedding_backward(t, out[:1].expand(2, 8), w, ws), lambda: lib.embedding_backward(t, out.cpu(), w, ws)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(lib.FsdpError):
        lib.embedding_backward(t, out, w, ws[:16])
