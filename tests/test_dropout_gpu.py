"""The dropout against its definition, operation by operation in fp32: every bit."""

import pytest
import torch

import model_ends_cases as E
from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

BF, F = torch.bfloat16, torch.float32
SIZES = [(1, 1, 0, 0), (1, 8, 0, 0), (3, 5, 2, 1), (2, 64, 0, 0), (7, 100, 3, 1), (65, 129, 0, 0), (1, 4096, 0, 0),
         (5, 1027, 73, 1), (3, 2049, 0, 3), (2, 9000, 8, 0), (400, 24, 0, 0), (1030, 256, 0, 0), (33, 20000, 1, 1)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("rows,dim,extra,shift", SIZES)
def test_dropout(lib, rows, dim, extra, shift, dtype, residual):
    x = E.rows_of(rows, dim, dim + extra, shift, dtype, 1.0, 1)
    res = E.rows_of(rows, dim, dim + extra, shift, dtype, 2.0, 2) if residual else None
    for p, seed, offset in ((0.1, 7, 0), (0.5, 2 ** 63 + 12345, 2 ** 40 + 3), (0.0, 1, 1), (1.0, 1, 1), (2.0 ** -17, 3, 3)):
        out = E.Guarded(rows, dim, dim + extra, shift, dtype)
        lib.dropout(x, out.t, p, seed, offset, residual=res)
        torch.cuda.synchronize()
        assert E.same_bits(out.t, E.dropout(x, p, seed, offset, res)), (p, seed, offset)
        assert out.intact()


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("rows,dim,extra", [(9000, 2056, 0), (3000, 8200, 8), (1100, 20001, 7)])
def test_large(lib, rows, dim, extra, dtype, residual):
    """Outputs that go past L2, and ones of that size that cannot."""
    x = E.rows_of(rows, dim, dim + extra, 0, dtype, 1.0, 1)
    res = E.rows_of(rows, dim, dim + extra, 0, dtype, 2.0, 2) if residual else None
    out = E.Guarded(rows, dim, dim + extra, 0, dtype)
    lib.dropout(x, out.t, 0.1, 7, 8, residual=res)
    torch.cuda.synchronize()
    assert E.same_bits(out.t, E.dropout(x, 0.1, 7, 8, res))
    assert out.intact()


@pytest.mark.parametrize("dtype", [BF, F])
def test_in_place(lib, dtype):
    x, res = torch.randn(37, 200).to(dtype), torch.randn(37, 200).to(dtype)
    want, plain = E.dropout(x, 0.3, 5, 6, res), E.dropout(x, 0.3, 5, 6)
    a, b = x.cuda(), res.cuda()
    lib.dropout(a, a, 0.3, 5, 6)
    lib.dropout(x.cuda(), b, 0.3, 5, 6, residual=b)
    torch.cuda.synchronize()
    assert E.same_bits(a, plain) and E.same_bits(b, want)
    a = x.cuda()
    lib.dropout(a, a, 0.3, 5, 6, residual=res.cuda())
    lib.dropout(b, b, 0.5, 5, 6, residual=b)               # both at once
    torch.cuda.synchronize()
    assert E.same_bits(a, want) and E.same_bits(b, E.dropout(want, 0.5, 5, 6, want))


@pytest.mark.parametrize("dtype", [BF, F])
def test_special_values(lib, dtype):
    """What is dropped is 0 whatever it held; what is kept stays NaN or infinite."""
    x = torch.randn(64, 64).to(dtype)
    x[::3], x[1::3, ::2], x[2::3, 1::2] = float("nan"), float("inf"), -float("inf")
    out = torch.empty(64, 64, dtype=dtype, device="cuda")
    lib.dropout(x.cuda(), out, 0.5, 9, 9)
    torch.cuda.synchronize()
    keep = torch.from_numpy(E.dropout_bits(64, 64, 9, 9) >= 32768)
    got = out.cpu()
    assert E.same_bits(got[~keep], torch.zeros(int((~keep).sum()), dtype=dtype))
    want = E.dropout(x, 0.5, 9, 9)
    assert torch.equal(got.isnan(), want.isnan()) and E.same_bits(got.nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))
    if dtype == BF:
        assert (E.bits(got)[got.isnan().numpy()] == 0x7FC0).all()


def test_gradient_is_the_same_call(lib):
    """sum(dropout(x) * dy) changes with x as dropout(dy) says."""
    torch.manual_seed(1)
    x, dy = torch.randn(20, 33), torch.randn(20, 33)
    dx, plus, minus = (torch.empty(20, 33, device="cuda") for _ in range(3))
    lib.dropout(dy.cuda(), dx, 0.25, 11, 12)
    for seed in range(4):
        v = torch.randn(20, 33, generator=torch.Generator().manual_seed(seed))
        lib.dropout((x + v).cuda(), plus, 0.25, 11, 12)
        lib.dropout((x - v).cuda(), minus, 0.25, 11, 12)
        torch.cuda.synchronize()
        d = ((plus - minus).double().cpu() / 2 * dy).sum()
        want = (dx.double().cpu() * v).sum()
        # linear: only fp32 roundings, of values up to 8, three each
        assert abs(d - want) <= 3 * E.F32 * 8 * float(dy.abs().sum())


def test_counter(lib):
    """The device's number is added to the offset, modulo 2^64."""
    x = torch.randn(9, 50, device="cuda")
    out, ref = torch.empty_like(x), torch.empty_like(x)
    for number, offset in ((0, 5), (3, 2 ** 40), (-1, 0), (2 ** 62, 2 ** 63)):
        lib.dropout(x, out, 0.4, 1, offset, counter=torch.tensor([number], device="cuda"))
        lib.dropout(x, ref, 0.4, 1, (offset + number) % 2 ** 64)
        torch.cuda.synchronize()
        assert E.same_bits(out, ref)


def test_captured(lib):
    """A graph whose replays differ by the device's number alone."""
    x = torch.randn(300, 1000, device="cuda").to(BF)
    out = torch.empty_like(x)
    number = torch.zeros(1, dtype=torch.int64, device="cuda")
    lib.dropout(x, out, 0.1, 3, 100, counter=number)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.dropout(x, out, 0.1, 3, 100, counter=number)
    for i in range(4):
        number.fill_(i)
        graph.replay()
        torch.cuda.synchronize()
        ref = torch.empty_like(x)
        lib.dropout(x, ref, 0.1, 3, 100 + i)
        torch.cuda.synchronize()
        assert E.same_bits(out, ref)


def test_offsets_past_32_bits(lib):
    rows, dim, pitch = 40000, 24, 80000
    x = torch.zeros(rows * pitch, dtype=BF, device="cuda").view(rows, pitch)[:, :dim]
    x.fill_(1.0)
    out = torch.empty(rows, dim, dtype=BF, device="cuda")
    lib.dropout(x, out, 0.5, 1, 2)
    lib.dropout(out, x, 0.5, 1, 3)
    torch.cuda.synchronize()
    first = E.dropout(torch.ones(rows, dim, dtype=BF), 0.5, 1, 2)
    assert E.same_bits(out, first) and E.same_bits(x, E.dropout(first, 0.5, 1, 3))


def test_refuses(lib):
    x = torch.zeros(4, 8, device="cuda")
    with pytest.raises(lib.FsdpError):
        lib.dropout(x, torch.empty_like(x), 1.5, 1)
    with pytest.raises(lib.FsdpError):
        lib.dropout(x[:3], x[1:], 0.1, 1)
    for call in (lambda: lib.dropout(x, x.bfloat16(), 0.1, 1), lambda: lib.dropout(x, x, 0.1, 1, residual=x.bfloat16()),
                 lambda: lib.dropout(x, x, 0.1, 1, counter=torch.zeros(1, device="cuda"))):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: lib.dropout(x, x[:2], 0.1, 1), lambda: lib.dropout(x.T, x.T, 0.1, 1),
                 lambda: lib.dropout(x, x, 0.1, 1, residual=x.cpu())):
        with pytest.raises(ValueError):
            call()
