"""Orthogonalisation of lists, by what decides how a launch is run: the number of products (arguments
for 4, 8 and 24), equal and unequal lengths, split contractions, the tile; and what a bound on an
easy matrix does not show: single elements, hard spectra, streams, the other matrices of a call."""

import pytest
import torch

import muon_cases as M
from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

BF, F = torch.bfloat16, torch.float32


def matrix(r, c, seed, dtype=BF):
    """A few strong directions over noise."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    k = max(1, min(r, c) // 16)
    return (1e-3 * (rn(r, k) @ rn(k, c) / k ** 0.5 + 0.5 * rn(r, c))).to(dtype)


def polar(g, steps=5, coeffs=M.COEFFS, eps=1e-7):
    """M.polar on the matrix's device; right operands are laid out, not views."""
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.T.contiguous() if tall else x
    x = x / (x.norm() + eps)
    a, b, c = coeffs
    for _ in range(steps):
        s = x @ x.T.contiguous()
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.T if tall else x


def run(lib, mats, stream=None, **kw):
    """Outputs and workspace are made and filled on the stream that the call goes to."""
    torch.cuda.synchronize()                              # the inputs come from another
    with torch.cuda.stream(stream):
        outs = [torch.full(m.shape, float("nan"), dtype=BF, device="cuda") for m in mats]
        ws = torch.full((max(1, lib.orthogonalize_workspace(mats)),), 255, dtype=torch.uint8, device="cuda")
        lib.orthogonalize(mats, outs, ws, stream=stream, **kw)
    torch.cuda.synchronize()
    return outs


def check(mats, outs, steps=5):
    for m, o in zip(mats, outs):
        if m.numel():
            want = polar(m, steps=steps)
            assert (o.double() - want).norm() <= M.polar_tolerance(steps) * want.norm(), tuple(m.shape)


MIXED = [(130, 200), (200, 130), (64, 500), (300, 300), (77, 90), (1, 50), (260, 90), (400, 410), (33, 600)]
LONG = [(100, 4000), (4096, 60), (128, 2048), (90, 100), (64, 8192), (190, 2900), (70, 4096), (128, 128)]


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("count", [1, 3, 4, 5, 7, 8, 9, 24, 25])
@pytest.mark.parametrize("shapes", [[(200, 330)], MIXED, LONG], ids=["equal", "mixed", "split"])
def test_counts(lib, shapes, count, dtype):
    mats = [matrix(*shapes[i % len(shapes)], seed=i, dtype=dtype) for i in range(count)]
    check(mats, run(lib, mats))


@pytest.mark.parametrize("shapes", [
    [(2048, 2048)] * 7,                                   # 256 tiles, 8 products
    [(2048, 2048)] * 5 + [(2304, 2048), (2048, 4096)],    # 256 and 128 tiles, equal and unequal lengths
    [(2048, 2048)] * 9,                                   # 128 tiles, 24 products
    [(128, 8192)] * 6,                                    # 64 tiles split and joined
    [(512, 8192)] * 5,                                    # 128 tiles split, joined by 64 tiles
    [(768, 8192)] * 4 + [(512, 12000)],                   # the same with unequal lengths, then 256 tiles
    [(512, 4096)] * 9, [(64, 9000)] * 10,                 # split, with arguments for 24
    [(1100, 1500)] * 8, [(1024, 2048)] * 5,               # 128 tiles, more than one a CU and fewer
    [(256, 1024), (1024, 256)], [(1024, 8192)] * 2, [(4096, 4096)],
    [(515, 1373), (2049, 771), (1000, 1000)],
], ids=lambda s: "%dx%dx%d" % (len(s), *s[-1]))
def test_launch_shapes(lib, shapes):
    mats = [matrix(*s, seed=i) for i, s in enumerate(shapes)]
    outs = run(lib, mats)
    check(mats, outs)
    for a, b in zip(outs, run(lib, mats)):
        assert M.same_bits(a, b)


def fixed_point(r, c, j, k, seed):
    """2^j orthogonal lines of 2^k values +-1 at random places of zeros (j + k even), signs at random. With
    eps 0 X_0 is +-2^(-(j+k)/2) there and S is 2^-j on the diagonal; coefficients (2, -2 2^j, 4^j) have
    p(2^-j) = 1, so X_0 is every step's X, and every value on the way a power of two: no rounding anywhere."""
    gen = torch.Generator().manual_seed(seed)
    h = torch.ones(1, 1)
    for _ in range(k):
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)])
    h = h[torch.randperm(2 ** k, generator=gen)[:2 ** j]][:, torch.randperm(2 ** k, generator=gen)]
    h = h * (2.0 * torch.randint(0, 2, (2 ** j, 1), generator=gen) - 1) * (2.0 * torch.randint(0, 2, (1, 2 ** k), generator=gen) - 1)
    m, n = min(r, c), max(r, c)
    x = torch.zeros(m, n)
    lines, places = torch.randperm(m, generator=gen)[:2 ** j].sort()[0], torch.randperm(n, generator=gen)[:2 ** k].sort()[0]
    x[lines[:, None], places[None, :]] = h
    return (x.T.contiguous() if r > c else x).cuda()


@pytest.mark.parametrize("steps", [1, 2, 5])
@pytest.mark.parametrize("shapes,j,k", [
    ([(5, 9)], 1, 3), ([(64, 64)], 6, 6), ([(65, 130), (130, 65), (33, 64)], 4, 6), ([(300, 1029), (256, 1024)], 8, 10),
    ([(128, 8192)] * 6, 7, 13), ([(512, 4096)] * 9, 8, 12), ([(1024, 1024), (1027, 2047)], 10, 10),
    ([(1100, 1500)] * 8, 10, 10), ([(2048, 2100)] * 7, 10, 10), ([(2048, 2048)], 11, 11), ([(4096, 4096), (4100, 4111)], 12, 12),
    ([(8200, 4100), (4096, 8192)], 11, 13), ([(1024, 8192)] * 2, 9, 13),
], ids=lambda v: "%dx%dx%d" % (len(v), *v[-1]) if isinstance(v, list) else str(v))
def test_every_element_where_nothing_is_rounded(lib, shapes, j, k, steps):
    """A value lost, misplaced or stale anywhere in a product or an epilogue shows by its bits, where a
    bound on the whole matrix hides it (one of 4096 x 4096 is 2.4e-4 of the norm)."""
    mats = [fixed_point(*s, j, k, seed=i) for i, s in enumerate(shapes)]
    outs = run(lib, mats, steps=steps, coeffs=(2.0, -2.0 * 2 ** j, 4.0 ** j), eps=0.0)
    for m, o in zip(mats, outs):
        assert torch.equal(o, (m * 2.0 ** (-(j + k) / 2)).to(BF)), (tuple(m.shape), int((o != m * 2.0 ** (-(j + k) / 2)).sum()))


def spectrum(r, c, values, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    k = min(r, c)
    u = torch.linalg.qr(torch.randn(r, k, generator=gen, device="cuda", dtype=torch.float64))[0]
    v = torch.linalg.qr(torch.randn(c, k, generator=gen, device="cuda", dtype=torch.float64))[0]
    return (u * values(torch.arange(1, k + 1, device="cuda").double())) @ v.T.contiguous()


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("shape", [(384, 1536), (300, 310), (700, 90)])
@pytest.mark.parametrize("values", [lambda k: 1 / k, lambda k: k ** -2, lambda k: (k == 1) + 1e-2, lambda k: 0.8 ** k],
                         ids=["1/k", "1/k^2", "one", "0.8^k"])
def test_hard_spectra(lib, values, shape, dtype):
    """Small singular values are raised, and with them what roundings put there. A rounding of the
    operands changes an element by at most 2^-11 of it, by 0.4 of that in the mean square (values
    spread over a binade); the 16 of 5 steps are independent and none is raised more than X_0's. So the
    error is below twice what a change of 2^-11 in every element of the matrix makes."""
    g = spectrum(*shape, values, seed=shape[0]).to(dtype)
    want = polar(g)
    sign = torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").sign()
    change = (polar(g.double() * (1 + M.F16 * sign)) - want).norm()
    (o,) = run(lib, [g])
    assert (o.double() - want).norm() <= M.BF16 * want.norm() + 2 * change


def test_the_other_matrices_of_a_call_may_change_bits_but_not_the_value(lib):
    """Pairs of steps are taken, or not, by all matrices of a call, and the tile by what fits them all."""
    a, b, c = matrix(515, 1373, 1), matrix(771, 2049, 2), matrix(64, 70, 3)
    for mats in ([a], [a, b], [b, a], [a, c], [c], [c, b, a]):
        check(mats, run(lib, mats))
    (x, _), (_, y) = run(lib, [a, b]), run(lib, [b, a])
    assert M.same_bits(x, y)                              # the order of the same sizes does not matter


@pytest.mark.parametrize("shapes", [[(150, 260), (260, 90)], [(128, 8192)] * 6])
def test_side_stream(lib, shapes):
    mats = [matrix(*s, seed=i) for i, s in enumerate(shapes)]
    want = run(lib, mats)
    for a, b in zip(want, run(lib, mats, stream=torch.cuda.Stream())):
        assert M.same_bits(a, b)
