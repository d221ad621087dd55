"""Edges of the Muon step and the RMS norm: ranges, coefficients, NaN bits, absent tensors."""

import pytest
import torch

import muon_cases as M
from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

BF, F = torch.bfloat16, torch.float32


def ortho(lib, mats, **kw):
    outs = [torch.empty(m.shape, dtype=BF, device="cuda") for m in mats]
    ws = torch.full((max(1, lib.orthogonalize_workspace(mats)),), 255, dtype=torch.uint8, device="cuda")
    lib.orthogonalize(mats, outs, ws, **kw)
    torch.cuda.synchronize()
    return outs


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("scale", [1e-33, 1e-36, 1e-38, 1e37])
def test_norms_at_the_ends_of_fp32(lib, scale, dtype):
    """X / |X| is of order 1 whatever |X| is, subnormal elements among them; eps is not narrowed."""
    gen = torch.Generator().manual_seed(1)
    m = (torch.randn(70, 90, generator=gen) * scale).to(dtype).cuda()
    for eps in (0.0, 1e-50):
        (o,) = ortho(lib, [m], eps=eps)
        want = M.polar(m, eps=eps)
        assert (o.double().cpu() - want).norm() <= M.polar_tolerance(5) * want.norm()


@pytest.mark.parametrize("eps", [1e-30, 1e-36, 1e-45, 1e-60, 1e-310])
def test_zero_matrix_with_a_tiny_eps_is_zero(lib, eps):
    (o,) = ortho(lib, [torch.zeros(30, 50, device="cuda")], eps=eps)
    assert bool((o == 0).all())


# Every value of these is exact in the operands' format, so the results are the formula's bits: one
# row of 2^-5 or so in absolute value whose norm is a power of two, among rows of zeros.
@pytest.mark.parametrize("shape", [(1, 1), (64, 4096), (4096, 64), (1024, 1024)])
@pytest.mark.parametrize("steps,coeffs", [
    (5, (3.0, 0.0, 0.0)),            # 3^k: 243 in the end
    (2, (8.5, -14.0, 6.0)),          # below 4 on [0, 1.3], and the polynomials' product 72.25 where X is 0
    (3, (-60.0, 30.0, 31.0)), (2, (100.0, -200.0, 101.0)), (7, (2.0, 0.0, 0.0)),
])
def test_coefficients_that_grow(lib, steps, coeffs, shape):
    m = torch.zeros(*shape, device="cuda")
    line = m[0] if shape[0] <= shape[1] else m[:, 0]
    line.copy_(torch.randn(line.numel(), generator=torch.Generator().manual_seed(2)).sign())
    (o,) = ortho(lib, [m], steps=steps, coeffs=coeffs, eps=0.0)
    x = 1.0
    for _ in range(steps):
        x = coeffs[0] * x + coeffs[1] * x ** 3 + coeffs[2] * x ** 5
    want = (m.double() / line.numel() ** 0.5 * x).to(BF)
    assert torch.equal(o, want)


def test_coefficients_that_grow_on_any_matrix(lib):
    """Singular values that pass 16: powers of 2 are taken out of X, S and P."""
    gen = torch.Generator().manual_seed(3)
    for shape in ((90, 130), (300, 2000), (700, 500)):
        m = torch.randn(*shape, generator=gen).cuda()
        for steps, coeffs in ((5, (4.0, 0.0, 0.0)), (4, (3.0, 1.0, 0.0))):
            (o,) = ortho(lib, [m], steps=steps, coeffs=coeffs)
            want = M.polar(m, steps=steps, coeffs=coeffs)
            assert want.norm() > 20
            # as for polar_tolerance, each rounding amplified by the steps after it: relative to X
            # by 1 where p is a number, by less than 3 for 3 x + x^3
            tol = M.BF16 + (M.polar_tolerance(steps) - M.BF16) * (1 if coeffs[1] == 0 else 3 ** (steps - 1))
            assert (o.double().cpu() - want).norm() <= tol * want.norm()


@pytest.mark.parametrize("rows,dim,shift", [(3, 21, 0), (2, 4099, 1), (2, 16390, 0), (9000, 2049, 7)])
def test_norm_writes_one_nan(lib, rows, dim, shift):
    """Every NaN rounds to 0x7FC0, in a row's whole vectors and in its ragged end, in each way of storing."""
    payloads = torch.tensor([0x7FC1, -0x40, 0x7F81, -1, -0x7F], dtype=torch.int16).view(BF).cuda()   # both signs, quiet and not
    assert bool(torch.isnan(payloads).all())
    wide = torch.zeros(rows, dim + shift, dtype=BF, device="cuda")
    w, x = torch.ones(dim, dtype=BF, device="cuda"), torch.ones(rows, dim + shift, dtype=BF, device="cuda")[:, :dim]
    at = torch.arange(0, dim, 3, device="cuda")
    res = torch.zeros(rows, dim, dtype=BF, device="cuda")
    res[:, at] = payloads[at % 5]
    out, total, rstd = wide[:, :dim], torch.empty_like(wide)[:, :dim], torch.empty(rows, device="cuda")
    lib.rms_norm(x, w, out, residual=res, residual_out=total, rstd=rstd)
    dx, dw = torch.empty_like(wide)[:, :dim], torch.empty(dim, dtype=BF, device="cuda")
    ws = torch.empty(lib.rms_norm_backward_workspace(rows, dim), dtype=torch.uint8, device="cuda")
    lib.rms_norm_backward(res, x, w, torch.ones(rows, device="cuda"), dx, dw, ws, dresidual=res)
    torch.cuda.synchronize()
    for t in (out, total, dx, dw):
        nan = torch.isnan(t)
        assert bool((t.contiguous().view(torch.int16)[nan] == 0x7FC0).all())
    assert bool(torch.isnan(out).all()) and bool(torch.isnan(dx).all())      # a row's sum holds them
    here = torch.zeros(dim, dtype=torch.bool, device="cuda")
    here[at] = True
    assert torch.equal(torch.isnan(total), here.expand(rows, dim))
    assert bool((total[:, ~here] == 1).all()) and torch.equal(torch.isnan(dw), here)
    # a weight's NaN stays in its column
    w[5] = payloads[1]
    lib.rms_norm(x, w, out)
    torch.cuda.synchronize()
    here[:] = False
    here[5] = True
    assert torch.equal(torch.isnan(out), here.expand(rows, dim))
    assert bool((out.contiguous().view(torch.int16)[:, 5] == 0x7FC0).all())


def test_apply_takes_none_outside_the_window(lib):
    """A rank needs the tensors that reach into its window, and no others."""
    shapes, F_ = [(40, 100), (77,), (0, 3), (100, 40), (64, 64)], 4
    gen = torch.Generator().manual_seed(4)
    ts = [torch.randn(*s, generator=gen).to(BF).cuda() for s in shapes]
    scales = [1.0, 2.0, 0.5, 1.5, 0.25]
    hp = lib.MuonHparams(lr=0.1, weight_decay=0.05)
    for rank in range(F_):
        u = lib.Unit(shapes, F_, rank)
        end = u.shard_begin + u.shard_valid
        mine = [max(o, u.shard_begin) < min(o + n, end) for o, n in zip(u.offsets, u.numels)]
        assert not all(mine)
        p = torch.randn(u.shard_valid, generator=gen).cuda()
        q = p.clone()
        lib.muon_apply_shard(u, ts, scales, p, None, hp)
        lib.muon_apply_shard(u, [t if m else None for t, m in zip(ts, mine)],
                             [k if m else None for k, m in zip(scales, mine)], q, None, hp)
        torch.cuda.synchronize()
        assert M.same_bits(p, q)
        first = mine.index(True)
        with pytest.raises(TypeError, match=r"tensors\[%d\]" % first):
            lib.muon_apply_shard(u, [None if i == first else t for i, t in enumerate(ts)], scales, q, None, hp)


@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("dim", [40, 20000])
def test_norm_of_zeros_with_a_tiny_eps_is_zero(lib, dim, dtype):
    """A positive eps below fp32's least number is not taken for 0: rows of zeros stay zeros."""
    x, w = torch.zeros(3, dim, dtype=dtype, device="cuda"), torch.ones(dim, dtype=dtype, device="cuda")
    for eps in (1e-40, 1e-46, 1e-300):
        out, rstd = torch.full_like(x, 3.0), torch.empty(3, device="cuda")
        lib.rms_norm(x, w, out, eps=eps, rstd=rstd)
        torch.cuda.synchronize()
        assert bool((out == 0).all()) and bool(torch.isfinite(rstd).all())


def test_offsets_past_32_bits_in_the_step(lib):
    """A window of over 2^31 elements: every one of the momentum's, and of the master's."""
    u = lib.Unit([((1 << 16) + 1, 1 << 15), (77,)], 1, 0)
    n, hp = u.shard_valid, lib.MuonHparams(lr=0.5, momentum=0.5, nesterov=False, weight_decay=0.0)
    grad = torch.empty(n, dtype=BF, device="cuda").random_(-100, 100)
    m, upd = torch.ones(n, device="cuda"), torch.empty(n, dtype=BF, device="cuda")
    lib.reduce_momentum_shard(u, [grad], m, upd, hp, grad_scale=1.0)
    parts = [slice(a, min(a + (1 << 28), n)) for a in range(0, n, 1 << 28)]
    for s in parts:                                       # halves of small whole numbers: exact
        want = 0.5 + grad[s].float()
        assert torch.equal(m[s], want) and torch.equal(upd[s], want.to(BF))
    del m
    tensors = list(grad.split(u.numels))
    p, w = torch.full((n,), 3.0, device="cuda"), upd
    lib.muon_apply_shard(u, tensors, [1.0, 2.0], p, w, hp)
    for s in parts:
        want = 3.0 - 0.5 * grad[s].float()
        if s.stop == n:
            want[-77:] = 3.0 - grad[s][-77:].float()
        assert torch.equal(p[s], want) and torch.equal(w[s], want.to(BF))


@pytest.mark.parametrize("rows,dim,pitch", [((1 << 22) - 1, 513, 513), (3, 70, (1 << 31) + 8), (3, 17000, (1 << 30) + 1)])
def test_offsets_past_32_bits_in_the_norm(lib, rows, dim, pitch):
    x = torch.empty((rows - 1) * pitch + dim, dtype=BF, device="cuda").as_strided((rows, dim), (pitch, 1))
    out, dx = torch.empty_strided(x.shape, x.stride(), dtype=BF, device="cuda"), torch.empty(rows, dim, dtype=BF, device="cuda")
    step = 1 << 16
    gen = torch.Generator(device="cuda").manual_seed(6)
    for a in range(0, rows, step):
        x[a:a + step] = torch.randn(min(step, rows - a), dim, generator=gen, device="cuda").to(BF)
    w, rstd, dw = torch.ones(dim, dtype=BF, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(dim, dtype=BF, device="cuda")
    ws = torch.empty(lib.rms_norm_backward_workspace(rows, dim), dtype=torch.uint8, device="cuda")
    lib.rms_norm(x, w, out, rstd=rstd)
    lib.rms_norm_backward(x, x, w, rstd, dx, dw, ws)
    sums = torch.zeros(dim, dtype=torch.float64, device="cuda")
    for a in range(0, rows, step):
        X = x[a:a + step].double()
        y, r = M.norm_forward(X, w.double(), 1e-6)
        # as for shorter rows: a lane's chunks, the joins and a few products in fp32, then bf16
        fp32 = (128 + dim // 1024) * M.F32
        assert bool(((out[a:a + step].double() - y).abs() <= (fp32 + M.BF16) * 1.01 * y.abs()).all())
        want = M.norm_backward(X, X, w.double(), r)[0]
        size = r * (X.abs() + (X * r).abs() * (X * X * r).mean(1, keepdim=True))
        assert bool(((dx[a:a + step].double() - want).abs() <= 1.01 * fp32 * size + M.BF16 * want.abs()).all())
        sums += (X * X * r).sum(0)
    # a workgroup adds a 256th of the rows, then come the joins of its waves and of the workgroups
    assert bool(((dw.double() - sums).abs() <= (rows // 256 + 300) * M.F32 * sums + M.BF16 * sums.abs()).all())


def test_offsets_past_32_bits_in_a_matrix(lib):
    pitch = (1 << 30) + 3
    m = torch.empty(4 * pitch + 90, dtype=BF, device="cuda").as_strided((5, 90), (pitch, 1))
    m.copy_(torch.randn(5, 90, generator=torch.Generator().manual_seed(7)).to(BF))
    out = torch.empty_strided(m.shape, m.stride(), dtype=BF, device="cuda")
    ws = torch.empty(lib.orthogonalize_workspace([m]), dtype=torch.uint8, device="cuda")
    lib.orthogonalize([m], [out], ws)
    torch.cuda.synchronize()
    want = M.polar(m)
    assert (out.double().cpu() - want).norm() <= M.polar_tolerance(5) * want.norm()
