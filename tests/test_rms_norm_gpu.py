"""RMS norm, forward and backward, against the formulas in 64 bits."""

import pytest
import torch

import muon_cases as M
from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

BF, F = torch.bfloat16, torch.float32
HALF = {BF: M.BF16, F: M.F32}
# fp32 roundings on the way to an element: a lane's sum of up to 64 squares (more for rows over
# 32768, by dim / 8192 chunks of 8), the joins of 64 lanes and 16 waves, and a few products
SUMS = 128


def sums(dim):
    return (SUMS + dim // 1024) * M.F32


def rows_of(rows, dim, pitch, shift, dtype, scale, seed):
    """rows x dim inside rows of `pitch`, `shift` elements off the allocation's start."""
    gen = torch.Generator().manual_seed(seed)
    buf = torch.full((rows * pitch + shift + 3,), float("nan"), dtype=dtype, device="cuda")
    t = buf[shift:shift + rows * pitch].view(rows, pitch)[:, :dim]
    t.copy_((scale * torch.randn(rows, dim, generator=gen)).to(dtype))
    return t


SIZES = [(1, 1, 0, 0), (3, 5, 0, 0), (1, 4096, 0, 0), (7, 64, 0, 0), (5, 511, 3, 1), (4, 513, 0, 0),
         (9, 1024, 8, 0), (6, 1027, 73, 1), (3, 2049, 0, 3), (40, 4096, 0, 0), (2, 8191, 1, 0),
         (600, 130, 0, 0), (3, 8192, 0, 0), (2, 16384, 0, 0), (2, 16385, 0, 0), (2, 32768, 0, 0),
         (2, 33000, 0, 0), (1, 70001, 5, 1),
         # rows that share a wave, workgroups that are not full, and outputs that go past L2
         (513, 33, 0, 0), (257, 128, 8, 0), (1030, 100, 4, 0), (130, 255, 1, 1), (66000, 128, 0, 0),
         (33000, 256, 0, 0), (17000, 504, 8, 0)]


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("bits8", [False, True])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("rows,dim,extra,shift", SIZES)
def test_forward(lib, rows, dim, extra, shift, dtype, bits8, residual):
    pitch, eps = dim + extra, 1e-6
    x = rows_of(rows, dim, pitch, shift, dtype, 1.0, 1)
    w = (1 + 0.1 * torch.randn(dim, generator=torch.Generator().manual_seed(2))).to(dtype).cuda()
    res = rows_of(rows, dim, pitch, shift, dtype, 2.0, 3) if residual else None
    tot = rows_of(rows, dim, pitch, shift, dtype, 0.0, 4) if residual else None
    out_t = torch.float8_e4m3fn if bits8 else dtype
    obuf = torch.full((rows, pitch), 7.0, device="cuda").to(out_t)
    out = obuf[:, :dim]
    rstd = torch.empty(rows, device="cuda")
    scales = torch.empty(rows, device="cuda") if bits8 else None
    lib.rms_norm(x, w, out, eps=eps, residual=res, residual_out=tot, rstd=rstd, scales=scales)
    torch.cuda.synchronize()
    h = x
    if residual:
        h = (x.float() + res.float()).to(dtype)
        assert M.same_bits(tot, h)
    y, r = M.norm_forward(h.double(), w.double(), eps)
    assert bool(((rstd.double() - r[:, 0]).abs() <= sums(dim) * r[:, 0]).all())
    fp32 = sums(dim) * y.abs()
    if bits8:
        want = y.abs().amax(1) / 448
        assert bool(((scales.double() - want).abs() <= 2 * sums(dim) * want).all())
        s = scales.double()[:, None]
        got = out.float().double() * s
        # half an e4m3 step: 2^-4 of the value, 2^-10 among the subnormals; q = y / s is rounded
        # once more in fp32 before it
        assert bool(((got - y).abs() <= (1 + M.E4M3) * 2 * fp32 + M.E4M3 * y.abs() + 2.0 ** -10 * s).all())
        assert float(out.float().abs().max()) == 448.0
    else:
        assert bool(((out.double() - y).abs() <= (1 + HALF[dtype]) * fp32 + HALF[dtype] * y.abs()).all())
    obuf[:, :dim] = torch.tensor(7.0, device="cuda").to(out_t)
    assert bool((obuf.float() == 7.0).all())             # what lies between the rows stays


@pytest.mark.parametrize("dim", [40, 4096, 40000])
@pytest.mark.parametrize("dtype", [BF, F])
def test_forward_special_rows(lib, dtype, dim):
    """A row of zeros (also with eps 0), of NaN, with an infinity; its neighbours are untouched."""
    x = rows_of(5, dim, dim, 0, dtype, 1.0, 5)
    clean = x.clone()
    x[1] = 0.0
    x[2, 3], x[3, dim - 1] = float("nan"), float("inf")
    w = torch.ones(dim, dtype=dtype, device="cuda")
    for eps in (1e-6, 0.0):
        out, ref = torch.empty_like(x), torch.empty_like(x)
        q = torch.empty(5, dim, dtype=torch.float8_e4m3fn, device="cuda")
        s, rstd = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
        lib.rms_norm(x, w, out, eps=eps)
        lib.rms_norm(clean, w, ref, eps=eps)
        lib.rms_norm(x, w, q, eps=eps, scales=s, rstd=rstd)
        torch.cuda.synchronize()
        for r in (0, 4):
            assert M.same_bits(out[r], ref[r]) and bool(torch.isfinite(s[r]))
        zero = out[1].float()
        assert bool((zero == 0).all()) if eps else bool(torch.isnan(zero).all())
        if eps:
            assert float(s[1]) == 2.0 ** -126 and bool((q[1].float() == 0).all())
        assert bool(torch.isnan(out[2]).all()) and bool(torch.isnan(q[2].float()).all())
        assert bool(torch.isnan(s[2])) and bool(torch.isnan(rstd[2]))
        # infinity: rstd is 0, the infinite element NaN, the rest zeros; in 8 bits all NaN
        assert float(rstd[3]) == 0.0 and bool(torch.isnan(out[3, dim - 1]))
        assert bool((out[3, :dim - 1].float() == 0).all()) and bool(torch.isnan(q[3].float()).all())


def test_forward_extreme_scales(lib):
    """Rows whose largest value is tiny or huge keep their 8-bit values inside the type."""
    x = torch.randn(4, 256, device="cuda")
    w = torch.full((256,), 1.0, device="cuda")
    for k in (1e-30, 1e-18, 1e18):
        q, s = torch.empty(4, 256, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(4, device="cuda")
        lib.rms_norm(x * k, w, q, eps=1e-6, scales=s)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(q.float()).all()) and bool((s >= 2.0 ** -126).all())


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", [BF, F])
@pytest.mark.parametrize("rows,dim,extra,shift", SIZES + [(1300, 520, 0, 0), (1025, 17, 2, 1)])
def test_backward(lib, rows, dim, extra, shift, dtype, residual):
    pitch = dim + extra
    x = rows_of(rows, dim, pitch, shift, dtype, 1.0, 6)
    dy = rows_of(rows, dim, pitch, shift, dtype, 1e-2, 7)
    dres = rows_of(rows, dim, pitch, shift, dtype, 1e-2, 8) if residual else None
    w = (1 + 0.1 * torch.randn(dim, generator=torch.Generator().manual_seed(9))).to(dtype).cuda()
    rstd = torch.rsqrt(x.double().square().mean(1) + 1e-6).float()
    xbuf = torch.full((rows, pitch), 7.0, dtype=dtype, device="cuda")
    dx, dw = xbuf[:, :dim], torch.empty(dim, dtype=dtype, device="cuda")
    ws = torch.full((lib.rms_norm_backward_workspace(rows, dim),), 255, dtype=torch.uint8, device="cuda")
    lib.rms_norm_backward(dy, x, w, rstd, dx, dw, ws, dresidual=dres)
    torch.cuda.synchronize()
    X, DY, W, R = x.double(), dy.double(), w.double(), rstd.double()[:, None]
    want, wantw = M.norm_backward(DY, X, W, R)
    g, xh = (DY * W).abs(), (X * R).abs()
    size = R * (g + xh * (g * xh).mean(1, keepdim=True))
    if residual:
        want = want + dres.double()
        size = size + dres.double().abs()
    fp32 = sums(dim) * size
    assert bool(((dx.double() - want).abs() <= (1 + HALF[dtype]) * fp32 + HALF[dtype] * want.abs()).all())
    sizew = (DY * X * R).abs().sum(0) * (min(rows, 64) + rows // 8 + 20) * M.F32
    assert bool(((dw.double() - wantw).abs() <= (1 + HALF[dtype]) * sizew + HALF[dtype] * wantw.abs()).all())
    again, dw2 = torch.empty(rows, dim, dtype=dtype, device="cuda"), torch.empty_like(dw)
    lib.rms_norm_backward(dy, x, w, rstd, again, dw2, ws, dresidual=dres)
    alone = torch.empty_like(again)
    lib.rms_norm_backward(dy, x, w, rstd, alone, None, None, dresidual=dres)
    torch.cuda.synchronize()
    assert M.same_bits(again, dx) and M.same_bits(dw2, dw) and M.same_bits(alone, dx)
    xbuf[:, :dim] = 7.0
    assert bool((xbuf == 7.0).all())


def test_backward_against_differences(lib):
    """The gradients are those of the library's own forward pass."""
    rows, dim, eps = 6, 48, 1e-3
    torch.manual_seed(10)
    x, w, dy = torch.randn(rows, dim), 1 + 0.1 * torch.randn(dim), torch.randn(rows, dim)

    def forward(x, w):
        out, rstd = torch.empty(rows, dim, device="cuda"), torch.empty(rows, device="cuda")
        lib.rms_norm(x.cuda(), w.cuda(), out, eps=eps, rstd=rstd)
        torch.cuda.synchronize()
        return out.double().cpu(), rstd

    rstd = forward(x, w)[1]
    dx, dw = torch.empty(rows, dim, device="cuda"), torch.empty(dim, device="cuda")
    ws = torch.empty(lib.rms_norm_backward_workspace(rows, dim), dtype=torch.uint8, device="cuda")
    lib.rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), rstd, dx, dw, ws)
    torch.cuda.synchronize()
    h = 2.0 ** -7
    for seed in range(4):
        v = torch.randn(rows, dim, generator=torch.Generator().manual_seed(seed)).sign()
        d = ((forward(x + h * v, w)[0] - forward(x - h * v, w)[0]) * dy).sum() / (2 * h)
        # central differences: h^2 / 6 of the third derivative (values of order 1, rows * dim
        # terms) and fp32 roundings over h
        tol = rows * dim * (h * h + 8 * M.F32 / h)
        assert abs(float(d - (dx.double().cpu() * v).sum())) <= tol
        u = v[0]
        d = ((forward(x, w + h * u)[0] - forward(x, w - h * u)[0]) * dy).sum() / (2 * h)
        assert abs(float(d - (dw.double().cpu() * u).sum())) <= tol


def test_backward_of_no_rows_is_zero(lib):
    e = torch.empty(0, 33, device="cuda")
    w, dw = torch.ones(33, device="cuda"), torch.full((33,), 5.0, device="cuda")
    lib.rms_norm_backward(e, e, w, torch.empty(0, device="cuda"), e, dw, None)
    lib.rms_norm(e, w, e)
    torch.cuda.synchronize()
    assert bool((dw == 0).all())


def test_streams_and_graph(lib):
    rows, dim = 70, 600
    x, res = torch.randn(rows, dim, device="cuda").bfloat16(), torch.randn(rows, dim, device="cuda").bfloat16()
    w, dy = torch.ones(dim, dtype=BF, device="cuda"), torch.randn(rows, dim, device="cuda").bfloat16()

    def buffers():
        new = lambda t, *s: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        return {"sum": new(BF, rows, dim), "out": new(torch.float8_e4m3fn, rows, dim), "rstd": new(F, rows),
                "scales": new(F, rows), "dx": new(BF, rows, dim), "dw": new(BF, dim),
                "ws": new(torch.uint8, lib.rms_norm_backward_workspace(rows, dim))}

    def both(b, stream=None):
        lib.rms_norm(x, w, b["out"], residual=res, residual_out=b["sum"], rstd=b["rstd"], scales=b["scales"],
                     stream=stream)
        lib.rms_norm_backward(dy, b["sum"], w, b["rstd"], b["dx"], b["dw"], b["ws"], stream=stream)

    a, b, c = buffers(), buffers(), buffers()
    torch.cuda.synchronize()
    both(c, torch.cuda.Stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        both(b)
    for i in range(3):
        x.mul_(1.0 + i)
        torch.cuda.synchronize()
        g.replay()
        both(a)
        torch.cuda.synchronize()
        for k in a:
            assert M.same_bits(a[k], b[k]), k
        if i == 0:
            for k in a:
                assert M.same_bits(a[k], c[k]), k


def test_binding_says_which_argument_is_wrong(lib):
    new = lambda *s, t=BF: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    x, w, out = new(4, 32), new(32), new(4, 32)
    good = dict(rstd=new(4, t=F), residual=new(4, 32), residual_out=new(4, 32))
    lib.rms_norm(x, w, out, **good)
    lib.rms_norm(x, w, out, stream=torch.cuda.current_stream(), **good)
    lib.rms_norm(x, w, out, stream=torch.cuda.current_stream().cuda_stream, **good)
    for args, kw, error, name in (
            ((x, w.float(), out), {}, TypeError, "weight"), ((x, new(31), out), {}, ValueError, "weight"),
            ((x, w, new(4, 31)), {}, ValueError, "out"), ((x, w, out.cpu()), {}, ValueError, "out"),
            ((x, w, out), {"rstd": new(3, t=F)}, ValueError, "rstd"), ((x, w, out), {"rstd": new(4)}, TypeError, "rstd"),
            ((x, w, out), {"residual": x}, ValueError, "residual"), ((x, w, out), {"scales": new(4, t=F)}, TypeError, "out"),
            ((x.T, new(4), new(32, 4)), {}, ValueError, "x"), ((x, w, None), {}, TypeError, "out")):
        with pytest.raises(error, match=name):
            lib.rms_norm(*args, **kw)
    with pytest.raises(ValueError, match="dresidual"):
        lib.rms_norm_backward(x, x, w, new(4, t=F), out, None, None, dresidual=new(5, 32))
    with pytest.raises(lib.FsdpError):                   # no workspace for dweight
        lib.rms_norm_backward(x, x.clone(), w, new(4, t=F), out, new(32), None)
    u = lib.Unit([(4, 32)], 1, 0)
    hp, m = lib.MuonHparams(), new(128, t=F)
    with pytest.raises(ValueError, match=r"grads\[1\]"):
        lib.reduce_momentum_shard(u, [new(128), new(127)], m, new(128), hp)
    with pytest.raises(TypeError, match="momentum"):
        lib.reduce_momentum_shard(u, [new(128)], new(128), new(128), hp)
    with pytest.raises(ValueError, match="scales"):
        lib.muon_apply_shard(u, [x], [], m, None, hp)
    with pytest.raises(TypeError, match=r"tensors\[0\]"):
        lib.muon_apply_shard(u, [m], [1.0], m, None, hp)
