"""Newton-Schulz orthogonalisation against the definition in 64 bits."""

import pytest
import torch

import muon_cases as M
from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def matrix(r, c, seed, dtype=torch.bfloat16, pitch=None):
    """A few strong directions over noise, in rows of `pitch` elements."""
    gen = torch.Generator().manual_seed(seed)
    k = max(1, min(r, c) // 16)
    rn = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    g = 1e-3 * (rn(r, k) @ rn(k, c) / k ** 0.5 + 0.5 * rn(r, c))
    buf = torch.full((r, pitch or c), float("nan")).to(dtype)
    buf[:, :c] = g.to(dtype)
    return buf.cuda()[:, :c]


def run(lib, mats, outs=None, stream=None, **kw):
    outs = [torch.empty(m.shape, dtype=torch.bfloat16, device="cuda") for m in mats] if outs is None else outs
    ws = torch.full((max(1, lib.orthogonalize_workspace(mats)),), 255, dtype=torch.uint8, device="cuda")
    lib.orthogonalize(mats, outs, ws, stream=stream, **kw)      # a workspace of NaN bits
    torch.cuda.synchronize()
    return outs


def check(mats, outs, steps=5, **kw):
    for m, o in zip(mats, outs):
        want = M.polar(m, steps=steps, **kw)
        err = (o.double().cpu() - want).norm() / want.norm()
        assert err <= M.polar_tolerance(steps), (tuple(m.shape), float(err))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (7, 1), (2, 2), (3, 65), (64, 64), (63, 129),
                                   (200, 100), (128, 128), (129, 127), (256, 1024), (1025, 256),
                                   (300, 301)])
def test_shapes(lib, shape, dtype):
    m = matrix(*shape, seed=shape[0] * 7 + shape[1], dtype=dtype)
    check([m], run(lib, [m]))


@pytest.mark.parametrize("shape", [(64, 3001), (1531, 700), (1024, 1024), (513, 2055)])
def test_larger_shapes(lib, shape):
    m = matrix(*shape, seed=5)
    check([m], run(lib, [m]))


def test_large_square(lib):
    """Over one workgroup per CU; compared in 64 bits on the GPU."""
    m = matrix(2560, 3000, seed=6)
    (o,) = run(lib, [m])
    x = m.double()
    x = x / (x.norm() + 1e-7)
    for _ in range(5):
        s = x @ x.T.contiguous()
        x = M.COEFFS[0] * x + (M.COEFFS[1] * s + M.COEFFS[2] * (s @ s)) @ x
    assert (o.double() - x).norm() / x.norm() <= M.polar_tolerance(5)


@pytest.mark.parametrize("shapes", [[(4096, 4096)], [(2048, 8192)], [(8200, 2040), (3000, 4100)], [(1024, 8192)] * 2])
def test_largest_tiles(lib, shapes):
    """Launches on the largest tiles and split ones; the same bits again, and the value in 64 bits
    on the GPU."""
    mats = [matrix(*s, seed=i) for i, s in enumerate(shapes)]
    outs = run(lib, mats)
    for _ in range(2):
        for a, b in zip(outs, run(lib, mats)):
            assert M.same_bits(a, b)
    for m, o in zip(mats, outs):
        x = (m.T if m.shape[0] > m.shape[1] else m).double().contiguous()
        x = x / (x.norm() + 1e-7)
        for _ in range(5):
            s = x @ x.T.contiguous()
            x = M.COEFFS[0] * x + (M.COEFFS[1] * s + M.COEFFS[2] * (s @ s)) @ x
        x = x.T if m.shape[0] > m.shape[1] else x
        assert (o.double() - x).norm() / x.norm() <= M.polar_tolerance(5)


@pytest.mark.parametrize("shapes", [[(1024, 4096), (300, 320)], [(64, 200), (256, 8192)], [(700, 90), (4000, 513), (1300, 2600)],
                                    [(2048, 260), (260, 2048), (65, 66)], [(9000, 100), (120, 500)]])
def test_one_product_split_and_others_not(lib, shapes):
    """Launches whose long contractions are split over workgroups, next to short ones that are not."""
    mats = [matrix(*s, seed=i) for i, s in enumerate(shapes)]
    check(mats, run(lib, mats))


def test_many_matrices_one_call(lib):
    """More matrices than a launch holds, wide, tall, square and empty ones mixed."""
    shapes = [(32, 64), (64, 32), (0, 9), (33, 31), (1, 50)] * 11 + [(400, 150), (150, 400)]
    mats = [matrix(*s, seed=i) if s[0] else torch.empty(s, dtype=torch.bfloat16, device="cuda")
            for i, s in enumerate(shapes)]
    outs = run(lib, mats)
    check([m for m in mats if m.numel()], [o for o in outs if o.numel()])


@pytest.mark.parametrize("dtype,pitch,out_pitch", [(torch.bfloat16, 111, 105), (torch.float32, 104, 130),
                                                   (torch.float32, 103, 101)])
def test_pitches_and_guards(lib, dtype, pitch, out_pitch):
    """Rows inside wider ones, starting off any boundary; what lies between them stays."""
    m = matrix(90, 100, seed=8, dtype=dtype, pitch=pitch)
    flat = torch.full((90 * out_pitch + 3,), 7.0, dtype=torch.bfloat16, device="cuda")
    buf = flat[3:].view(90, out_pitch)
    before = flat.clone()
    run(lib, [m], outs=[buf[:, :100]])
    check([m], [buf[:, :100]])
    buf[:, :100] = 7.0
    assert M.same_bits(flat, before)


@pytest.mark.parametrize("steps,coeffs", [(1, M.COEFFS), (2, (1.875, -1.25, 0.375)), (3, M.COEFFS),
                                          (7, (1.5, -0.5, 0.0))])
def test_steps_and_coefficients(lib, steps, coeffs):
    mats = [matrix(130, 200, seed=9), matrix(200, 130, seed=10)]
    check(mats, run(lib, mats, steps=steps, coeffs=coeffs), steps=steps, coeffs=coeffs)


def test_eps_and_ranges(lib):
    """Values whose squares leave fp32's range, in both directions, and a norm near eps."""
    m = matrix(70, 90, seed=11, dtype=torch.float32)
    for scale, eps in ((1e25, 1e-7), (1e-10, 0.0), (1e-20, 0.0), (1.0, 0.05)):
        g = m * scale
        check([g], run(lib, [g], eps=eps), eps=eps)


def test_zero_matrix_and_special_values(lib):
    z = torch.zeros(50, 70, dtype=torch.bfloat16, device="cuda")
    (o,) = run(lib, [z])
    assert torch.equal(o.float().cpu(), torch.zeros(50, 70))
    good = matrix(60, 80, seed=12)
    for bad in (float("nan"), float("inf"), -float("inf")):
        g = matrix(80, 60, seed=13)
        g[17, 5] = bad
        a, b = run(lib, [g, good])
        assert torch.isnan(a).all()
        check([good], [b])                               # the other matrix of the call is untouched


def test_repeats_and_grouping_give_the_same_bits(lib):
    mats = [matrix(300, 500, seed=14), matrix(500, 260, seed=15)]
    first = run(lib, mats)
    again = run(lib, mats)
    for a, b in zip(first, again):
        assert M.same_bits(a, b)


def test_other_stream_and_graph(lib):
    mats = [matrix(150, 260, seed=16), matrix(260, 90, seed=17)]
    want = run(lib, mats)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(lib, mats, stream=s)
    for a, b in zip(want, got):
        assert M.same_bits(a, b)
    outs = [torch.empty_like(o) for o in want]
    ws = torch.empty(lib.orthogonalize_workspace(mats), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.orthogonalize(mats, outs, ws)
    for i in range(4):
        keep = [m.clone() for m in mats]
        for m in mats:
            m.mul_(-1.0 if i % 2 else 1.0)               # eager work between the replays
        for o in outs:
            o.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        eager = run(lib, mats)
        for a, b in zip(eager, outs):
            assert M.same_bits(a, b)
        for m, k in zip(mats, keep):
            m.copy_(k)


def test_refuses_a_small_workspace_on_the_device(lib):
    m = matrix(64, 64, seed=18)
    with pytest.raises(lib.FsdpError) as e:
        lib.orthogonalize([m], [torch.empty_like(m)], torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 2
    with pytest.raises(ValueError):
        lib.orthogonalize([m.T], [torch.empty_like(m)], torch.empty(256, dtype=torch.uint8, device="cuda"))
