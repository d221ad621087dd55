"""The element-wise halves of the Muon step against their formulas in 64 bits."""

import pytest
import torch

import muon_cases as M
from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]


def window(u):
    return slice(u.shard_begin, u.shard_begin + u.shard_valid)


def off(n, dtype, shift):
    """An n-element tensor that starts `shift` elements off an allocation's start, in a buffer of
    sevens whose ends guard it."""
    buf = torch.full((n + shift + 5,), 7.0, dtype=dtype, device="cuda")
    return buf, buf[shift:shift + n]


def close(got, want, size, rel):
    """|got - want| <= rel * size element by element (size: what the roundings are relative to)."""
    d = (got.double() - want).abs()
    assert bool((d <= rel * size).all()), float((d / size.clamp_min(1e-300)).max())


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shapes,F,rank,rows,shift", [
    ([(5, 7), (3,)], 4, 1, 4, 0), ([(1,)], 1, 0, 1, 0), ([(33, 77), (1001,)], 7, 3, 7, 1),
    ([(256, 1024), (1024,), (1024, 256), (256,)], 4, 1, 4, 0), ([(1000, 1037)], 8, 7, 8, 0),
    ([(1000, 1037)], 8, 5, 8, 3), ([(300, 301)], 2, 1, 11, 2), ([(300, 300)], 3, 0, 16, 0),
    ([(97, 89)], 64, 63, 64, 1), ([(2048, 2048)], 1, 0, 2, 0),
    ([(4099, 2051)], 2, 1, 3, 0), ([(4099, 2051)], 2, 1, 9, 0), ([(4099, 2051)], 2, 0, 1, 0),
])
def test_reduce_momentum(lib, shapes, F, rank, rows, shift, nesterov):
    u = lib.Unit(shapes, F, rank)
    torch.manual_seed(rank + rows)
    grads = [off(u.U, torch.bfloat16, shift)[1].normal_(0, 1e-3) for _ in range(rows)]
    mbuf, m = off(u.shard_valid, torch.float32, shift)
    m.normal_(0, 1e-3)
    ubuf, upd = off(u.shard_valid, torch.bfloat16, shift)
    m0 = m.double().clone()
    hp = lib.MuonHparams(momentum=0.95, nesterov=nesterov)
    lib.reduce_momentum_shard(u, grads, m, upd, hp)
    torch.cuda.synchronize()
    mine = [g[window(u)].double() for g in grads]
    g = M.mean_rows(mine, 1.0 / rows)
    want = 0.95 * m0 + g
    # rows - 1 adds, the scale, 1/rows and 0.95 as fp32, one product, one add: each 2^-24 of at
    # most the sum of magnitudes; then the bf16 rounding
    mags = M.mean_rows([x.abs() for x in mine], 1.0 / rows)
    size = 0.95 * m0.abs() + mags
    close(m, want, size, (rows + 5) * M.F32)
    up = g + 0.95 * want if nesterov else want
    # the rounding of the computed value, which is itself off by the fp32 part; a subnormal's
    # half step is far below
    close(upd, up, (1 + M.BF16) * (rows + 9) * M.F32 * (mags + 0.95 * size) + M.BF16 * up.abs(), 1.0)
    for buf, n in ((mbuf, u.shard_valid), (ubuf, u.shard_valid)):
        assert bool((buf[:shift] == 7).all()) and bool((buf[shift + n:] == 7).all())


def test_reduce_momentum_scale_specials_and_repeat(lib):
    u = lib.Unit([(1000,)], 2, 1)
    grads = [torch.randn(1000, device="cuda").bfloat16() for _ in range(2)]
    grads[1][700], grads[0][800] = float("inf"), float("nan")
    m = torch.zeros(500, device="cuda")
    upd = torch.empty(500, dtype=torch.bfloat16, device="cuda")
    lib.reduce_momentum_shard(u, grads, m, upd, lib.MuonHparams(momentum=0.0), grad_scale=3.0)
    torch.cuda.synchronize()
    want = (grads[0].float() + grads[1].float())[500:] * 3.0
    assert torch.equal(m.nan_to_num(7.0, 9.0), want.nan_to_num(7.0, 9.0))
    # g + 0 * m: an infinite momentum makes the Nesterov update NaN, as the formula does
    assert torch.isinf(m[200]) and torch.isnan(m[300])
    assert torch.isnan(upd[[200, 300]]).all() and int(torch.isfinite(upd).sum()) == 498


@pytest.mark.parametrize("shapes,F,rank,shift,emit", [
    ([(5, 7), (3,)], 4, 1, 0, True), ([(1,)], 1, 0, 0, True), ([(33, 77), (0, 4), (1001,), (2, 3)], 2, 1, 1, True),
    ([(256, 1024), (1024,), (1024, 256), (256,)], 4, 1, 0, True), ([(1000, 1037)], 8, 7, 0, False),
    ([(7,)] * 150 + [(400, 33)], 1, 0, 0, True), ([(3, 5)] * 333, 3, 2, 2, True),
    ([(2000, 1024), (999,)], 2, 0, 0, True), ([(4099, 2051), (5,)], 2, 1, 0, True),
])
def test_apply(lib, shapes, F, rank, shift, emit):
    u = lib.Unit(shapes, F, rank)
    torch.manual_seed(rank)
    bufs = [off(n, torch.bfloat16, (shift + i) % 4) for i, n in enumerate(u.numels)]
    ts = [t.normal_(0, 0.02) for _, t in bufs]
    scales = [1.0 + 0.37 * (i % 3) for i in range(len(ts))]
    pbuf, p = off(u.shard_valid, torch.float32, shift)
    p.normal_(0, 0.02)
    wbuf, w = off(u.shard_valid, torch.bfloat16, shift)
    p0 = p.double().clone()
    hp = lib.MuonHparams(lr=0.02, weight_decay=0.01)
    lib.muon_apply_shard(u, ts, scales, p, w if emit else None, hp)
    torch.cuda.synchronize()
    flat = torch.cat([k * t.double() for k, t in zip(scales, ts)])[window(u)]
    want = p0 - 0.02 * (flat + 0.01 * p0)
    # three fp32 constants, three products, two adds
    size = p0.abs() + 0.02 * (flat.abs() + 0.01 * p0.abs())
    close(p, want, size, 8 * M.F32)
    if emit:
        assert M.same_bits(w, p.bfloat16())
    else:
        assert bool((wbuf == 7).all())
    for buf in (pbuf, wbuf):
        assert bool((buf[:shift] == 7).all()) and bool((buf[shift + u.shard_valid:] == 7).all())


def test_step_over_all_ranks_matches_the_whole_unit(lib):
    """F ranks' momentum, the gathered update, the orthogonalisation and F ranks' apply give the
    unsharded step: windows, gather and segments agree."""
    shapes, F = [(96, 200), (200,), (200, 96)], 4
    torch.manual_seed(0)
    units = [lib.Unit(shapes, F, r) for r in range(F)]
    U, S = units[0].U, units[0].S
    grads = [(1e-3 * torch.randn(U, device="cuda")).bfloat16() for _ in range(F)]
    master = 0.02 * torch.randn(U, device="cuda")
    hp = lib.MuonHparams(lr=0.02, weight_decay=0.1)
    shards = []
    for u in units:
        m = torch.zeros(u.shard_valid, device="cuda")
        upd = torch.zeros(S, dtype=torch.bfloat16, device="cuda")
        lib.reduce_momentum_shard(u, grads, m, upd[:u.shard_valid], hp)
        shards.append(upd)
    outs = [torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in shapes]
    lib.cast_unflatten(units[0], shards, outs)
    mats = [o for o in outs if o.dim() == 2]
    orth = [torch.empty_like(m) for m in mats]
    ws = torch.empty(lib.orthogonalize_workspace(mats), dtype=torch.uint8, device="cuda")
    lib.orthogonalize(mats, orth, ws)
    final = [orth[0], outs[1], orth[1]]
    scales = [max(1.0, s[0] / s[1]) ** 0.5 if len(s) == 2 else 1.0 for s in shapes]
    new = []
    for u in units:
        p = master[window(u)].clone()
        lib.muon_apply_shard(u, final, scales, p, None, hp)
        new.append(p)
    got = torch.cat(new)
    flat = torch.cat([k * t.double().reshape(-1) for k, t in zip(scales, final)])
    want = master.double() - 0.02 * (flat + 0.1 * master.double())
    close(got, want, master.double().abs() + 0.02 * flat.abs() + 0.002 * master.double().abs(), 8 * M.F32)
    for m, o in zip(mats, orth):
        ref = M.polar(m)
        assert (o.double().cpu() - ref).norm() / ref.norm() <= M.polar_tolerance(5)


def test_streams_and_graph(lib):
    u = lib.Unit([(256, 300), (77,)], 2, 1)
    grads = [(1e-3 * torch.randn(u.U, device="cuda")).bfloat16() for _ in range(2)]
    ts = [torch.randn(n, device="cuda").bfloat16() for n in u.numels]
    hp = lib.MuonHparams()

    def state():
        torch.manual_seed(1)
        return (torch.randn(u.shard_valid, device="cuda"), torch.randn(u.shard_valid, device="cuda"),
                torch.empty(u.shard_valid, dtype=torch.bfloat16, device="cuda"),
                torch.empty(u.shard_valid, dtype=torch.bfloat16, device="cuda"))

    def step(s, stream=None):
        m, p, upd, w = s
        lib.reduce_momentum_shard(u, grads, m, upd, hp, stream=stream)
        lib.muon_apply_shard(u, ts, [1.0, 2.0], p, w, hp, stream=stream)

    eager = state()
    captured, side = state(), state()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    step(side, st)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(captured)
    for _ in range(3):
        g.replay()
        step(eager)
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert M.same_bits(a, b)
    one = state()
    step(one)
    torch.cuda.synchronize()
    for a, b in zip(one, side):
        assert M.same_bits(a, b)


def test_example_learns():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "muon_block.py")
    spec = importlib.util.spec_from_file_location("muon_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses = example.train(steps=12)
    assert all(b == b for b in losses) and losses[-1] < 0.5 * losses[0]
