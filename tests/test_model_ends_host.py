"""Host-side checks of the embedding, the dropout and the head's loss (no GPU, no kernel launched):
refusals, workspace sizes, and the definitions that the GPU tests compare with."""

import ctypes

import numpy as np
import pytest
import torch

import model_ends_cases as E

FAKE = 1 << 40     # 256-byte aligned, never dereferenced: validation fails first
INVALID, RANGE, ALIAS, UNSUPPORTED = 1, 2, 3, 4


def at(i):
    return FAKE + (i << 36)


def refused(lib, call, args, status):
    assert getattr(lib._lib, call)(ctypes.byref(args), None) == status, (call, lib._lib.fsdp_last_error())
    assert lib._lib.fsdp_last_error()


def changed(args, kw):
    for k, v in kw.items():
        setattr(args, k, v)
    return args


def embed_args(lib, **kw):
    return changed(lib._EmbeddingArgs(tokens=at(0), weight=at(1), out=at(2), rows=4, vocab=50, dim=32,
                                      weight_pitch=32, out_pitch=32, scale=1.0, dtype=1), kw)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), RANGE), (dict(rows=1 << 22), RANGE), (dict(dim=0), RANGE), (dict(dim=(1 << 24) + 1), RANGE),
    (dict(vocab=0), RANGE), (dict(vocab=1 << 22), RANGE), (dict(dtype=2), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(tokens=None), INVALID), (dict(tokens=at(0) + 4), INVALID), (dict(weight=None), INVALID),
    (dict(weight=at(1) + 1), INVALID), (dict(out=None), INVALID), (dict(out=at(2) + 1), INVALID),
    (dict(weight_pitch=31), RANGE), (dict(out_pitch=31), RANGE), (dict(out_pitch=(1 << 32) + 1), RANGE),
    (dict(out=at(1) + 64 * 49), ALIAS), (dict(out=at(0)), ALIAS),
])
def test_embedding_refuses(lib, change, status):
    refused(lib, "fsdp_embedding", embed_args(lib, **change), status)


def embed_back_args(lib, **kw):
    return changed(lib._EmbeddingBackwardArgs(
        tokens=at(0), dy=at(1), dweight=at(2), workspace=at(3), workspace_bytes=1 << 20, rows=4, vocab=50, dim=32,
        dy_pitch=32, dweight_pitch=32, padding_idx=-1, scale=1.0, dtype=0, accumulate=0), kw)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), RANGE), (dict(vocab=0), RANGE), (dict(vocab=1 << 22), RANGE), (dict(dim=0), RANGE),
    (dict(dtype=9), UNSUPPORTED), (dict(scale=float("nan")), INVALID), (dict(accumulate=2), INVALID),
    (dict(tokens=None), INVALID), (dict(dy=None), INVALID), (dict(dweight=None), INVALID),
    (dict(dy=at(1) + 2), INVALID), (dict(dweight=at(2) + 2), INVALID), (dict(dy_pitch=1), RANGE),
    (dict(dweight_pitch=1), RANGE), (dict(workspace=None), INVALID), (dict(workspace=at(3) + 8), INVALID),
    (dict(workspace_bytes=16), RANGE), (dict(dweight=at(1)), ALIAS), (dict(workspace=at(2)), ALIAS),
    (dict(workspace=at(0)), ALIAS),
])
def test_embedding_backward_refuses(lib, change, status):
    refused(lib, "fsdp_embedding_backward", embed_back_args(lib, **change), status)


def drop_args(lib, **kw):
    return changed(lib._DropoutArgs(x=at(0), out=at(1), rows=4, dim=32, x_pitch=32, residual_pitch=32, out_pitch=32,
                                    seed=1, offset=2, p=0.1, dtype=1), kw)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), RANGE), (dict(dim=0), RANGE), (dict(dtype=3), UNSUPPORTED), (dict(p=-0.1), INVALID),
    (dict(p=1.01), INVALID), (dict(p=float("nan")), INVALID), (dict(x=None), INVALID), (dict(out=None), INVALID),
    (dict(x=at(0) + 1), INVALID), (dict(residual=at(2) + 1), INVALID), (dict(x_pitch=31), RANGE),
    (dict(out_pitch=31), RANGE), (dict(residual=at(2), residual_pitch=31), RANGE), (dict(counter=at(3) + 4), INVALID),
    (dict(out=at(0) + 2), ALIAS), (dict(out=at(0), out_pitch=33), ALIAS), (dict(residual=at(1) + 64), ALIAS),
    (dict(counter=at(1)), ALIAS), (dict(residual=at(0) + 64, out=at(0) + 64), ALIAS),
])
def test_dropout_refuses(lib, change, status):
    refused(lib, "fsdp_dropout", drop_args(lib, **change), status)


def loss_args(lib, **kw):
    return changed(lib._LossArgs(
        hidden=at(0), weight=at(1), targets=at(2), loss=at(3), losses=at(4), dhidden=at(5), dweight=at(6),
        workspace=at(7), workspace_bytes=1 << 30, rows=10, vocab=50, dim=32, hidden_pitch=32, weight_pitch=32,
        dhidden_pitch=32, dweight_pitch=32, piece=0, grad_scale=1.0, reduction=0), kw)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), RANGE), (dict(rows=1 << 22), RANGE), (dict(vocab=0), RANGE), (dict(vocab=1 << 22), RANGE),
    (dict(dim=0), RANGE), (dict(dim=(1 << 20) + 1), RANGE), (dict(piece=-1), RANGE),
    (dict(vocab=1 << 20, dim=1 << 16, weight_pitch=1 << 16), RANGE),
    (dict(grad_scale=float("inf")), INVALID), (dict(reduction=2), INVALID), (dict(hidden=None), INVALID),
    (dict(weight=None), INVALID), (dict(targets=None), INVALID), (dict(loss=None), INVALID),
    (dict(hidden=at(0) + 1), INVALID), (dict(targets=at(2) + 4), INVALID), (dict(loss=at(3) + 2), INVALID),
    (dict(losses=at(4) + 2), INVALID), (dict(dhidden=at(5) + 1), INVALID), (dict(dweight=at(6) + 1), INVALID),
    (dict(hidden_pitch=31), RANGE), (dict(weight_pitch=31), RANGE), (dict(dhidden_pitch=31), RANGE),
    (dict(dweight_pitch=31), RANGE), (dict(workspace=None), INVALID), (dict(workspace=at(7) + 16), INVALID),
    (dict(workspace_bytes=100), RANGE), (dict(dhidden=at(0)), ALIAS), (dict(dweight=at(1) + 64), ALIAS),
    (dict(loss=at(4)), ALIAS), (dict(losses=at(2)), ALIAS), (dict(workspace=at(6)), ALIAS),
])
def test_loss_refuses(lib, change, status):
    refused(lib, "fsdp_linear_cross_entropy", loss_args(lib, **change), status)


def test_null_and_empty(lib):
    for call in ("fsdp_embedding", "fsdp_embedding_backward", "fsdp_dropout", "fsdp_linear_cross_entropy"):
        assert getattr(lib._lib, call)(None, None) == INVALID
    need = ctypes.c_int64()
    assert lib._lib.fsdp_embedding_backward_workspace(4, 4, 4, None) == INVALID
    assert lib._lib.fsdp_embedding_backward_workspace(4, 0, 4, ctypes.byref(need)) == RANGE
    assert lib._lib.fsdp_linear_cross_entropy_workspace(None, ctypes.byref(need)) == INVALID
    assert lib._lib.fsdp_linear_cross_entropy_workspace(ctypes.byref(loss_args(lib)), None) == INVALID
    assert lib._lib.fsdp_linear_cross_entropy_workspace(ctypes.byref(loss_args(lib, dim=0)), ctypes.byref(need)) == RANGE
    assert lib._lib.fsdp_embedding(ctypes.byref(embed_args(lib, rows=0, tokens=None, weight=None, out=None)), None) == 0
    assert lib._lib.fsdp_dropout(ctypes.byref(drop_args(lib, rows=0, x=None, out=None)), None) == 0
    assert lib._lib.fsdp_embedding_backward(ctypes.byref(embed_back_args(
        lib, rows=0, tokens=None, dy=None, accumulate=1, workspace=None, workspace_bytes=0)), None) == 0


def test_workspaces(lib):
    meta = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="meta")  # noqa: E731
    assert lib.embedding_backward_workspace(8192, 32000, 4096) >= 4 * (8192 + 32001)
    x, w = meta(8192, 4096), meta(32000, 4096)
    none = lib.linear_cross_entropy_workspace(x, w, dhidden=False, dweight=False)
    both = lib.linear_cross_entropy_workspace(x, w)
    assert 8192 * 4096 * 2 <= none < both <= none + (1 << 30) + (1 << 26)
    # pieces: a smaller scratch, and dweight's sums between them
    part = lib.linear_cross_entropy_workspace(x, w, dweight=False, piece=1024)
    assert part < both
    assert lib.linear_cross_entropy_workspace(x, w, piece=1024) >= 8192 * 4096 * 2 + 32000 * 4096 * 4
    # a vocabulary so large that a scratch of all rows would pass 1 GiB
    x, w = meta(1 << 17, 64), meta(1 << 17, 64)
    assert lib.linear_cross_entropy_workspace(x, w) < (3 << 30)


def test_binding_refuses(lib):
    bf, i64 = torch.bfloat16, torch.int64
    cpu, tokens, ws = torch.zeros(4, 8), torch.zeros(4, dtype=i64), torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError):
        lib.embedding(tokens, cpu, torch.zeros(4, 8))
    with pytest.raises(TypeError):
        lib.embedding(tokens, cpu.half(), cpu)
    with pytest.raises(ValueError):
        lib.embedding(tokens, cpu[0], cpu)
    with pytest.raises(ValueError):
        lib.embedding_backward(tokens, cpu, cpu, ws)
    with pytest.raises(TypeError):
        lib.embedding_backward(tokens, cpu, cpu.int(), ws)
    with pytest.raises(ValueError):
        lib.dropout(cpu, cpu, 0.1, 1)
    with pytest.raises(TypeError):
        lib.dropout(cpu.half(), cpu, 0.1, 1)
    with pytest.raises(ValueError):
        lib.dropout(cpu[0], cpu, 0.1, 1)
    x = cpu.to(bf)
    with pytest.raises(ValueError):
        lib.linear_cross_entropy(x, x, tokens, cpu, ws)
    with pytest.raises(ValueError):
        lib.linear_cross_entropy(x, x, tokens, cpu, ws, reduction="none")
    with pytest.raises(TypeError):
        lib.linear_cross_entropy(cpu, x, tokens, cpu, ws)
    with pytest.raises(ValueError):
        lib.linear_cross_entropy(x, x[:, :4], tokens, cpu, ws)
    with pytest.raises(ValueError):
        lib.linear_cross_entropy_workspace(x, x[:, :4])
    with pytest.raises(TypeError):
        lib.linear_cross_entropy_workspace(cpu, x)


def test_philox_known_answers():
    """Published known answers of Philox 4 x 32 with 10 and 7 rounds."""
    ones = 0xFFFFFFFF
    for rounds, counter, key, want in (
            (10, [0] * 4, [0] * 2, [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]),
            (10, [ones] * 4, [ones] * 2, [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]),
            (10, [0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0],
             [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1])):
        got = E.philox([np.array([c]) for c in counter], key, rounds)
        assert [int(g[0]) for g in got] == want


def test_dropout_definition():
    """The kept share and the mean are those of p; the bits of two offsets are unlike."""
    x = torch.ones(400, 1003)
    for p in (0.0, 0.1, 0.5, 1.0):
        y = E.dropout(x, p, 12345, 6)
        n = x.numel()
        kept = float((y != 0).double().mean())
        assert abs(kept - (1 - round(p * 65536) / 65536)) <= 5 * (p * (1 - p) / n) ** 0.5 + 1e-12
        if p < 1:
            assert abs(float(y.double().mean()) - 1.0) <= 5 * (p / (1 - p) / n) ** 0.5 + 1e-6
    a, b = E.dropout_bits(50, 64, 1, 0), E.dropout_bits(50, 64, 1, 1)
    assert float((a == b).mean()) < 0.01
    # a part of the rows, and wider rows, have the same bits
    assert np.array_equal(E.dropout_bits(20, 64, 1, 0, row0=30), a[30:])
    assert np.array_equal(E.dropout_bits(50, 100, 1, 0)[:, :64], a)


def test_loss_gradient_formulas_against_differences():
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(5, 7, generator=gen, dtype=torch.float64)
    w = torch.randn(6, 7, generator=gen, dtype=torch.float64)
    t = torch.tensor([0, 5, -100, 2, 6])                 # two rows do not count
    for mean in (True, False):
        d = E.loss(x, w, t, 0.7, mean)
        f = lambda x, w: float(0.7 * E.loss(x, w, t, 1.0, mean)["loss"][0])  # noqa: E731
        h = 1e-5
        for a, grad, make in ((x, d["dhidden"][0], lambda s: (x + s, w)), (w, d["dweight"][0], lambda s: (x, w + s))):
            for at_ in np.ndindex(*a.shape):
                step = torch.zeros_like(a)
                step[at_] = h
                # central differences: O(h^2) truncation, 1e-16 / h of rounding
                assert abs((f(*make(step)) - f(*make(-step))) / (2 * h) - grad[at_]) < 1e-8
    assert float(d["losses"][0][2]) == 0 and float(d["dhidden"][0][[2, 4]].abs().max()) == 0


def test_embedding_gradient_formula_against_differences():
    gen = torch.Generator().manual_seed(4)
    w = torch.randn(5, 3, generator=gen, dtype=torch.float64)
    tokens = torch.tensor([[1, 4, 1], [9, -1, 3]])
    dy = torch.randn(6, 3, generator=gen, dtype=torch.float64)
    want, _, n = E.embedding_backward(tokens, dy, 5, 2.5, padding=3)
    flat = tokens.reshape(-1)
    ok = (flat >= 0) & (flat < 5)
    f = lambda w: float((torch.where(ok[:, None], w[flat.clamp(0, 4)] * 2.5, torch.zeros(1, dtype=torch.float64)) * dy).sum())  # noqa: E731
    for at_ in np.ndindex(5, 3):
        step = torch.zeros_like(w)
        step[at_] = 1e-4
        d = (f(w + step) - f(w - step)) / 2e-4
        assert abs(d - want[at_]) < 1e-9 or at_[0] == 3          # the padding row's gradient is none
    assert n.tolist() == [0, 2, 0, 0, 1] and float(want[3].abs().max()) == 0
