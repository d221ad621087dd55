"""Host-side checks of the Muon step and the RMS norm (no GPU, no kernel launched): refusals,
workspace sizes, and the definitions the GPU tests compare with."""

import ctypes

import numpy as np
import pytest
import torch

import muon_cases as M

FAKE = 1 << 40     # 256-byte aligned, never dereferenced: validation fails first
I64 = ctypes.c_int64
INVALID, RANGE, ALIAS, UNSUPPORTED = 1, 2, 3, 4


def i64s(*v):
    return (I64 * max(1, len(v)))(*v)


def ortho(lib, shapes, *, dtype=1, mats=None, outs=None, ld=None, out_ld=None, ws=FAKE + (1 << 38),
          ws_bytes=1 << 36, steps=5, coeffs=M.COEFFS, eps=1e-7):
    n = len(shapes)
    rows, cols = i64s(*[s[0] for s in shapes]), i64s(*[s[1] for s in shapes])
    mats = [FAKE + (i << 30) for i in range(n)] if mats is None else mats
    outs = [FAKE + ((i + n) << 30) for i in range(n)] if outs is None else outs
    return lib._lib.fsdp_orthogonalize(
        n, dtype, lib._ptr_array(mats), rows, cols, i64s(*(ld or [s[1] for s in shapes])),
        lib._ptr_array(outs), i64s(*(out_ld or [s[1] for s in shapes])), ws, ws_bytes, steps,
        None if coeffs is None else (ctypes.c_double * 3)(*coeffs), eps, None)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(steps=0), INVALID), (dict(steps=65), INVALID),
    (dict(coeffs=None), INVALID), (dict(coeffs=(1.0, float("nan"), 0.0)), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(mats=[FAKE, 0]), INVALID), (dict(outs=[0, FAKE]), INVALID),
    (dict(mats=[FAKE + 1, FAKE + (1 << 30)]), INVALID),
    (dict(outs=[FAKE + (2 << 30) + 1, FAKE + (3 << 30)]), INVALID),
    (dict(ld=[99, 200]), RANGE), (dict(out_ld=[100, 199]), RANGE),
    (dict(ld=[1 << 41, 200]), RANGE),
    (dict(ws=0), INVALID), (dict(ws=FAKE + (1 << 38) + 16), INVALID),
    (dict(ws_bytes=1024), RANGE),
    (dict(outs=[FAKE + 64, FAKE + (3 << 30)]), ALIAS),
    (dict(outs=[FAKE + (2 << 30), FAKE + (2 << 30) + 2]), ALIAS),
    (dict(ws=FAKE), ALIAS),
])
def test_orthogonalize_refuses(lib, change, status):
    assert ortho(lib, [(50, 100), (300, 200)], **change) == status
    assert lib._lib.fsdp_last_error()


def test_orthogonalize_refuses_sizes(lib):
    assert ortho(lib, [(-1, 4)]) == INVALID
    assert ortho(lib, [(4, (1 << 20) + 1)]) == RANGE
    assert ortho(lib, [(0, 7), (5, 0)], mats=[0, 0], outs=[0, 0], ws=0, ws_bytes=0) == 0
    assert ortho(lib, []) == 0
    need = I64()
    assert lib._lib.fsdp_orthogonalize_workspace(1, i64s(4), i64s(4), None) == INVALID
    assert lib._lib.fsdp_orthogonalize_workspace(-1, i64s(4), i64s(4), ctypes.byref(need)) == INVALID
    assert lib._lib.fsdp_orthogonalize_workspace(1, None, i64s(4), ctypes.byref(need)) == INVALID


def test_orthogonalize_workspace_covers_the_operands(lib):
    for shapes in ([(1, 1)], [(64, 64)], [(515, 1373), (2049, 771)], [(4096, 4096)] * 4, [(0, 5)]):
        mats = [torch.empty(s, dtype=torch.bfloat16, device="meta") for s in shapes]
        need = lib.orthogonalize_workspace(mats)
        least = sum(2 * r * c + 2 * min(r, c) ** 2 for r, c in shapes)
        assert need >= least
        assert (need == 0) == (least == 0)


def muon_hp(lib, **kw):
    base = dict(lr=0.02, momentum=0.95, weight_decay=0.01, grad_scale=0.25, nesterov=1)
    base.update(kw)
    return lib._MuonHparams(**base)


BAD_HP = [dict(lr=-1.0), dict(lr=float("nan")), dict(momentum=1.0), dict(momentum=-0.1),
          dict(momentum=float("nan")), dict(nesterov=2), dict(weight_decay=float("inf")),
          dict(grad_scale=float("nan"))]


def test_momentum_refuses(lib):
    u = lib.Unit([(4096,)], 4, 1)
    grads = [FAKE + (k << 20) for k in range(4)]
    m, w = FAKE + (1 << 30), FAKE + (2 << 30)

    def call(n=4, g=grads, m=m, w=w, unit=u.handle, **hp):
        arr = None if g is None else lib._ptr_array(g)
        h = muon_hp(lib, **hp)
        return lib._lib.fsdp_reduce_momentum_shard(unit, n, arr, m, w, ctypes.byref(h), None)

    assert call(unit=None) == INVALID
    assert call(n=0) == INVALID and call(n=65) == INVALID
    assert call(g=None) == INVALID
    assert call(g=grads[:3] + [0]) == INVALID and call(g=[FAKE + 1] + grads[1:]) == INVALID
    assert call(m=0) == INVALID and call(m=m + 2) == INVALID
    assert call(w=0) == INVALID and call(w=w + 1) == INVALID
    assert call(w=m) == ALIAS and call(m=FAKE + 2 * 1024) == ALIAS
    for bad in BAD_HP:
        assert call(**bad) == INVALID, bad
    assert lib._lib.fsdp_reduce_momentum_shard(u.handle, 4, lib._ptr_array(grads), m, w, None,
                                               None) == INVALID
    empty = lib.Unit([(3,)], 4, 3)                       # a window of pad only
    assert empty.shard_valid == 0
    assert call(unit=empty.handle, g=None, m=0, w=0) == 0


def test_apply_refuses(lib):
    u = lib.Unit([(10, 100), (500,), (7, 3)], 2, 0)      # the last tensor is outside the window
    tensors = [FAKE + (k << 20) for k in range(3)]
    p, w = FAKE + (1 << 30), FAKE + (2 << 30)

    def call(t=tensors, s=(1.0, 1.0, 1.0), p=p, w=w, unit=u.handle, **hp):
        arr = None if t is None else lib._ptr_array(t)
        sc = None if s is None else (ctypes.c_double * 3)(*s)
        h = muon_hp(lib, **hp)
        return lib._lib.fsdp_muon_apply_shard(unit, arr, sc, p, w, ctypes.byref(h), None)

    assert call(unit=None) == INVALID
    assert call(t=None) == INVALID and call(s=None) == INVALID
    assert call(t=[0] + tensors[1:]) == INVALID and call(t=[FAKE + 1] + tensors[1:]) == INVALID
    assert call(s=(float("inf"), 1.0, 1.0)) == INVALID
    assert call(p=0) == INVALID and call(p=p + 2) == INVALID and call(w=w + 1) == INVALID
    assert call(w=p) == ALIAS and call(p=FAKE) == ALIAS
    for bad in BAD_HP:
        assert call(**bad) == INVALID, bad
    empty = lib.Unit([(1,), (1,), (1,)], 4, 3)
    assert call(unit=empty.handle, t=None, s=None, p=0, w=0) == 0


def norm_args(lib, **kw):
    a = lib._NormArgs(x=FAKE, weight=FAKE + (1 << 30), out=FAKE + (2 << 30), rows=4, dim=32,
                      x_pitch=32, residual_pitch=32, residual_out_pitch=32, out_pitch=32,
                      eps=1e-6, dtype=1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), RANGE), (dict(rows=1 << 22), RANGE), (dict(dim=0), RANGE),
    (dict(dim=(1 << 24) + 1), RANGE), (dict(dtype=2), UNSUPPORTED), (dict(eps=-1e-9), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(x=None), INVALID), (dict(x=FAKE + 1), INVALID),
    (dict(weight=None), INVALID), (dict(out=None), INVALID), (dict(out=FAKE + (2 << 30) + 1), INVALID),
    (dict(x_pitch=31), RANGE), (dict(out_pitch=31), RANGE), (dict(x_pitch=(1 << 32) + 1), RANGE),
    (dict(residual=FAKE + (3 << 30)), INVALID), (dict(residual_out=FAKE + (3 << 30)), INVALID),
    (dict(residual=FAKE + (3 << 30), residual_out=FAKE + (4 << 30), residual_pitch=8), RANGE),
    (dict(residual=FAKE + (3 << 30), residual_out=FAKE + (3 << 30)), ALIAS),
    (dict(out=FAKE), ALIAS), (dict(rstd=FAKE + (2 << 30)), ALIAS), (dict(rstd=FAKE + 2), INVALID),
    (dict(scales=FAKE + 2), INVALID), (dict(scales=FAKE + (1 << 30)), ALIAS),
])
def test_norm_refuses(lib, change, status):
    a = norm_args(lib, **change)
    assert lib._lib.fsdp_rms_norm(ctypes.byref(a), None) == status
    assert lib._lib.fsdp_last_error()


def back_args(lib, **kw):
    a = lib._NormBackwardArgs(dy=FAKE, x=FAKE + (1 << 30), weight=FAKE + (2 << 30),
                              rstd=FAKE + (3 << 30), dx=FAKE + (4 << 30), dweight=FAKE + (5 << 30),
                              workspace=FAKE + (6 << 30), workspace_bytes=4 * 32 * 4, rows=4,
                              dim=32, dy_pitch=32, x_pitch=32, dresidual_pitch=32, dx_pitch=32,
                              dtype=0)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), RANGE), (dict(dim=0), RANGE), (dict(dtype=7), UNSUPPORTED),
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(weight=None), INVALID),
    (dict(rstd=None), INVALID), (dict(dx=None), INVALID), (dict(dx=FAKE + (4 << 30) + 2), INVALID),
    (dict(dresidual=FAKE + 3), INVALID), (dict(workspace=None), INVALID),
    (dict(workspace=FAKE + (6 << 30) + 8), INVALID), (dict(workspace_bytes=4), RANGE),
    (dict(dy_pitch=1), RANGE), (dict(dx_pitch=1), RANGE), (dict(dx=FAKE), ALIAS),
    (dict(dweight=FAKE + (2 << 30)), ALIAS), (dict(workspace=FAKE + (4 << 30)), ALIAS),
])
def test_norm_backward_refuses(lib, change, status):
    a = back_args(lib, **change)
    assert lib._lib.fsdp_rms_norm_backward(ctypes.byref(a), None) == status
    assert lib._lib.fsdp_last_error()


def test_norm_empty_and_null(lib):
    a = norm_args(lib, rows=0, x=None, weight=None, out=None)
    assert lib._lib.fsdp_rms_norm(ctypes.byref(a), None) == 0
    assert lib._lib.fsdp_rms_norm(None, None) == INVALID
    b = back_args(lib, rows=0, dy=None, x=None, weight=None, rstd=None, dx=None, dweight=None,
                  workspace=None, workspace_bytes=0)
    assert lib._lib.fsdp_rms_norm_backward(ctypes.byref(b), None) == 0
    assert lib._lib.fsdp_rms_norm_backward(None, None) == INVALID
    assert lib._lib.fsdp_rms_norm_backward_workspace(1, 1, None) == INVALID
    assert lib.rms_norm_backward_workspace(0, 100) == 0
    assert lib.rms_norm_backward_workspace(3, 100) >= 400        # a row of fp32 sums, at least


def test_binding_refuses(lib):
    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        lib.rms_norm(cpu, torch.zeros(8), torch.zeros(4, 8))
    with pytest.raises(TypeError):
        lib.rms_norm(cpu.half(), torch.zeros(8), torch.zeros(4, 8))
    with pytest.raises(ValueError):
        lib.rms_norm(cpu[0], torch.zeros(8), torch.zeros(8))
    with pytest.raises(ValueError):
        lib.rms_norm(cpu, torch.zeros(8), torch.zeros(4, 8), residual=cpu)
    with pytest.raises(TypeError):
        lib.orthogonalize([cpu.half()], [cpu.bfloat16()], torch.zeros(1, dtype=torch.uint8))
    with pytest.raises(ValueError):
        lib.orthogonalize([cpu], [], torch.zeros(1, dtype=torch.uint8))
    with pytest.raises(ValueError):
        lib.orthogonalize([cpu], [cpu.bfloat16()], torch.zeros(1, dtype=torch.uint8))
    u = lib.Unit([(4, 8)], 1, 0)
    with pytest.raises(ValueError):
        lib.muon_apply_shard(u, [], [], cpu, None, lib.MuonHparams())
    with pytest.raises(ValueError):
        lib.reduce_momentum_shard(u, [], cpu, cpu, lib.MuonHparams())


def test_norm_gradient_formula_against_differences():
    gen = torch.Generator().manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, dy, eps = r(5, 11), 1 + 0.1 * r(11), r(5, 11), 1e-3
    f = lambda x, w: (M.norm_forward(x, w, eps)[0] * dy).sum()  # noqa: E731
    dx, dw = M.norm_backward(dy, x, w, M.norm_forward(x, w, eps)[1])
    h = 1e-5
    for at in np.ndindex(5, 11):
        step = torch.zeros_like(x)
        step[at] = h
        # central differences: O(h^2) truncation, 1e-16 / h of rounding
        assert abs((f(x + step, w) - f(x - step, w)) / (2 * h) - dx[at]) < 1e-8
    for j in range(11):
        step = torch.zeros_like(w)
        step[j] = h
        assert abs((f(x, w + step) - f(x, w - step)) / (2 * h) - dw[j]) < 1e-8


def test_polar_definition_against_singular_values():
    """The composed polynomial acts on the singular values alone."""
    gen = torch.Generator().manual_seed(4)
    for shape in ((20, 50), (50, 20), (7, 7), (1, 9)):
        g = torch.randn(*shape, generator=gen, dtype=torch.float64)
        u, s, vt = torch.linalg.svd(g, full_matrices=False)
        s = s / (g.norm() + 1e-7)
        a, b, c = M.COEFFS
        for _ in range(5):
            s = a * s + b * s ** 3 + c * s ** 5
        assert torch.allclose(M.polar(g), (u * s) @ vt, atol=1e-11)
