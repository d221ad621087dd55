"""Python binding of libfsdpshard.so (argument marshalling only), through ctypes, and for the
calls with the shortest kernels through the extension module ``_calls`` (csrc/calls.cpp), which
nothing else needs.

Every step of the path runs in the HIP library; this module only turns torch
tensors into device pointers, picks the current HIP stream, and turns status
codes into exceptions. torch is imported first so that the library binds to
the HIP runtime torch has already loaded.

Names follow the C ABI in include/fsdp_shard.h:

* ``Unit(shapes, F, rank)``                 -> fsdp_unit_create / query / tensor
* ``flatten_pad(unit, tensors, dst, ...)``  -> fsdp_flatten_pad
* ``reduce_shard(unit, grads, out, ...)``   -> fsdp_reduce_shard
* ``adamw_shard(unit, grad, master, exp_avg, exp_avg_sq, param_out, hp)``
                                            -> fsdp_adamw_shard
* ``reduce_adamw_shard(unit, grads, master, exp_avg, exp_avg_sq, param_out, hp)``
                                            -> fsdp_reduce_adamw_shard
* ``reduce_adamw_units(steps, hp, step)``   -> fsdp_reduce_adamw_units
* ``reduce_shard_hybrid`` / ``reduce_adamw_shard_hybrid`` -> the hybrid-sharding forms
* ``reduce_shard_bf16acc`` / ``reduce_adamw_shard_bf16acc`` -> bf16 partial sums
* ``cast_unflatten(unit, shards, outs)``    -> fsdp_cast_unflatten (bf16 outputs)
* ``unflatten(unit, shards, outs)``         -> fsdp_unflatten (dtypes from the tensors)
* ``reduce_momentum_shard(unit, grads, momentum, update, hp)``
                                            -> fsdp_reduce_momentum_shard
* ``orthogonalize(mats, outs, workspace)`` / ``orthogonalize_workspace(mats)``
                                            -> fsdp_orthogonalize
* ``muon_apply_shard(unit, tensors, scales, master, param_out, hp)``
                                            -> fsdp_muon_apply_shard
* ``rms_norm(x, weight, out, ...)``         -> fsdp_rms_norm
* ``rms_norm_backward(dy, x, weight, rstd, dx, dweight, workspace, ...)``
                                            -> fsdp_rms_norm_backward
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

__all__ = [
    "FsdpError", "Unit", "AdamWHparams", "flatten_pad", "reduce_shard", "adamw_shard",
    "reduce_adamw_shard", "reduce_adamw_units", "UnitsStep", "cast_unflatten", "unflatten",
    "reduce_shard_hybrid", "reduce_adamw_shard_hybrid", "reduce_shard_bf16acc",
    "reduce_adamw_shard_bf16acc", "MuonHparams", "reduce_momentum_shard", "muon_apply_shard",
    "orthogonalize", "orthogonalize_workspace", "rms_norm", "rms_norm_backward",
    "rms_norm_backward_workspace", "abi_version", "library_path",
    "F32", "BF16",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libfsdpshard.so"
F32, BF16 = 0, 1
MAX_RANKS = 64

_c_void_p_p = ctypes.POINTER(ctypes.c_void_p)


class FsdpError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[{status}] {message}")
        self.status = status


class _UnitInfo(ctypes.Structure):
    _fields_ = [("U", ctypes.c_int64), ("S", ctypes.c_int64), ("padded", ctypes.c_int64),
                ("pad", ctypes.c_int64), ("shard_begin", ctypes.c_int64),
                ("shard_valid", ctypes.c_int64), ("persistent_bytes", ctypes.c_int64),
                ("F", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("n_tensors", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("fingerprint", ctypes.c_uint64)]


class _UnitStep(ctypes.Structure):
    _fields_ = [("unit", ctypes.c_void_p), ("grads", ctypes.POINTER(ctypes.c_void_p)),
                ("master", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("param_bf16_out", ctypes.c_void_p)]


class _Hparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double),
                ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("step", ctypes.c_int64)]


class _MuonHparams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("momentum", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("nesterov", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class _NormArgs(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("weight", ctypes.c_void_p), ("residual_out", ctypes.c_void_p),
                ("out", ctypes.c_void_p), ("rstd", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("x_pitch", ctypes.c_int64), ("residual_pitch", ctypes.c_int64),
                ("residual_out_pitch", ctypes.c_int64), ("out_pitch", ctypes.c_int64),
                ("eps", ctypes.c_double), ("dtype", ctypes.c_int), ("reserved", ctypes.c_int32)]


class _NormBackwardArgs(ctypes.Structure):
    _fields_ = [("dy", ctypes.c_void_p), ("x", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("rstd", ctypes.c_void_p), ("dresidual", ctypes.c_void_p),
                ("dx", ctypes.c_void_p), ("dweight", ctypes.c_void_p),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("dy_pitch", ctypes.c_int64), ("x_pitch", ctypes.c_int64),
                ("dresidual_pitch", ctypes.c_int64), ("dx_pitch", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("reserved", ctypes.c_int32)]


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def _load():
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
            "(or python sharded_flatparameter_flatten_amd/build.py) first")
    lib = ctypes.CDLL(path)
    st = ctypes.c_int
    vp = ctypes.c_void_p
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    sig = {
        "fsdp_abi_version": (i32, []),
        "fsdp_status_string": (ctypes.c_char_p, [st]),
        "fsdp_last_error": (ctypes.c_char_p, []),
        "fsdp_unit_create": (st, [i32, i32, i32, ctypes.POINTER(i32), ctypes.POINTER(i64),
                                  ctypes.POINTER(vp)]),
        "fsdp_unit_destroy": (st, [vp]),
        "fsdp_unit_query": (st, [vp, ctypes.POINTER(_UnitInfo)]),
        "fsdp_unit_tensor": (st, [vp, i32, ctypes.POINTER(i64), ctypes.POINTER(i64)]),
        "fsdp_flatten_pad": (st, [vp, st, _c_void_p_p, i64, i64, vp, vp]),
        "fsdp_reduce_shard": (st, [vp, i32, _c_void_p_p, ctypes.c_double, vp, vp]),
        "fsdp_adamw_shard": (st, [vp, vp, vp, vp, vp, vp, ctypes.POINTER(_Hparams), vp]),
        "fsdp_reduce_adamw_shard": (st, [vp, i32, _c_void_p_p, vp, vp, vp, vp,
                                         ctypes.POINTER(_Hparams), vp]),
        "fsdp_cast_unflatten": (st, [vp, st, _c_void_p_p, _c_void_p_p, vp]),
        "fsdp_reduce_adamw_units": (st, [i32, ctypes.POINTER(_UnitStep), i32,
                                         ctypes.POINTER(_Hparams), vp]),
        "fsdp_unflatten": (st, [vp, st, st, _c_void_p_p, _c_void_p_p, vp]),
        "fsdp_reduce_shard_hybrid": (st, [vp, i32, _c_void_p_p, ctypes.c_double, vp, vp]),
        "fsdp_reduce_shard_bf16acc": (st, [vp, i32, _c_void_p_p, ctypes.c_double, vp, vp]),
        "fsdp_reduce_adamw_shard_bf16acc": (st, [vp, i32, _c_void_p_p, vp, vp, vp, vp,
                                                 ctypes.POINTER(_Hparams), vp]),
        "fsdp_reduce_adamw_shard_hybrid": (st, [vp, i32, _c_void_p_p, vp, vp, vp, vp,
                                                ctypes.POINTER(_Hparams), vp]),
        "fsdp_reduce_momentum_shard": (st, [vp, i32, _c_void_p_p, vp, vp,
                                            ctypes.POINTER(_MuonHparams), vp]),
        "fsdp_muon_apply_shard": (st, [vp, _c_void_p_p, ctypes.POINTER(ctypes.c_double), vp, vp,
                                       ctypes.POINTER(_MuonHparams), vp]),
        "fsdp_orthogonalize_workspace": (st, [i32, ctypes.POINTER(i64), ctypes.POINTER(i64),
                                              ctypes.POINTER(i64)]),
        "fsdp_orthogonalize": (st, [i32, st, _c_void_p_p, ctypes.POINTER(i64),
                                    ctypes.POINTER(i64), ctypes.POINTER(i64), _c_void_p_p,
                                    ctypes.POINTER(i64), vp, i64, i32,
                                    ctypes.POINTER(ctypes.c_double), ctypes.c_double, vp]),
        "fsdp_rms_norm": (st, [ctypes.POINTER(_NormArgs), vp]),
        "fsdp_rms_norm_backward_workspace": (st, [i64, i64, ctypes.POINTER(i64)]),
        "fsdp_rms_norm_backward": (st, [ctypes.POINTER(_NormBackwardArgs), vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


class _NoCalls:
    """Stands for the extension module where it cannot be loaded (not built, or built for another
    torch): the calls it marshals raise, the others, which need the library alone, work."""

    def __init__(self, why: ImportError):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(
            f"{name} needs the extension module _calls.so, which does not load ({self._why}); run "
            "`python -c 'import __graft_entry__ as g; g.build()'` "
            "(or python sharded_flatparameter_flatten_amd/build.py)") from self._why


_lib = _load()
try:
    from . import _calls  # noqa: E402  (links against the library that _load opened)
except ImportError as e:
    _calls = _NoCalls(e)


def abi_version() -> int:
    return int(_lib.fsdp_abi_version())


def _check(status: int | None):
    if status is None:
        raise TypeError("an argument cannot be used")
    if status != 0:
        msg = _lib.fsdp_last_error().decode() or _lib.fsdp_status_string(status).decode()
        raise FsdpError(status, msg)


def _ptr_array(ptrs):
    return (ctypes.c_void_p * max(1, len(ptrs)))(*ptrs)


# The current stream's handle without a torch.cuda.Stream object around it (0.1 us
# instead of 2 us a call, which shows in the calls whose kernels take 3 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if not isinstance(_calls, _NoCalls):
    _calls.set_current_stream(_raw_stream or (lambda index: torch.cuda.current_stream(index).cuda_stream))


def _stream(stream, device=None):
    if stream is None:
        if _raw_stream is not None and device is not None and device.index is not None:
            return _raw_stream(device.index)
        return torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev(t: torch.Tensor, dtype: torch.dtype, name: str, min_numel: int = 0,
         index: int | None = None) -> int:
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and t.numel() >= min_numel):
        return t.data_ptr()
    if index is not None:
        name = f"{name}[{index}]"
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} has {t.numel()} elements, needs {min_numel}")


@dataclass
class AdamWHparams:
    lr: float = 1e-4
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    weight_decay: float = 0.01

    def _c(self, step: int, grad_scale: float = 0.0) -> _Hparams:
        return _Hparams(self.lr, self.beta1, self.beta2, self.eps, self.weight_decay,
                        grad_scale, int(step))


class Unit:
    """One FSDP unit (a list of tensor shapes) as seen by rank ``rank`` of ``F``."""

    def __init__(self, shapes, F: int, rank: int):
        shapes = [tuple(int(d) for d in s) for s in shapes]
        ndim = (ctypes.c_int32 * len(shapes))(*[len(s) for s in shapes])
        flat = [d for s in shapes for d in s]
        dims = (ctypes.c_int64 * max(1, len(flat)))(*flat)
        h = ctypes.c_void_p()
        _check(_lib.fsdp_unit_create(F, rank, len(shapes), ndim, dims, ctypes.byref(h)))
        self._h = h
        self._address = h.value
        self.shapes = shapes
        info = _UnitInfo()
        _check(_lib.fsdp_unit_query(self._h, ctypes.byref(info)))
        for name, _ in _UnitInfo._fields_:
            if name != "reserved":
                setattr(self, name, int(getattr(info, name)))
        self.offsets, self.numels = [], []
        for i in range(len(shapes)):
            off, n = ctypes.c_int64(), ctypes.c_int64()
            _check(_lib.fsdp_unit_tensor(self._h, i, ctypes.byref(off), ctypes.byref(n)))
            self.offsets.append(off.value)
            self.numels.append(n.value)

    @property
    def handle(self):
        return self._h

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value and _lib is not None:
            _lib.fsdp_unit_destroy(h)
            self._h = None


def flatten_pad(unit: Unit, tensors, dst: torch.Tensor, begin: int | None = None,
                length: int | None = None, stream=None):
    """dst[q] = padded_flat[begin + q]; defaults to this rank's shard window."""
    begin = unit.shard_begin if begin is None else int(begin)
    length = unit.S if length is None else int(length)
    dtype = dst.dtype
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("dst must be float32 or bfloat16")
    code = F32 if dtype == torch.float32 else BF16
    ptrs = [_dev(t, dtype, "tensors", n, i) for i, (t, n) in
            enumerate(zip(tensors, unit.numels))]
    if len(ptrs) != unit.n_tensors:
        raise ValueError(f"need {unit.n_tensors} tensors, got {len(ptrs)}")
    d = _dev(dst, dtype, "dst", length)
    _check(_lib.fsdp_flatten_pad(unit.handle, code, _ptr_array(ptrs), begin, length, d,
                                 _stream(stream, dst.device)))


def _grad_ptrs(unit: Unit, grads):
    if not 1 <= len(grads) <= MAX_RANKS:
        raise ValueError(f"need 1..{MAX_RANKS} gradient buffers, got {len(grads)}")
    return [_dev(g, torch.bfloat16, "grads", unit.U, k) for k, g in enumerate(grads)]


def reduce_shard(unit: Unit, grads, out: torch.Tensor, grad_scale: float | None = None,
                 stream=None):
    ptrs = _grad_ptrs(unit, grads)
    gs = 1.0 / len(grads) if grad_scale is None else float(grad_scale)
    o = _dev(out, torch.float32, "out", unit.shard_valid)
    _check(_lib.fsdp_reduce_shard(unit.handle, len(ptrs), _ptr_array(ptrs), gs, o,
                                  _stream(stream, out.device)))


def _state_ptrs(unit: Unit, master, exp_avg, exp_avg_sq, param_out):
    n = unit.shard_valid
    p = _dev(master, torch.float32, "master", n)
    m = _dev(exp_avg, torch.float32, "exp_avg", n)
    v = _dev(exp_avg_sq, torch.float32, "exp_avg_sq", n)
    w = None if param_out is None else _dev(param_out, torch.bfloat16, "param_out", n)
    return p, m, v, w


def adamw_shard(unit: Unit, grad, master, exp_avg, exp_avg_sq, param_out,
                hp: AdamWHparams, step: int, stream=None):
    g = _dev(grad, torch.float32, "grad", unit.shard_valid)
    p, m, v, w = _state_ptrs(unit, master, exp_avg, exp_avg_sq, param_out)
    c = hp._c(step)
    _check(_lib.fsdp_adamw_shard(unit.handle, g, p, m, v, w, ctypes.byref(c),
                                 _stream(stream, master.device)))


def reduce_adamw_shard(unit: Unit, grads, master, exp_avg, exp_avg_sq, param_out,
                       hp: AdamWHparams, step: int, grad_scale: float | None = None,
                       stream=None):
    ptrs = _grad_ptrs(unit, grads)
    gs = 1.0 / len(grads) if grad_scale is None else float(grad_scale)
    p, m, v, w = _state_ptrs(unit, master, exp_avg, exp_avg_sq, param_out)
    c = hp._c(step, gs)
    _check(_lib.fsdp_reduce_adamw_shard(unit.handle, len(ptrs), _ptr_array(ptrs), p, m, v, w,
                                        ctypes.byref(c), _stream(stream, master.device)))


def reduce_shard_bf16acc(unit: Unit, grads, out: torch.Tensor, grad_scale: float | None = None,
                         stream=None):
    """reduce_shard with bf16 partial sums (reduce dtype bf16)."""
    ptrs = _grad_ptrs(unit, grads)
    gs = 1.0 / len(grads) if grad_scale is None else float(grad_scale)
    o = _dev(out, torch.float32, "out", unit.shard_valid)
    _check(_lib.fsdp_reduce_shard_bf16acc(unit.handle, len(ptrs), _ptr_array(ptrs), gs, o,
                                          _stream(stream, out.device)))


def reduce_adamw_shard_bf16acc(unit: Unit, grads, master, exp_avg, exp_avg_sq, param_out,
                               hp: AdamWHparams, step: int, grad_scale: float | None = None,
                               stream=None):
    """reduce_adamw_shard with bf16 partial sums (reduce dtype bf16)."""
    ptrs = _grad_ptrs(unit, grads)
    gs = 1.0 / len(grads) if grad_scale is None else float(grad_scale)
    p, m, v, w = _state_ptrs(unit, master, exp_avg, exp_avg_sq, param_out)
    c = hp._c(step, gs)
    _check(_lib.fsdp_reduce_adamw_shard_bf16acc(unit.handle, len(ptrs), _ptr_array(ptrs),
                                                p, m, v, w, ctypes.byref(c),
                                                _stream(stream, master.device)))


def reduce_shard_hybrid(unit: Unit, replicas: int, grads, out: torch.Tensor,
                        grad_scale: float | None = None, stream=None):
    """Hybrid sharding: grads = replicas*F rows, replica-major."""
    ptrs = _grad_ptrs(unit, grads)
    gs = 1.0 / len(grads) if grad_scale is None else float(grad_scale)
    o = _dev(out, torch.float32, "out", unit.shard_valid)
    _check(_lib.fsdp_reduce_shard_hybrid(unit.handle, int(replicas), _ptr_array(ptrs), gs, o,
                                         _stream(stream, out.device)))


def reduce_adamw_shard_hybrid(unit: Unit, replicas: int, grads, master, exp_avg, exp_avg_sq,
                              param_out, hp: AdamWHparams, step: int,
                              grad_scale: float | None = None, stream=None):
    ptrs = _grad_ptrs(unit, grads)
    gs = 1.0 / len(grads) if grad_scale is None else float(grad_scale)
    p, m, v, w = _state_ptrs(unit, master, exp_avg, exp_avg_sq, param_out)
    c = hp._c(step, gs)
    _check(_lib.fsdp_reduce_adamw_shard_hybrid(unit.handle, int(replicas), _ptr_array(ptrs),
                                               p, m, v, w, ctypes.byref(c),
                                               _stream(stream, master.device)))


class UnitsStep:
    """A multi-unit optimizer step with its arguments marshalled once.

    ``steps``: sequence of (unit, grads, master, exp_avg, exp_avg_sq, param_out or None);
    every entry uses the same number of gradient rows. The tensors must stay
    alive (and at the same addresses) while the object is used; each call only
    fills in the hyper-parameters and the stream."""

    def __init__(self, steps):
        steps = list(steps)
        if not steps:
            raise ValueError("need at least one unit")
        self.n_grads = len(steps[0][1])
        self._keep = [steps]
        self._arr = (_UnitStep * len(steps))()
        for j, (unit, grads, master, exp_avg, exp_avg_sq, param_out) in enumerate(steps):
            if len(grads) != self.n_grads:
                raise ValueError("every unit needs the same number of gradient rows")
            rows = _ptr_array(_grad_ptrs(unit, grads))
            self._keep.append(rows)
            p, m, v, w = _state_ptrs(unit, master, exp_avg, exp_avg_sq, param_out)
            self._arr[j] = _UnitStep(unit.handle.value,
                                     ctypes.cast(rows, ctypes.POINTER(ctypes.c_void_p)), p, m, v, w)
        self.n_units = len(steps)
        self.device = steps[0][2].device

    def __call__(self, hp: AdamWHparams, step: int, grad_scale: float | None = None,
                 stream=None):
        gs = 1.0 / self.n_grads if grad_scale is None else float(grad_scale)
        c = hp._c(step, gs)
        _check(_lib.fsdp_reduce_adamw_units(self.n_units, self._arr, self.n_grads,
                                            ctypes.byref(c), _stream(stream, self.device)))


def reduce_adamw_units(steps, hp: AdamWHparams, step: int, grad_scale: float | None = None,
                       stream=None):
    """One optimizer step over many units (see UnitsStep for the argument layout)."""
    steps = list(steps)
    if steps:
        UnitsStep(steps)(hp, step, grad_scale, stream)


def unflatten(unit: Unit, shards, outs, stream=None):
    """Per-tensor outputs from the F shards; element types from the tensors (fp32/bf16)."""
    if len(shards) != unit.F:
        raise ValueError(f"need {unit.F} shards, got {len(shards)}")
    if len(outs) != unit.n_tensors:
        raise ValueError(f"need {unit.n_tensors} outputs, got {len(outs)}")
    sdtype, ddtype = shards[0].dtype, outs[0].dtype
    codes = {torch.float32: F32, torch.bfloat16: BF16}
    if sdtype not in codes or ddtype not in codes:
        raise TypeError("shards and outputs must be float32 or bfloat16")
    sp = []
    for k, s in enumerate(shards):
        valid = max(0, min(unit.S, unit.U - k * unit.S))
        sp.append(_dev(s, sdtype, "shards", valid, k))
    op = [_dev(o, ddtype, "outs", n, i) for i, (o, n) in enumerate(zip(outs, unit.numels))]
    _check(_lib.fsdp_unflatten(unit.handle, codes[sdtype], codes[ddtype], _ptr_array(sp),
                               _ptr_array(op), _stream(stream, outs[0].device)))


def cast_unflatten(unit: Unit, shards, outs, stream=None):
    """The all-gather arithmetic: F shards -> per-tensor bf16 parameters."""
    if outs and outs[0].dtype != torch.bfloat16:
        raise TypeError("cast_unflatten writes bf16 tensors; use unflatten for fp32 outputs")
    unflatten(unit, shards, outs, stream)


# --- the sharded Muon step ------------------------------------------------------------------


@dataclass
class MuonHparams:
    lr: float = 0.02
    momentum: float = 0.95
    nesterov: bool = True
    weight_decay: float = 0.0


def reduce_momentum_shard(unit: Unit, grads, momentum: torch.Tensor, update: torch.Tensor,
                          hp: MuonHparams, grad_scale: float | None = None, stream=None):
    """The gradient rows reduced into this rank's momentum; ``update``: its bf16 update."""
    if not grads:
        _grad_ptrs(unit, grads)
    status = _calls.reduce_momentum_shard(
        unit._address, unit.U, unit.shard_valid, grads, momentum, update, hp.lr, hp.momentum,
        hp.weight_decay, hp.nesterov, 1.0 / len(grads) if grad_scale is None else grad_scale,
        stream if stream is None else _stream(stream))
    if status == 0:
        return
    if status is None:
        _grad_ptrs(unit, grads)
        _dev(momentum, torch.float32, "momentum", unit.shard_valid)
        _dev(update, torch.bfloat16, "update", unit.shard_valid)
    _check(status)


def muon_apply_shard(unit: Unit, tensors, scales, master: torch.Tensor,
                     param_out: torch.Tensor | None, hp: MuonHparams, stream=None):
    """This rank's window of the whole update tensors, each times its scale, applied to its
    master weights (and the bf16 parameter). Tensors that do not reach into the window, and
    their scales, may be None: a rank orthogonalises only what it applies."""
    status = _calls.muon_apply_shard(
        unit._address, unit.numels, unit.shard_begin, unit.shard_valid, tensors, scales, master,
        param_out, hp.lr, hp.momentum, hp.weight_decay, hp.nesterov,
        stream if stream is None else _stream(stream))
    if status == 0:
        return
    if status is None:
        if len(tensors) != unit.n_tensors or len(scales) != unit.n_tensors:
            raise ValueError(f"need {unit.n_tensors} tensors and scales, got {len(tensors)} and "
                             f"{len(scales)}")
        end = unit.shard_begin + unit.shard_valid
        for i, (t, at, n) in enumerate(zip(tensors, unit.offsets, unit.numels)):
            if t is not None or max(at, unit.shard_begin) < min(at + n, end):
                _dev(t, torch.bfloat16, "tensors", n, i)
        _dev(master, torch.float32, "master", unit.shard_valid)
        if param_out is not None:
            _dev(param_out, torch.bfloat16, "param_out", unit.shard_valid)
    _check(status)


def _dev_rows(t: torch.Tensor, dtype: torch.dtype, name: str, shape=None):
    """A 2-d device tensor with contiguous rows: pointer and row pitch in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    size = t.shape
    if len(size) != 2 or (shape is not None and size != shape):
        want = "2-d" if shape is None else f"of shape {tuple(shape)}"
        raise ValueError(f"{name} must be {want}, got {tuple(size)}")
    rows, cols = size
    pitch, step = t.stride()
    if rows <= 1:
        pitch = cols
    if (cols > 1 and step != 1) or pitch < cols:
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return t.data_ptr(), pitch


def _i64_array(values):
    return (ctypes.c_int64 * max(1, len(values)))(*values)


def orthogonalize_workspace(mats) -> int:
    """Bytes of device workspace that ``orthogonalize`` needs for matrices of these shapes."""
    need = ctypes.c_int64()
    _check(_lib.fsdp_orthogonalize_workspace(
        len(mats), _i64_array([m.shape[0] for m in mats]),
        _i64_array([m.shape[1] for m in mats]), ctypes.byref(need)))
    return need.value


def orthogonalize(mats, outs, workspace: torch.Tensor, steps: int = 5,
                  coeffs=(3.4445, -4.7750, 2.0315), eps: float = 1e-7, stream=None):
    """Newton-Schulz orthogonalisation of 2-d matrices (all bf16 or all fp32) into bf16 ``outs``.

    ``workspace``: a device byte tensor of ``orthogonalize_workspace(mats)`` bytes."""
    if len(outs) != len(mats):
        raise ValueError(f"need {len(mats)} outputs, got {len(outs)}")
    if len(coeffs) != 3:
        raise ValueError("coeffs must be three numbers")
    if not mats:
        return
    dtype = mats[0].dtype
    if dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("matrices must be float32 or bfloat16")
    src = [_dev_rows(m, dtype, f"mats[{i}]") for i, m in enumerate(mats)]
    dst = [_dev_rows(o, torch.bfloat16, f"outs[{i}]", m.shape)
           for i, (o, m) in enumerate(zip(outs, mats))]
    ws = _dev(workspace, torch.uint8, "workspace")
    _check(_lib.fsdp_orthogonalize(
        len(mats), F32 if dtype == torch.float32 else BF16, _ptr_array([p for p, _ in src]),
        _i64_array([m.shape[0] for m in mats]), _i64_array([m.shape[1] for m in mats]),
        _i64_array([ld for _, ld in src]), _ptr_array([p for p, _ in dst]),
        _i64_array([ld for _, ld in dst]), ws, workspace.numel(), int(steps),
        (ctypes.c_double * 3)(*coeffs), float(eps), _stream(stream, mats[0].device)))


# --- RMS norm -------------------------------------------------------------------------------


def _check_norm_type(x: torch.Tensor):
    if not isinstance(x, torch.Tensor) or x.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("x must be a float32 or bfloat16 tensor")
    if x.dim() != 2:
        raise ValueError(f"x must be 2-d (rows, dim), got {tuple(x.shape)}")


def rms_norm(x: torch.Tensor, weight: torch.Tensor, out: torch.Tensor, eps: float = 1e-6,
             residual: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
             rstd: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """``out`` = the RMS norm of x's rows (of x + residual, which goes to ``residual_out``)
    times weight: in x's type, or in e4m3 (torch.float8_e4m3fn) with a scale a row in ``scales``.
    ``rstd`` (fp32, a value a row) is kept for the backward pass."""
    status = _calls.rms_norm(x, weight, out, residual, residual_out, rstd, scales, eps,
                             stream if stream is None else _stream(stream))
    if status == 0:
        return
    if status is None:
        _check_norm_type(x)
        dtype, size = x.dtype, x.shape
        if (residual is None) != (residual_out is None):
            raise ValueError("residual and residual_out go together")
        _dev_rows(x, dtype, "x")
        _dev_rows(out, dtype if scales is None else torch.float8_e4m3fn, "out", size)
        if residual is not None:
            _dev_rows(residual, dtype, "residual", size)
            _dev_rows(residual_out, dtype, "residual_out", size)
        _dev(weight, dtype, "weight", size[1])
        for t, name in ((rstd, "rstd"), (scales, "scales")):
            if t is not None:
                _dev(t, torch.float32, name, size[0])
    _check(status)


def rms_norm_backward_workspace(rows: int, dim: int) -> int:
    """Bytes of device workspace that ``rms_norm_backward`` needs."""
    need = ctypes.c_int64()
    _check(_lib.fsdp_rms_norm_backward_workspace(int(rows), int(dim), ctypes.byref(need)))
    return need.value


def rms_norm_backward(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                      rstd: torch.Tensor, dx: torch.Tensor, dweight: torch.Tensor | None,
                      workspace: torch.Tensor | None, dresidual: torch.Tensor | None = None,
                      stream=None):
    """Gradients of ``rms_norm``: dx (plus dresidual, the gradient that reaches the summed
    residual from elsewhere) and dweight (None: not computed, and no workspace needed)."""
    status = _calls.rms_norm_backward(dy, x, weight, rstd, dx, dweight, workspace, dresidual,
                                      stream if stream is None else _stream(stream))
    if status == 0:
        return
    if status is None:
        _check_norm_type(x)
        dtype, size = x.dtype, x.shape
        for t, name in ((dy, "dy"), (x, "x"), (dx, "dx"), (dresidual, "dresidual")):
            if t is not None or name != "dresidual":
                _dev_rows(t, dtype, name, size)
        _dev(weight, dtype, "weight", size[1])
        _dev(rstd, torch.float32, "rstd", size[0])
        if dweight is not None:
            _dev(dweight, dtype, "dweight", size[1])
            if workspace is not None:
                _dev(workspace, torch.uint8, "workspace")
    _check(status)
