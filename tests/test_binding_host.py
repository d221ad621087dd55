"""The binding without its extension module (no GPU): what needs the library alone still loads."""

import os
import shutil
import subprocess
import sys

import pytest

PROGRAM = """
import torch
import sharded_flatparameter_flatten_amd as fsdp
u = fsdp.Unit([(5, 7), (3,)], 4, 1)
assert (u.S, u.shard_begin) == (10, 10) and fsdp.abi_version() > 0
assert fsdp.orthogonalize_workspace([torch.empty(64, 64, device="meta")]) > 0
x, hp = torch.zeros(10), fsdp.AdamWHparams()
try:
    fsdp.reduce_adamw_shard(u, [x], x, x, x, None, hp, 1)     # refused for what it is given
except ValueError as e:
    assert "device tensor" in str(e)
else:
    raise AssertionError("a host tensor was taken")
for name, call in (
        ("rms_norm", lambda: fsdp.rms_norm(x, x, x)),
        ("rms_norm_backward", lambda: fsdp.rms_norm_backward(x, x, x, x, x, None, None)),
        ("reduce_momentum_shard", lambda: fsdp.reduce_momentum_shard(u, [x], x, x, fsdp.MuonHparams())),
        ("muon_apply_shard", lambda: fsdp.muon_apply_shard(u, [x, x], [1, 1], x, None, fsdp.MuonHparams()))):
    try:
        call()
    except ImportError as e:
        assert name in str(e) and "_calls.so" in str(e) and "build" in str(e), e
    else:
        raise AssertionError(name)
print("fine")
"""


@pytest.mark.parametrize("left", ["none", "not loadable"])
def test_library_alone(lib, tmp_path, left):
    package = tmp_path / "sharded_flatparameter_flatten_amd"
    package.mkdir()
    here = os.path.dirname(lib.library_path())
    for name in ("__init__.py", os.path.basename(lib.library_path())):
        shutil.copy(os.path.join(here, name), package / name)
    if left == "not loadable":
        (package / "_calls.so").write_bytes(b"no library")
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=tmp_path, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stdout + r.stderr


def test_extension_module_is_built(lib):
    """Beside the built library the calls are the extension module's."""
    assert lib._calls.__file__.endswith("_calls.so")
