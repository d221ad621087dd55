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
