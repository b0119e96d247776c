"""The Muon update at the ends of its ranges: magnitudes, numbers of steps, matrices that lack directions.

The reference is the definition in float64. No tolerance here comes from an emulation
of the kernels: each bound is written out where it is used.
"""
import pytest

import helpers as H
from host_offloaded_layer_b200 import _lib as L

pytestmark = pytest.mark.gpu

NA, NB, NC = 3.4445, -4.7750, 2.0315
UB = 2.0 ** -8  # half a bf16 step, relative


def _exact(u, steps, eps):
    x = u / (u.norm() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(steps):
        a = x @ x.T
        x = NA * x + (NB * a + NC * (a @ a)) @ x
    return x.T if tall else x


def _update(g, cfg, m=None, m_out=None):
    import torch
    rows, cols = g.shape
    o = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    n = L.mt_muon_workspace_bytes(rows, cols)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN in every format
    L.mt_muon_update(g, cols, m, m_out, cols, o, cols, rows, cols, cfg, ws, n)
    torch.cuda.synchronize()
    assert L.mt_device_error(clear=True) == 0
    return o.double()


@pytest.mark.parametrize("rows,cols", [(30, 500), (500, 30), (64, 64), (1, 900)])
def test_short_sides_of_zeros_and_tiny_norms_with_an_eps_as_tiny(rows, cols):
    """u / (|u| + eps) is in [0, 1] whatever the two are: subnormal gradients with a subnormal eps, and zeros, which
    stay zeros. The Gram matrix and what follows from it are in fp32 or more: against bf16's rounding, 2^-12 of the
    result covers five steps on it (each step's polynomial has a few roundings of 2^-24, and weak directions take no
    more than 3.4445^5 = 485 of them)."""
    import torch
    gen = torch.Generator().manual_seed(cols)
    for eps in (1e-38, 1e-44):
        cfg = L.make_muon_cfg(eps=eps)
        assert bool((_update(torch.zeros(rows, cols, device="cuda"), cfg) == 0).all())
        for size in (1e-37, 1e-39, 1e-41):
            g = (torch.randn(rows, cols, generator=gen, dtype=torch.float64) * size).float().cuda()
            ref = _exact(g.double(), cfg.steps, cfg.eps)
            assert (_update(g, cfg) - ref).norm() <= (1.01 * UB + 2.0 ** -12) * ref.norm(), (eps, size)


@pytest.mark.parametrize("rows,cols", [(250, 500), (500, 250), (1200, 1300)])
def test_subnormal_gradients_lose_no_bits(rows, cols):
    """u / |u| of a gradient made of 2^-149 times small whole numbers is that of the whole numbers: scaling by a power of
    two changes no rounding where neither side is subnormal on the way, so the two results are equal bit for bit."""
    import torch
    gen = torch.Generator().manual_seed(rows)
    whole = torch.randint(-7, 8, (rows, cols), generator=gen).double()
    cfg = L.make_muon_cfg(eps=1e-45)  # 2^-149, against norms of a thousand times that
    tiny = (whole * 2.0 ** -149).float().cuda()
    assert bool((tiny.double() == (whole * 2.0 ** -149).cuda()).all())
    cfg1 = L.make_muon_cfg(eps=1.0)
    assert torch.equal(_update(tiny, cfg), _update(whole.float().cuda(), cfg1))
