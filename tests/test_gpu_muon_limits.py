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


def _matrix(kind, rows, cols, seed):
    """Gradients that lack directions. Those of whole numbers lack them exactly, in fp32 as in float64."""
    gen = torch_generator(seed)
    import torch
    whole = lambda *s: torch.randint(-8, 9, s, generator=gen).double()  # noqa: E731
    if kind == "rank 1":
        g = whole(rows, 1) @ whole(1, cols)
    elif kind == "rank 8":
        g = whole(rows, 8) @ whole(8, cols)
    elif kind == "equal":
        g = torch.ones(rows, cols, dtype=torch.float64)
    elif kind == "rows four times":
        g = torch.randn((rows + 3) // 4, cols, generator=gen).double().repeat_interleave(4, 0)[:rows]
    elif kind == "strong + 1e-3":
        g = (torch.randn(rows, 1, generator=gen) @ torch.randn(1, cols, generator=gen)
             + 1e-3 * torch.randn(rows, cols, generator=gen)).double()
    else:
        g = torch.randn(rows, cols, generator=gen).double()
    return (g * 2.0 ** -10).float()


def torch_generator(seed):
    import torch
    return torch.Generator().manual_seed(seed)


def _after(s, steps):
    """What `steps` steps make of singular values s, and |s f'/f|, how they pass on a relative change."""
    d = s * 0 + 1
    x = s.clone()
    for _ in range(steps):
        d = d * (NA + 3 * NB * x ** 2 + 5 * NC * x ** 4)
        x = NA * x + NB * x ** 3 + NC * x ** 5
    return x, (s * d / x).abs()


KINDS = ["rank 1", "rank 8", "equal", "rows four times", "strong + 1e-3", "full"]


@pytest.mark.parametrize("steps", [1, 5, 6, 7, 10, 12, 20])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(48, 2000), (2000, 48), (64, 64), (32, 500), (13, 70)])
def test_short_sides_follow_the_exact_steps(rows, cols, kind, steps):
    """Up to five steps the header's 2e-3 (2-norm); more run in fp64: each singular value's X X^T is off by at most
    2^-53 times 512 and the longest chain of additions (what is added to the diagonal), relative to s^2 half of that,
    and a step's products by 2^-53 times 64 terms a few times, below 2^-40 for all steps; the scalar map passes both on.
    The reference has noise of its own in directions that u lacks: 2^-46 of |u| grown by 3.4445 a step."""
    import torch
    g = _matrix(kind, rows, cols, rows + steps).cuda()
    cfg = L.make_muon_cfg(steps=steps)
    ref = _exact(g.double(), steps, cfg.eps)
    off = (_update(g, cfg) - ref).norm()
    allowed = 1.01 * UB * ref.norm()
    if steps <= 5:
        allowed += 2e-3 * ref.norm()
    else:
        u = g.double().cpu()
        s = torch.linalg.svdvals(u / (u.norm() + cfg.eps))
        s = s[s > 1e-9]
        x, pass_on = _after(s, steps)
        n = max(rows, cols)
        floor = (-(-n // 64 // 148) * 64 + 64 + 28 + 512) * 2.0 ** -53
        allowed += (x * pass_on * (floor / (2 * s * s) + 2.0 ** -40)).norm() + 2.0 ** -46 * NA ** steps
    assert off <= allowed, (float(off / ref.norm()), float(allowed / ref.norm()))


@pytest.mark.parametrize("steps", [5, 6, 12, 20])
@pytest.mark.parametrize("ratio", [1e-3, 1e-6, 1e-9])
@pytest.mark.parametrize("rows,cols", [(48, 2000), (500, 30)])
def test_short_sides_under_an_eps_that_dwarfs_the_norm(rows, cols, ratio, steps):
    """X starts at |u| / eps, as small as it may be, and the steps raise it. Gaussian rows have singular values within a
    factor of two of one another: what is passed on of a relative 2^-40 is as in the test above, and five steps in fp32
    stay within the header's 1e-3."""
    import torch
    g = torch.randn(rows, cols, generator=torch_generator(steps))
    g = (g * (ratio / float(g.norm()))).cuda()
    cfg = L.make_muon_cfg(steps=steps, eps=1.0)
    ref = _exact(g.double(), steps, cfg.eps)
    s = torch.linalg.svdvals(g.double().cpu() / (g.double().cpu().norm() + cfg.eps))
    x, pass_on = _after(s, steps)
    floor = 1400 * 2.0 ** -53 * (ratio * ratio)  # 512, and a chain of less than 800, of the trace
    allowed = 1.01 * UB * ref.norm() + (1e-3 * ref.norm() if steps <= 5 else (x * pass_on * (floor / (2 * s * s) + 2.0 ** -40)).norm())
    assert (_update(g, cfg) - ref).norm() <= allowed


@pytest.mark.parametrize("steps", [30, 100])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(48, 2000), (300, 64)])
def test_short_sides_stay_bounded_for_any_number_of_steps(rows, cols, kind, steps):
    """The polynomial maps [0, 1] into [0, 1.2024]: so do the steps on any matrix near u, and bf16 adds 2^-8 at most."""
    import torch
    o = _update(_matrix(kind, rows, cols, steps).cuda(), L.make_muon_cfg(steps=steps))
    assert bool(torch.isfinite(o).all()) and float(torch.linalg.matrix_norm(o, 2)) <= 1.2024 * (1 + UB)
    assert float(torch.linalg.matrix_norm(o, 2)) > 0.5  # nor does the strongest direction vanish


# ---------------------------------------------------------------- tensor cores: short sides above 64
def _fp16_bound(s, steps, pair):
    """What half a step (2^-11) in every fp16 operand does to the results of singular values s, relative to them, to first
    order and with all the roundings of a matrix falling the same way: the sum over the operands' derivatives. That is
    what a matrix of equal entries can come to; roundings that fall either way stay far below. (X's rest in the first
    steps leaves 2^-22, which is nothing beside; a factor of 1.1 covers the second order.)"""
    import torch
    n_roundings = 6 * steps + 2
    e = torch.zeros(n_roundings, len(s), dtype=torch.float64, requires_grad=True)
    it = iter(range(n_roundings))
    r = lambda v: v * (1 + e[next(it)])  # noqa: E731  one operand, rounded
    x, done = s.clone(), 0
    if pair and steps >= 4:
        h = r(x)
        a = r(h * h)
        p = r(NB * a + NC * a * a)
        m = r(p * a)
        a1 = r(NA ** 2 * a + 2 * NA * m + p * m)
        p1 = r(NB * a1 + NC * a1 * a1)
        x, done = NA ** 2 * x + r(NA * (p + p1) + p1 * p) * h, 2
    for i in range(done, steps):
        h = r(x)
        a = r(h * h)
        if i < steps - 2:
            x = NA * x + r(NB * a + NC * a * a) * h
        else:  # a I in the same operand: its diagonal rounds too
            x = (r(NB * a + NC * a * a) + r(torch.full_like(a, NA))) * h
    g, = torch.autograd.grad(x.sum(), e)
    return 1.1 * 2.0 ** -11 * g.abs().sum(0) / x.detach().abs()


@pytest.mark.parametrize("steps", [1, 2, 5, 7])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(65, 200), (300, 128), (333, 500), (1200, 1300), (1200, 2600), (2600, 1200), (100, 19000)])
def test_other_matrices_follow_the_exact_steps(rows, cols, kind, steps):
    """Against float64 steps, whatever the matrix lacks: the roundings' bound of its singular values (those above 1e-6: in
    the others nothing but the noise of X's two terms, 2^-22 of |u| in the 2-norm each step, grown by 3.4445 a step),
    and bf16's."""
    import torch
    g = _matrix(kind, rows, cols, rows + steps).cuda()
    cfg = L.make_muon_cfg(steps=steps)
    ref = _exact(g.double(), steps, cfg.eps)
    off = (_update(g, cfg) - ref).norm()
    u = g.double()
    s = torch.linalg.svdvals(u / (u.norm() + cfg.eps)).cpu()
    s = s[s > 1e-6]
    short, long = min(rows, cols), max(rows, cols)
    shared = long >= 2 * short and -(-short // 128) * -(-long // 128) > 148  # the first two steps on one Gram matrix
    rel = float(_fp16_bound(s, steps, shared).max())
    noise = sum(2.0 ** -22 * NA ** k for k in range(1, steps + 1))
    allowed = (1.01 * UB + rel) * ref.norm() + noise
    assert off <= allowed
    if steps == 5:  # and what the header states, with bf16's own share of 2^-8 / sqrt(3) at most
        stated = 3e-3 if kind in ("full", "rows four times", "strong + 1e-3", "rank 8") else 2e-2 if shared else 5e-3
        assert off <= (stated + 2.3e-3) * ref.norm()


@pytest.mark.parametrize("steps", [20, 100])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(65, 200), (300, 128), (1200, 2600)])
def test_other_matrices_stay_bounded_for_any_number_of_steps(rows, cols, kind, steps):
    """The polynomial maps [0, 1.2024] into itself, and up to 1.264 back below: 2e-2 of roundings do not lead out."""
    import torch
    o = _update(_matrix(kind, rows, cols, steps).cuda(), L.make_muon_cfg(steps=steps))
    assert bool(torch.isfinite(o).all())
    top = float(torch.linalg.matrix_norm(o.float(), 2))
    assert 0.5 < top <= 1.23


@pytest.mark.parametrize("where", ["g", "m"])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("rows,cols,steps", [(30, 500, 5), (500, 30, 5), (30, 500, 8), (1, 64, 5), (250, 500, 5), (500, 250, 1),
                                             (1200, 1300, 5), (2600, 1200, 5)])
def test_one_infinity_or_nan_makes_the_whole_result_nan(rows, cols, steps, bad, where):
    import torch
    gen = torch_generator(rows)
    g, m = (torch.randn(rows, cols, generator=gen).cuda() for _ in range(2))
    (g if where == "g" else m)[rows // 2, cols // 3] = bad
    m_out = torch.empty_like(m)
    o = _update(g, L.make_muon_cfg(steps=steps), m, m_out)
    assert bool(o.isnan().all())
    assert int((~torch.isfinite(m_out)).sum()) == 1  # the momentum is element by element
