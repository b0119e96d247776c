"""The Muon update on the B200 against its definition in float64.

Tolerances come from the arithmetic that the header states, not from the kernel's
results: `_emulate` runs the same steps in float64 with that arithmetic's roundings
(fp16 operands with an fp16 rest of X in all steps but the last two; fp32 on the
Gram matrix for short sides of at most 64). Its distance from the exact steps,
computed on the same inputs, is what the roundings cost; sums in another order move
single roundings, so twice that is allowed, in the 2-norm. Rounding the result to
bf16 adds at most half a step an element, 2^-8 of its value. m' is one fma.

The emulation leaves the sums themselves exact. With fp16 operands that is nothing
(2^-24 against 2^-11 of the same products); on the Gram path the last product's sum
is what an element is off by: s terms r_j u_j added one after another in fp32 (each
an fma) are at most s * 2^-24 * sum |r_j u_j| off, r's own rounding and u's are one
more 2^-24 of each term, so (s + 2) 2^-24 sum |r_j u_j| is added there, element by
element (strong directions cancel in these sums: the bound goes by the terms).
"""
import numpy as np
import pytest

import helpers as H
from host_offloaded_layer_b200 import _lib as L

pytestmark = pytest.mark.gpu

NA, NB, NC = 3.4445, -4.7750, 2.0315
U, UB = 2.0 ** -24, 2.0 ** -8


def _exact(u, steps, eps):
    x = u / (u.norm() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(steps):
        a = x @ x.T
        x = NA * x + (NB * a + NC * (a @ a)) @ x
    return x.T if tall else x


def _emulate(u, steps, eps):
    """The result with the roundings, and the bound of its elements' sums."""
    import torch
    x = u / (u.norm() + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    eye = torch.eye(len(x), dtype=x.dtype, device=x.device)
    sums = torch.zeros_like(x)
    if len(x) <= 64:
        f = lambda t: t.float().double()  # noqa: E731
        a, q = f(x @ x.T), eye
        for _ in range(steps):
            p = f(NA * eye + NB * a + NC * f(a @ a))
            q = f(p @ q)
            a = f(f(p @ a) @ p)
        sums = (len(x) + 2) * U * (q.abs() @ x.abs())
        x = f(q) @ x
    else:
        h = lambda t, s: (t * s).half().double() / s  # noqa: E731
        for i in range(steps):
            head = h(x, 16384.)
            a = h(head @ head.T, 16384.)
            if i < steps - 2:
                x = NA * (head + h(x - head, 16384.)) + h(NB * a + NC * (a @ a), 8192.) @ head
            else:
                x = h(NA * eye + NB * a + NC * (a @ a), 8192.) @ head
    return (x.T, sums.T) if tall else (x, sums)


def _gradient(gen, rows, cols, ld, kind="low rank"):
    """A few strong directions over noise (what a weight gradient looks like), or noise alone."""
    import torch
    t = torch.full((rows, ld), float("nan"))
    r = min(6, rows, cols)
    v = 0.3 * torch.randn(rows, cols, generator=gen)
    if kind == "low rank":
        v += torch.randn(rows, r, generator=gen) @ torch.randn(r, cols, generator=gen)
    t[:, :cols] = v * 1e-3
    return t.cuda()


def _run(g, ld_g, m_in, m_out, ld_m, o, ld_o, rows, cols, cfg, stream=None, ws=None):
    import torch
    n = L.mt_muon_workspace_bytes(rows, cols)
    if ws is None:
        ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")  # NaN in every format
    L.mt_muon_update(g, ld_g, m_in, m_out, ld_m, o, ld_o, rows, cols, cfg, ws, n, stream)
    return ws


def _check(o, u, cfg):
    import torch
    ref = _exact(u, cfg.steps, cfg.eps) * cfg.scale
    rounded, sums = _emulate(u, cfg.steps, cfg.eps)
    cost = rounded * cfg.scale - ref
    sums = sums * abs(cfg.scale)
    off = o.double() - ref
    # bf16 rounding (of a value that is `cost` off) and the roundings on the way
    assert off.norm() <= UB * ref.norm() * 1.01 + 2 * cost.norm() + sums.norm() + 1e-12
    # no element stands out: rounding noise is spread over the matrix, 16 times its rms covers its tail (and the
    # few elements of the smallest matrices)
    rms = cost.square().mean().sqrt()
    assert bool((off.abs() <= 1.01 * UB * ref.abs() + 16 * rms + 1.01 * sums + 1e-12).all())
    assert L.mt_device_error(clear=True) == 0
    torch.cuda.synchronize()


# short sides of the Gram path and around its end, odd sizes, one tile and many, K split over 1 to 8 CTAs,
# SM pairs (the last ones; whole waves of tiles, and a last wave in halves), the first two steps on one Gram matrix
# (long side at least twice the short one), each wide and tall
SIZES = [(1, 1), (1, 700), (3, 64), (17, 33), (64, 64), (64, 1111), (63, 5000), (65, 65), (65, 9000), (100, 130), (128, 128), (129, 4100),
         (200, 210), (256, 688), (300, 1500), (511, 777), (640, 640), (1024, 2560), (1100, 1300), (2300, 2500),
         (2900, 2950), (2850, 5800)]


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("short,long", SIZES)
def test_muon_update(short, long, tall):
    import torch
    rows, cols = (long, short) if tall else (short, long)
    gen = torch.Generator().manual_seed(short * 31 + long)
    pad = {0: 0, 1: 3, 2: 4}[(short + long) % 3]
    g, m = _gradient(gen, rows, cols, cols + pad), _gradient(gen, rows, cols, cols + pad)
    m_out = torch.full_like(m, 5.0)
    ld_o = cols + (0 if short % 2 else 8)
    o = torch.full((rows, ld_o), 7.0, dtype=torch.bfloat16, device="cuda")
    cfg = L.make_muon_cfg(momentum=0.9, scale=0.5 if short % 2 else 1.0)
    _run(g, cols + pad, m, m_out, cols + pad, o, ld_o, rows, cols, cfg)
    torch.cuda.synchronize()
    mu = float(np.float32(0.9))
    g64, m64 = g[:, :cols].double(), m[:, :cols].double()
    want_m = mu * m64 + g64
    assert bool(((m_out[:, :cols].double() - want_m).abs() <= U * want_m.abs() + 1e-45).all())
    assert bool((m_out[:, cols:] == 5.0).all()) and bool((o[:, cols:] == 7.0).all())
    _check(o[:, :cols], g64 + mu * m_out[:, :cols].double(), cfg)


@pytest.mark.parametrize("rows,cols", [(40, 300), (300, 200), (1024, 2600)])
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 7])
def test_muon_steps_without_momentum(rows, cols, steps):
    import torch
    gen = torch.Generator().manual_seed(steps)
    g = _gradient(gen, rows, cols, cols)
    o = H.empty_bf16(rows, cols)
    cfg = L.make_muon_cfg(steps=steps)
    _run(g, cols, None, None, 0, o, cols, rows, cols, cfg)
    _check(o, g.double(), cfg)


@pytest.mark.parametrize("rows,cols", [(33, 200), (200, 333)])
def test_muon_plain_momentum_in_place(rows, cols):
    import torch
    gen = torch.Generator().manual_seed(5)
    g, m = _gradient(gen, rows, cols, cols), _gradient(gen, rows, cols, cols)
    cfg = L.make_muon_cfg(momentum=0.95, nesterov=False)
    m2, o, o2 = torch.empty_like(m), H.empty_bf16(rows, cols), H.empty_bf16(rows, cols)
    _run(g, cols, m, m2, cols, o, cols, rows, cols, cfg)
    ws = _run(g, cols, m, m, cols, o2, cols, rows, cols, cfg)
    torch.cuda.synchronize()
    assert torch.equal(m, m2) and torch.equal(o, o2)
    _check(o, m.double(), cfg)
    del ws


@pytest.mark.parametrize("rows,cols", [(30, 500), (250, 500), (500, 250)])
@pytest.mark.parametrize("size", [1e-33, 1e-20, 1e25, 3e36])
def test_muon_takes_any_magnitude(rows, cols, size):
    """The norm's square leaves fp32 at either end; eps = 1e-38 counts at none of these sizes (1e-33 sqrt(n) >> 1e-38)."""
    import torch
    gen = torch.Generator().manual_seed(6)
    g = (_gradient(gen, rows, cols, cols).double() * (1e3 * size)).float()  # entries of about `size`
    assert bool(torch.isfinite(g).all())
    o = H.empty_bf16(rows, cols)
    cfg = L.make_muon_cfg(eps=1e-38)
    _run(g, cols, None, None, 0, o, cols, rows, cols, cfg)
    _check(o, g.double(), cfg)


@pytest.mark.parametrize("rows,cols", [(30, 500), (250, 500), (500, 250)])
def test_muon_of_zeros_and_of_nan(rows, cols):
    import torch
    g = torch.zeros(rows, cols, device="cuda")
    o = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    cfg = L.make_muon_cfg()
    _run(g, cols, None, None, 0, o, cols, rows, cols, cfg)
    torch.cuda.synchronize()
    assert bool((o == 0).all())
    g += 1.0
    g[2, 3] = float("nan")
    _run(g, cols, None, None, 0, o, cols, rows, cols, cfg)
    torch.cuda.synchronize()
    assert bool(o.isnan().any())
    assert L.mt_device_error(clear=True) == 0


def test_muon_of_an_orthogonal_matrix_and_of_one_row():
    """X = u / |u| of s orthonormal rows has all its singular values at 1/sqrt(s): the result is the polynomial's
    iterate times the rows, which is known in closed form (no matrix products in the reference)."""
    import torch
    for s, n in ((1, 300), (16, 400), (128, 512)):
        gen = torch.Generator().manual_seed(s)
        rows = torch.linalg.qr(torch.randn(n, s, generator=gen, dtype=torch.float64))[0].T.contiguous()
        g = rows.float().cuda()
        o = H.empty_bf16(s, n)
        cfg = L.make_muon_cfg(eps=1e-30)
        _run(g, n, None, None, 0, o, n, s, n, cfg)
        torch.cuda.synchronize()
        v = s ** -0.5
        for _ in range(5):
            v = NA * v + NB * v ** 3 + NC * v ** 5
        ref = rows.cuda() * v
        # the map's slope along the iterates is below 1.9 a step from here on; fp16 operands lose at most 3 * 2^-11 a step
        assert (o.double() - ref).norm() <= (UB + 5 * 3 * 2.0 ** -11) * ref.norm()


def test_muon_is_repeatable_on_another_stream_and_in_a_replayed_graph():
    import torch
    for rows, cols in ((48, 700), (257, 900), (2304, 1100)):
        gen = torch.Generator().manual_seed(rows)
        g, m = _gradient(gen, rows, cols, cols), _gradient(gen, rows, cols, cols)
        cfg = L.make_muon_cfg()
        outs = [(torch.empty_like(m), H.empty_bf16(rows, cols)) for _ in range(4)]
        _run(g, cols, m, outs[0][0], cols, outs[0][1], cols, rows, cols, cfg)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        ws1 = _run(g, cols, m, outs[1][0], cols, outs[1][1], cols, rows, cols, cfg, stream=side)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        ws2 = torch.empty(L.mt_muon_workspace_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        with torch.cuda.graph(graph):
            _run(g, cols, m, outs[2][0], cols, outs[2][1], cols, rows, cols, cfg, torch.cuda.current_stream(), ws2)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in outs[1:3]:
            assert torch.equal(a, outs[0][0]) and torch.equal(b, outs[0][1])
        g.mul_(-1.0)
        m.mul_(-1.0)
        graph.replay()  # the graph takes what its inputs hold now
        torch.cuda.synchronize()
        assert torch.equal(outs[2][1], -outs[0][1]) and torch.equal(outs[2][0], -outs[0][0])
        del ws1


def test_muon_updates_on_two_streams_at_once():
    """Two updates in flight together (each with its own workspace), of kernels that want every SM: the results of
    running alone, and no wait that ran out."""
    import torch
    shapes = [(300, 1100), (512, 3584), (60, 900), (1024, 2560)]
    gen = torch.Generator().manual_seed(17)
    cfg, sets = L.make_muon_cfg(), []
    for rows, cols in shapes:
        g, m = _gradient(gen, rows, cols, cols), _gradient(gen, rows, cols, cols)
        n = L.mt_muon_workspace_bytes(rows, cols)
        alone = (torch.empty_like(m), H.empty_bf16(rows, cols))
        _run(g, cols, m, alone[0], cols, alone[1], cols, rows, cols, cfg)
        sets.append((rows, cols, g, m, alone, [(torch.empty_like(m), H.empty_bf16(rows, cols), H.workspace(n)) for _ in range(2)]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for i in range(len(sets)):
            for k in range(2):  # different sizes side by side, too
                rows, cols, g, m, _, outs = sets[(i + k) % len(sets)]
                mo, o, ws = outs[k]
                _run(g, cols, m, mo, cols, o, cols, rows, cols, cfg, stream=streams[k], ws=ws)
    torch.cuda.synchronize()
    assert L.mt_device_error(clear=True) == 0
    for rows, cols, g, m, alone, outs in sets:
        for mo, o, _ in outs:
            assert torch.equal(mo, alone[0]) and torch.equal(o, alone[1]), (rows, cols)
