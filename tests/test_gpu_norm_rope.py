"""LayerNorm and multi-axis rotary positions on the B200 against float64, element by element.

Tolerances, derived from the arithmetic. u = 2^-24 (half an fp32 step), ub = 2^-8
(half a bf16 step, relative). A result rounded to bf16 once is off by ub |value|;
what fp32 adds before that is bounded by a few u times the magnitudes that were
added up, which each test writes out. Sums over n values carry at most
(log2-shaped or short sequential) n_seq u times the sum of magnitudes, n_seq the
longest chain of additions: 64 covers a thread's, a warp's and a group's for the
row sums; the column sums' chain is written where it is used.
"""
import numpy as np
import pytest

import helpers as H
from host_offloaded_layer_b200 import _lib as L

pytestmark = pytest.mark.gpu

U, UB = 2.0 ** -24, 2.0 ** -8
EPS = 1e-5


def _rows(gen, rows, width, ld, std=1.0, off=0):
    """A bf16 [rows, width] view with row stride ld, `off` elements into its storage, and the storage (a
    sentinel fills what lies between the rows)."""
    import torch
    store = torch.full((off + rows * ld + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    view = torch.as_strided(store, (rows, width), (ld, 1), off)
    view.copy_((torch.randn(rows, width, generator=gen) * std).cuda())
    return view, store


def _outside_untouched(store, rows, width, ld, off):
    import torch
    mask = torch.ones(store.numel(), dtype=torch.bool, device="cuda")
    torch.as_strided(mask, (rows, width), (ld, 1), off).fill_(False)
    return bool((store[mask] == 7.0).all())


def _within(got, ref, tol):
    got, ref, tol = np.broadcast_arrays(got, ref, tol)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} against {ref[bad][0]}, allowed {tol[bad][0]}"


# (rows, H, row stride, offset): one element, odd widths and strides, rows of 2- and 16-byte alignment,
# both register shapes of each pass and the widths around their borders, and rows too wide for registers
LN_SIZES = [(1, 1, 1, 0), (5, 2, 2, 0), (3, 7, 9, 1), (1, 8, 8, 0), (17, 64, 64, 0), (300, 256, 256, 0), (33, 257, 264, 0),
            (64, 264, 272, 8), (100, 1000, 1000, 2), (77, 1153, 1160, 0), (40, 2050, 2052, 2), (129, 3584, 3584, 0),
            (9, 4096, 4104, 0), (9, 4098, 4098, 0), (21, 5120, 5120, 0), (3, 8192, 8192, 0), (6, 8200, 8200, 0),
            (4, 8191, 8195, 3), (2, 16384, 16384, 0), (3, 16385, 16385, 0), (5000, 40, 40, 0), (1300, 896, 896, 0)]


@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("rows,width,ld,off", LN_SIZES + [(9000, 256, 256, 0), (4000, 3584, 3584, 0), (2500, 5119, 5121, 0)])
def test_layernorm_forward(rows, width, ld, off, affine):
    import torch
    gen = torch.Generator().manual_seed(rows * 7919 + width)
    x, xs = _rows(gen, rows, width, ld, off=off)
    # rows at levels far from zero against their spread
    x.add_((torch.randn(rows, 1, generator=gen) * 8).cuda())
    g = torch.randn(width, generator=gen).bfloat16().cuda() if affine else None
    b = torch.randn(width, generator=gen).bfloat16().cuda() if affine else None
    ys = torch.full_like(xs, 7.0)
    y = torch.as_strided(ys, (rows, width), (ld, 1), off)
    mean, rstd = H.empty_f32(rows), H.empty_f32(rows)
    L.mt_layernorm_fwd(x, ld, g, b, y, ld, mean, rstd, rows, width, EPS)
    torch.cuda.synchronize()
    x64 = H.host_f64(x)
    g64 = H.host_f64(g) if affine else np.ones(width)
    b64 = H.host_f64(b) if affine else np.zeros(width)
    eps = float(np.float32(EPS))
    m64 = x64.mean(1)
    c64 = x64 - m64[:, None]
    v64 = (c64 ** 2).mean(1)
    r64 = 1 / np.sqrt(v64 + eps)
    dm = 64 * U * np.abs(x64).mean(1) + 2 * U * np.abs(m64)   # the mean's error
    _within(H.host_f64(mean), m64, dm)
    # the variance of x - mean': the mean's own error adds its square, each difference one rounding (2u c^2)
    dv = (64 + 4) * U * v64 + dm ** 2
    drel = 0.5 * dv / (v64 + eps) + 4 * U
    _within(H.host_f64(rstd), r64, drel * r64)
    xh = c64 * r64[:, None]
    dxh = np.abs(xh) * (drel[:, None] + 3 * U) + dm[:, None] * r64[:, None]
    ref = xh * g64 + b64
    _within(H.host_f64(y), ref, (UB + 2 * U) * np.abs(ref) + 1.01 * (dxh * np.abs(g64) + 2 * U * np.abs(xh * g64)) + 1e-38)
    assert _outside_untouched(ys, rows, width, ld, off)
    # in place, without the statistics
    L.mt_layernorm_fwd(x, ld, g, b, x, ld, None, None, rows, width, EPS)
    torch.cuda.synchronize()
    assert torch.equal(x, y) and _outside_untouched(xs, rows, width, ld, off)


def _ln_bwd_ref(dy, x, mean, rstd, g, dres):
    xh = (x - mean[:, None]) * rstd[:, None]
    w = dy * g
    n = x.shape[1]
    c1, c2 = w.mean(1), (w * xh).mean(1)
    dx = rstd[:, None] * (w - c1[:, None] - xh * c2[:, None]) + dres
    return xh, w, c1, c2, dx, (dy * xh).sum(0), dy.sum(0), n


# many rows for every group, so that each ring goes round: its shapes are those of 8 to 40 warps of one or two vectors, with
# and without a third operand
LN_ROUNDS = [(4000, 64, 72, 0), (9000, 256, 256, 0), (5000, 1024, 1024, 0), (3300, 2048, 2048, 0), (2600, 3584, 3584, 0),
             (2600, 4104, 4104, 0), (2500, 5120, 5120, 0), (1900, 6144, 6144, 0), (1800, 8192, 8192, 0), (2500, 5119, 5121, 0),
             (1800, 8180, 8180, 2), (5001, 777, 777, 0)]


@pytest.mark.parametrize("affine,res,alias", [(True, True, None), (True, False, "dy"), (False, True, "dres")])
@pytest.mark.parametrize("rows,width,ld,off", LN_SIZES + LN_ROUNDS + [(0, 24, 24, 0)])
def test_layernorm_backward(rows, width, ld, off, affine, res, alias):
    import torch
    gen = torch.Generator().manual_seed(rows * 7919 + width)
    x, _ = _rows(gen, rows, width, ld, off=off)
    dy, dys = _rows(gen, rows, width, ld, off=off)
    dres, drs = _rows(gen, rows, width, ld, off=off) if res else (None, None)
    g = torch.randn(width, generator=gen).bfloat16().cuda() if affine else None
    mean = torch.randn(rows, generator=gen).cuda()   # the saved statistics are inputs of their own
    rstd = (0.5 + torch.rand(rows, generator=gen)).cuda()
    outs = dys if alias == "dy" else drs if alias == "dres" else torch.full_like(dys, 7.0)
    dx = torch.as_strided(outs, (rows, width), (ld, 1), off)
    dg, db = H.empty_f32(width), H.empty_f32(width)
    n = L.mt_layernorm_bwd_workspace_bytes(rows, width)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns: nothing may be read before it is written
    i64 = [H.host_f64(t) if t is not None else None for t in (dy, x, mean, rstd, g, dres)]
    i64[4] = np.ones(width) if g is None else i64[4]
    i64[5] = np.zeros((rows, width)) if dres is None else i64[5]
    xh, w, c1, c2, rdx, rdg, rdb, _ = _ln_bwd_ref(*i64)
    L.mt_layernorm_bwd(dy, ld, x, ld, g, mean, rstd, dres, ld, dx, ld, dg, db, rows, width, ws, n)
    torch.cuda.synchronize()
    ax = (np.abs(i64[1]) + np.abs(i64[2])[:, None]) * np.abs(i64[3])[:, None]  # |x| + |mean|, scaled: what xh's rounding goes by
    dxh = 3 * U * ax
    if rows:
        e1 = 66 * U * np.abs(w).mean(1)
        e2 = 68 * U * np.abs(w * xh).mean(1) + (np.abs(w) * dxh).mean(1)
        err = np.abs(i64[3])[:, None] * (4 * U * (np.abs(w) + np.abs(c1)[:, None] + np.abs(xh * c2[:, None])) + e1[:, None]
                                         + np.abs(xh) * e2[:, None] + dxh * np.abs(c2)[:, None])
        _within(H.host_f64(dx), rdx, UB * np.abs(rdx) + 1.01 * err + 2 * U * np.abs(rdx) + 1e-38)
    # the column sums' longest chain: a group's rows, then groups, then partial rows
    chain = rows / 32 + 64 + 4 * 148 / 8
    _within(H.host_f64(dg), rdg, chain * U * np.abs(i64[0] * xh).sum(0) + (np.abs(i64[0]) * dxh).sum(0) + 1e-38)
    _within(H.host_f64(db), rdb, chain * U * np.abs(i64[0]).sum(0) + 1e-38)
    assert L.mt_device_error(clear=True) == 0  # no wait ran out
    if rows:
        assert _outside_untouched(outs, rows, width, ld, off)
    # again, bit for bit, without the column sums
    if alias is None and rows:
        dx2 = torch.as_strided(torch.full_like(dys, 7.0), (rows, width), (ld, 1), off)
        L.mt_layernorm_bwd(dy, ld, x, ld, g, mean, rstd, dres, ld, dx2, ld, None, None, rows, width, ws, n)
        dg2, db2 = H.empty_f32(width), H.empty_f32(width)
        L.mt_layernorm_bwd(dy, ld, x, ld, g, mean, rstd, dres, ld, dx, ld, dg2, db2, rows, width, ws, n)
        torch.cuda.synchronize()
        assert torch.equal(dx, dx2) and torch.equal(dg, dg2) and torch.equal(db, db2)


def test_layernorm_backward_is_the_forwards_derivative():
    """dx, dg and db against central differences of a float64 LayerNorm that shares the kernel's inputs."""
    import torch
    rows, width = 5, 48
    gen = torch.Generator().manual_seed(3)
    x, _ = _rows(gen, rows, width, width)
    dy, _ = _rows(gen, rows, width, width)
    g = torch.randn(width, generator=gen).bfloat16().cuda()
    b = torch.randn(width, generator=gen).bfloat16().cuda()
    y, dx = H.empty_bf16(rows, width), H.empty_bf16(rows, width)
    mean, rstd, dg, db = H.empty_f32(rows), H.empty_f32(rows), H.empty_f32(width), H.empty_f32(width)
    L.mt_layernorm_fwd(x, width, g, b, y, width, mean, rstd, rows, width, EPS)
    n = L.mt_layernorm_bwd_workspace_bytes(rows, width)
    ws = H.workspace(n)
    L.mt_layernorm_bwd(dy, width, x, width, g, mean, rstd, None, 0, dx, width, dg, db, rows, width, ws, n)
    torch.cuda.synchronize()
    x64, dy64, g64, b64 = (H.host_f64(t) for t in (x, dy, g, b))

    def loss(x_, g_, b_):
        c = x_ - x_.mean(1, keepdims=True)
        return (dy64 * (c / np.sqrt((c ** 2).mean(1, keepdims=True) + float(np.float32(EPS))) * g_ + b_)).sum()

    h = 1e-5

    def diff(arr, at):
        out = np.zeros_like(arr)
        for i in np.ndindex(arr.shape):
            up, dn = arr.copy(), arr.copy()
            up[i] += h
            dn[i] -= h
            out[i] = (loss(*at(up)) - loss(*at(dn))) / (2 * h)
        return out

    # central differences: h^2 of truncation and 2^-53 / h of rounding, both below 1e-8 of these sums
    ndx = diff(x64, lambda v: (v, g64, b64))
    _within(H.host_f64(dx), ndx, UB * np.abs(ndx) + 1e-5)
    _within(H.host_f64(dg), diff(g64, lambda v: (x64, v, b64)), 1e-5)
    _within(H.host_f64(db), diff(b64, lambda v: (x64, g64, v)), 1e-5)


def test_layernorm_rows_with_infinities_and_nan_leave_the_other_rows_alone():
    import torch
    rows, width = 40, 512
    gen = torch.Generator().manual_seed(4)
    x, _ = _rows(gen, rows, width, width)
    x[3, 5], x[7, 500], x[11, 0] = float("inf"), float("nan"), float("-inf")
    x[20] = 2.5  # a row without spread: xh = 0
    y = torch.empty_like(x)
    mean, rstd = H.empty_f32(rows), H.empty_f32(rows)
    L.mt_layernorm_fwd(x, width, None, None, y, width, mean, rstd, rows, width, EPS)
    dx, n = torch.empty_like(x), L.mt_layernorm_bwd_workspace_bytes(rows, width)
    dy, _ = _rows(gen, rows, width, width)
    L.mt_layernorm_bwd(dy, width, x, width, None, mean, rstd, None, 0, dx, width, None, None, rows, width,
                       H.workspace(n), n)
    torch.cuda.synchronize()
    bad = torch.zeros(rows, dtype=torch.bool)
    bad[[3, 7, 11]] = True
    assert torch.equal(y.isnan().any(1).cpu(), bad) and torch.equal(dx.isnan().any(1).cpu(), bad)
    assert bool((y[20] == 0).all()) and bool(torch.isfinite(dx[20]).all())


# ------------------------------------------------------------------ rotary positions
def _mrope_ref(x, pos, sections, heads, d, theta, interleaved, per_axis, inverse):
    """float64, from the definition; x [rows, heads * d], pos [axes, rows]."""
    left, order = list(sections), []
    if interleaved:
        while sum(left):
            for a in range(len(sections)):
                if left[a]:
                    order.append((a, sections[a] - left[a]))
                    left[a] -= 1
    else:
        order = [(a, j) for a, s in enumerate(sections) for j in range(s)]
    P = len(order)
    y = x.reshape(len(x), heads, d).copy()
    src = y.copy()
    for i, (a, j) in enumerate(order):
        w = theta ** (-j / sections[a]) if per_axis else theta ** (-i / P)
        ang = pos[a].astype(np.float64) * w * (-1 if inverse else 1)
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        y[:, :, i] = src[:, :, i] * c - src[:, :, P + i] * s
        y[:, :, P + i] = src[:, :, P + i] * c + src[:, :, i] * s
    mag = np.zeros_like(y)
    mag[:, :, :P] = mag[:, :, P:2 * P] = np.abs(src[:, :, :P]) + np.abs(src[:, :, P:2 * P])
    return y.reshape(len(x), -1), mag.reshape(len(x), -1)


# rows, heads, d, sections, ld, offset: whole and partial rotation, one axis and many, vectors of 8, 4, 2 and 1
MROPE = [(1, 1, 2, [1], 2, 0), (3, 1, 16, [8], 16, 0), (128, 6, 64, [8, 12, 12], 512, 0), (50, 3, 128, [16, 24, 24], 384, 0),
         (1000, 32, 128, [24, 20, 20], 4608, 0), (77, 5, 80, [20, 20], 400, 0), (33, 2, 72, [18, 18], 144, 0),
         (19, 3, 20, [3, 2, 1], 61, 1), (9, 4, 256, [64, 32, 32], 1024, 0), (65, 2, 96, [4, 12, 8], 208, 0),
         (13, 2, 25, [2, 3, 1, 4], 50, 0), (700, 1, 32, [0, 16], 33, 0), (40, 2, 192, [1, 1, 1, 1, 1, 1, 1, 1], 384, 8),
         (5, 3, 36, [9, 9], 108, 2), (3, 700, 64, [32], 44800, 0)]


@pytest.mark.parametrize("interleaved,per_axis,inverse", [(0, 0, 0), (0, 1, 1), (1, 0, 1), (1, 1, 0)])
@pytest.mark.parametrize("rows,heads,d,sections,ld,off", MROPE)
def test_mrope(rows, heads, d, sections, ld, off, interleaved, per_axis, inverse):
    import torch
    gen = torch.Generator().manual_seed(rows + d)
    width = heads * d
    x, xs = _rows(gen, rows, width, ld, off=off)
    pos = torch.randint(-5, 3000, (len(sections), rows + 3), generator=gen, dtype=torch.int32)
    pos[:, 0] = torch.tensor([2 ** 31 - 1, -2 ** 31, 1 << 24, 1 << 20, 0, 1, 2, 3], dtype=torch.int64)[:len(sections)].int()
    ys = torch.full_like(xs, 7.0)
    y = torch.as_strided(ys, (rows, width), (ld, 1), off)
    args = (pos.cuda(), rows + 3, sections, rows, heads, d, 1e4, interleaved, per_axis, inverse)
    L.mt_mrope(x, ld, y, ld, *args)
    torch.cuda.synchronize()
    ref, mag = _mrope_ref(H.host_f64(x), pos[:, :rows].numpy(), sections, heads, d, 1e4, interleaved, per_axis, inverse)
    # cos and sin: the angle's fraction of a turn rounded to fp32 (pi u), the function (2u each, 2 ulp), and what fp64
    # leaves of 2^31 positions (2^31 turns/2pi * 4 * 2^-53 in turns, on either side); then two products and a sum
    trig = 4 * U + 2 * U + 4 * 2.0 ** 31 * 2.0 ** -53 * 2
    _within(H.host_f64(y), ref, UB * np.abs(ref) + 1.01 * mag * (trig + 3 * U) + 1e-38)
    assert _outside_untouched(ys, rows, width, ld, off)
    # in place
    L.mt_mrope(x, ld, x, ld, *args)
    torch.cuda.synchronize()
    assert torch.equal(x, y) and _outside_untouched(xs, rows, width, ld, off)


def test_mrope_of_one_axis_is_rope():
    """Positions 0..T-1 on one axis, all pairs: the operator that the layer uses (bf16 results, equal but for
    values at a rounding border, which are one step apart)."""
    import torch
    B, T, heads, d = 2, 300, 5, 128
    gen = torch.Generator().manual_seed(9)
    x, _ = _rows(gen, B * T, heads * d, heads * d)
    y = torch.empty_like(x)
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(B)
    L.mt_mrope(x, heads * d, y, heads * d, pos, B * T, [d // 2], B * T, heads, d, 1e6)
    L.mt_rope(x, heads * d, B, T, heads, d, 1e6, False)
    torch.cuda.synchronize()
    a, b = H.host_f64(x), H.host_f64(y)
    assert np.all(np.abs(a - b) <= 2 * UB * np.maximum(np.abs(a), np.abs(b)) + 16 * U * 8)
    assert (a != b).mean() < 1e-3


def test_mrope_inverse_is_the_adjoint():
    """<dy, R x> = <R^T dy, x> in float64 sums over the kernels' own outputs: both sides carry bf16 roundings
    of single elements (ub |y| |dy| each, of random sign), so n of them stay within ub sqrt(n) 8 of their rms."""
    import torch
    rows, heads, d, sections = 257, 3, 80, [10, 14, 16]
    gen = torch.Generator().manual_seed(11)
    x, _ = _rows(gen, rows, heads * d, heads * d)
    dy, _ = _rows(gen, rows, heads * d, heads * d)
    pos = torch.randint(0, 100000, (3, rows), generator=gen, dtype=torch.int32).cuda()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    ld = heads * d
    L.mt_mrope(x, ld, y, ld, pos, rows, sections, rows, heads, d, 1e4, True)
    L.mt_mrope(dy, ld, dx, ld, pos, rows, sections, rows, heads, d, 1e4, True, False, True)
    torch.cuda.synchronize()
    x, dy, y, dx = (H.host_f64(t) for t in (x, dy, y, dx))
    assert abs((dy * y).sum() - (dx * x).sum()) <= 8 * UB * (np.sqrt(((dy * y) ** 2).sum()) + np.sqrt(((dx * x) ** 2).sum()))


def test_calls_on_another_stream_and_in_a_replayed_graph():
    import torch
    rows, width = 600, 896
    gen = torch.Generator().manual_seed(13)
    x, _ = _rows(gen, rows, width, width)
    dy, _ = _rows(gen, rows, width, width)
    pos = torch.randint(0, 500, (3, rows), generator=gen, dtype=torch.int32).cuda()
    n = L.mt_layernorm_bwd_workspace_bytes(rows, width)

    def make():
        return dict(y=torch.empty_like(x), r=torch.empty_like(x), dx=torch.empty_like(x), mean=H.empty_f32(rows),
                    rstd=H.empty_f32(rows), dg=H.empty_f32(width), db=H.empty_f32(width), ws=H.workspace(n))

    def go(o, stream):
        L.mt_layernorm_fwd(x, width, None, None, o["y"], width, o["mean"], o["rstd"], rows, width, EPS, stream)
        L.mt_mrope(o["y"], width, o["r"], width, pos, rows, [16, 24, 24], rows, 7, 128, 1e6, stream=stream)
        L.mt_layernorm_bwd(dy, width, x, width, None, o["mean"], o["rstd"], o["r"], width, o["dx"], width, o["dg"], o["db"],
                           rows, width, o["ws"], n, stream)

    want = make()
    go(want, None)
    torch.cuda.synchronize()
    side, a = torch.cuda.Stream(), make()
    go(a, side)
    side.synchronize()
    b, graph = make(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(b, torch.cuda.current_stream())
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    half = make()
    go(half, None)
    torch.cuda.synchronize()
    for k in ("y", "r", "dx", "mean", "rstd", "dg", "db"):
        assert torch.equal(a[k], want[k]) and torch.equal(b[k], half[k]), k


def test_layernorm_passes_on_two_streams_at_once():
    """Forward and backward of different sizes in flight together, each backward with its own workspace."""
    import torch
    gen = torch.Generator().manual_seed(23)
    sets = []
    for rows, width in ((4000, 3584), (3000, 777), (2000, 5120), (6000, 256)):
        x, dy = _rows(gen, rows, width, width)[0], _rows(gen, rows, width, width)[0]
        n = L.mt_layernorm_bwd_workspace_bytes(rows, width)
        outs = [dict(y=torch.empty_like(x), dx=torch.empty_like(x), mean=H.empty_f32(rows), rstd=H.empty_f32(rows),
                     dg=H.empty_f32(width), db=H.empty_f32(width), ws=H.workspace(n)) for _ in range(3)]
        sets.append((rows, width, x, dy, n, outs))

    def go(s, o, stream):
        rows, width, x, dy, n, _ = s
        L.mt_layernorm_fwd(x, width, None, None, o["y"], width, o["mean"], o["rstd"], rows, width, EPS, stream)
        L.mt_layernorm_bwd(dy, width, x, width, None, o["mean"], o["rstd"], None, 0, o["dx"], width, o["dg"], o["db"], rows, width,
                           o["ws"], n, stream)

    for s in sets:
        go(s, s[5][0], None)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for i in range(len(sets)):
            for k in range(2):
                s = sets[(i + k) % len(sets)]
                go(s, s[5][1 + k], streams[k])
    torch.cuda.synchronize()
    assert L.mt_device_error(clear=True) == 0
    for s in sets:
        for o in s[5][1:]:
            for k in ("y", "dx", "mean", "rstd", "dg", "db"):
                assert torch.equal(o[k], s[5][0][k]), (s[:2], k)


def test_mrope_of_very_wide_rows():
    """One pair a head and half a million heads: a tile's work passes what few wide heads have."""
    import torch
    rows, heads = 5, 500000
    gen = torch.Generator().manual_seed(29)
    x, _ = _rows(gen, rows, heads * 2, heads * 2)
    y, pos = torch.empty_like(x), torch.arange(rows, dtype=torch.int32, device="cuda")
    L.mt_mrope(x, heads * 2, y, heads * 2, pos, rows, [1], rows, heads, 2, 1e4)
    torch.cuda.synchronize()
    ref, mag = _mrope_ref(H.host_f64(x), pos.cpu().numpy()[None], [1], heads, 2, 1e4, 0, 0, 0)
    _within(H.host_f64(y), ref, UB * np.abs(ref) + 10 * U * mag + 1e-38)


@pytest.mark.parametrize("off", [0, 1, 3, 6, 7])
@pytest.mark.parametrize("gap", [0, 1, 2, 4, 8])
def test_layernorm_rows_around_one_granule(off, gap):
    """Rows that start and end anywhere in their 16-byte granules: none, one or two whole ones, and elements before and
    behind them."""
    for width in (1, 2, 5, 7, 8, 9, 13, 15, 16, 17, 22, 31):
        test_layernorm_forward(19, width, width + gap, off, True)
        test_layernorm_backward(19, width, width + gap, off, True, True, None)


# three warps a row: five groups to a CTA, every ring many times round
@pytest.mark.parametrize("rows,width,ld,off", [(9000, 1152, 1152, 0), (9000, 1153, 1160, 0), (9000, 1401, 1401, 3), (8, 1536, 1536, 0),
                                               (741, 1280, 1284, 0), (2960, 1031, 1031, 0)])
def test_layernorm_of_three_warps_a_row(rows, width, ld, off):
    test_layernorm_forward(rows, width, ld, off, True)
    test_layernorm_backward(rows, width, ld, off, True, False, "dy")
    test_layernorm_backward(rows, width, ld, off, True, True, None)


@pytest.mark.parametrize("rows,width,ld,off", [(37, 9, 12, 1), (300, 257, 261, 0), (50, 1153, 1160, 0), (40, 4999, 5003, 5), (7, 8200, 8204, 0)])
def test_layernorm_takes_nothing_from_between_the_rows(rows, width, ld, off):
    """NaN between the rows and around them changes no bit of any result, and stays there."""
    import torch
    got = []
    for fill in (7.0, float("nan")):
        gen = torch.Generator().manual_seed(width)
        def padded():
            store = torch.full((off + rows * ld + 8,), fill, dtype=torch.bfloat16, device="cuda")
            view = torch.as_strided(store, (rows, width), (ld, 1), off)
            view.copy_(torch.randn(rows, width, generator=gen).cuda())
            return view, store
        x, _ = padded()
        dy, _ = padded()
        dres, _ = padded()
        y, ys = padded()
        dx, dxs = padded()
        g = torch.randn(width, generator=gen).bfloat16().cuda()
        mean, rstd, dg, db = H.empty_f32(rows), H.empty_f32(rows), H.empty_f32(width), H.empty_f32(width)
        n = L.mt_layernorm_bwd_workspace_bytes(rows, width)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        L.mt_layernorm_fwd(x, ld, g, g, y, ld, mean, rstd, rows, width, EPS)
        L.mt_layernorm_bwd(dy, ld, x, ld, g, mean, rstd, dres, ld, dx, ld, dg, db, rows, width, ws, n)
        torch.cuda.synchronize()
        for store in (ys, dxs):
            outside = torch.ones(store.numel(), dtype=torch.bool, device="cuda")
            torch.as_strided(outside, (rows, width), (ld, 1), off).fill_(False)
            assert bool(torch.isnan(store[outside]).all()) if fill != fill else bool((store[outside] == fill).all())
        got.append([t.clone() for t in (y, mean, rstd, dx, dg, db)])
    assert all(torch.equal(a, b) for a, b in zip(*got))
