"""LayerNorm at the ends of fp32's range, and rows far from zero against their spread: the register kernels (rows of
whole 16-byte granules, and of others) and the one that walks a row an element at a time give the same answers."""
import numpy as np
import pytest

import helpers as H
from host_offloaded_layer_b200 import _lib as L

pytestmark = pytest.mark.gpu

U, UB = 2.0 ** -24, 2.0 ** -8  # half a step of fp32 and of bf16, relative


def _strided(rows, width, ld, fill=0.0):
    import torch
    return torch.full((rows, ld), fill, dtype=torch.bfloat16, device="cuda")


def _forward(x, width, ld_y, g, b, eps):
    """y, mean, rstd of rows x [rows, ld_x]."""
    rows, ld_x = x.shape
    y, mean, rstd = _strided(rows, width, ld_y), H.empty_f32(rows), H.empty_f32(rows)
    L.mt_layernorm_fwd(x, ld_x, g, b, y, ld_y, mean, rstd, rows, width, eps)
    return y[:, :width], mean, rstd


# x's and y's row strides: whole granules alike, others alike, and unlike (the kernel for any operands)
PATHS = [(0, 0), (1, 1), (8, 1)]


@pytest.mark.parametrize("width", [8, 256, 1000, 3584, 5120, 8200])
@pytest.mark.parametrize("pad_x,pad_y", PATHS)
def test_variances_that_leave_fp32_and_none_at_all(width, pad_x, pad_y):
    """Elements of +-1e20: their squares are infinite in fp32, rstd = 0 and y = b. A row without spread and eps = 0: rstd
    is infinite and y NaN, as 0 times infinity is. In every kernel alike; the row between them is an ordinary one."""
    import torch
    gen = torch.Generator().manual_seed(width)
    rows = 37
    x = _strided(rows, width, width + pad_x)
    x[:, :width] = torch.randn(rows, width, generator=gen).cuda()
    big = torch.where(torch.arange(width) % 2 == 0, 1e20, -1e20).cuda()
    x[3, :width] = big
    x[5, :width] = 0.0
    b = torch.randn(width, generator=gen).bfloat16().cuda()
    y, mean, rstd = _forward(x, width, width + pad_y, None, b, 0.0)
    torch.cuda.synchronize()
    assert float(rstd[3]) == 0.0 and torch.equal(y[3], b)
    assert float(rstd[5]) == float("inf") and bool(y[5].isnan().all()) and float(mean[5]) == 0.0
    rest = [r for r in range(rows) if r not in (3, 5)]
    assert bool(torch.isfinite(y[rest]).all()) and bool(torch.isfinite(rstd[rest]).all())
    y, mean, rstd = _forward(x, width, width + pad_y, None, b, 1e-6)
    torch.cuda.synchronize()
    assert torch.equal(y[5], b) and abs(float(rstd[5]) - 1000.0) <= 4 * U * 1000 + 1e-3 * 1e-6


@pytest.mark.parametrize("width", [3, 7, 56, 896, 897, 3584, 3592, 7168, 14336])
@pytest.mark.parametrize("pad_x,pad_y", PATHS)
def test_rows_of_equal_elements_have_their_element_as_mean(width, pad_x, pad_y):
    """A bf16 element has 8 bits, and a sum of up to 2^16 equal ones fits fp32's 24 exactly, in whatever order: its quotient
    by H is the element, so x - mean is 0, the variance 0 and y = b bit for bit."""
    import torch
    vals = torch.tensor([1000.0, 5.5, -0.3359375, 3.0, 1e-3, 250.0, -7e4, 255.0, 1.0078125]).bfloat16().cuda()
    x = _strided(len(vals), width, width + pad_x)
    x[:, :width] = vals[:, None]
    gen = torch.Generator().manual_seed(width)
    g, b = (torch.randn(width, generator=gen).bfloat16().cuda() for _ in range(2))
    y, mean, rstd = _forward(x, width, width + pad_y, g, b, 1e-6)
    torch.cuda.synchronize()
    assert torch.equal(mean, vals.float())
    assert torch.equal(y, b[None].expand_as(y))
    assert bool(((rstd.double() - 1000.0).abs() <= 4 * U * 1000 + 1e-3).all())  # 1e-6 itself is half a step off in fp32


@pytest.mark.parametrize("rows,width", [(40, 256), (300, 1160), (64, 3584), (300, 1153), (20, 5120), (16, 5113), (7, 8200)])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_backward_of_rows_far_from_zero(rows, width, pad):
    """Rows at 1000, one bf16 step (4) up or down here and there, with a mean of 1000.1 and rstd 50: xh is the difference
    rounded (U) and the product rounded (U), whatever the mean's size. dx = rstd (w - c1) - (x - mean) rstd (rstd c2)
    + dres as written; sums of n terms carry 64 U of their absolute sum (test_gpu_norm_rope), the column sums the chain
    that is written there."""
    import torch
    gen = torch.Generator().manual_seed(width + pad)
    ld = width + pad
    x, dy, dx = _strided(rows, width, ld), _strided(rows, width, ld), _strided(rows, width, ld)
    x[:, :width] = (1000 + 4 * torch.randint(-1, 2, (rows, width), generator=gen)).cuda()
    dy[:, :width] = torch.randn(rows, width, generator=gen).cuda()
    mean, rstd = torch.full((rows,), 1000.1, device="cuda"), torch.full((rows,), 50.0, device="cuda")
    dg, db = H.empty_f32(width), H.empty_f32(width)
    n = L.mt_layernorm_bwd_workspace_bytes(rows, width)
    L.mt_layernorm_bwd(dy, ld, x, ld, None, mean, rstd, None, 0, dx, ld, dg, db, rows, width, H.workspace(n), n)
    torch.cuda.synchronize()
    w, x64 = H.host_f64(dy[:, :width].contiguous()), H.host_f64(x[:, :width].contiguous())
    m, r = H.host_f64(mean)[:, None], H.host_f64(rstd)[:, None]
    xh = (x64 - m) * r
    c1, c2 = w.mean(1, keepdims=True), (w * xh).mean(1, keepdims=True)
    ref = r * (w - c1 - xh * c2)
    e1, e2 = 66 * U * np.abs(w).mean(1, keepdims=True), 70 * U * np.abs(w * xh).mean(1, keepdims=True)
    err = r * (4 * U * (np.abs(w) + np.abs(c1) + np.abs(xh * c2)) + e1 + np.abs(xh) * e2 + 3 * U * np.abs(xh * c2))
    assert np.all(np.abs(H.host_f64(dx[:, :width].contiguous()) - ref) <= (UB + 2 * U) * np.abs(ref) + 1.01 * err)
    chain = rows / 32 + 64 + 4 * 148 / 8
    assert np.all(np.abs(H.host_f64(dg) - (w * xh).sum(0)) <= (chain + 3) * U * np.abs(w * xh).sum(0))


@pytest.mark.parametrize("lds,offs", [((0, 1, 2, 3), (0, 0, 0, 0)), ((8, 8, 8, 8), (0, 0, 0, 4)), ((8, 0, 8, 16), (0, 1, 0, 0)),
                                      ((0, 0, 0, 0), (0, 0, 0, 0))])
@pytest.mark.parametrize("rows,width", [(700, 512), (20000, 72), (130, 9000)])
def test_backward_of_operands_that_lie_unlike_and_of_one_sum_alone(rows, width, lds, offs):
    """dy, x, dres and dx with row strides and offsets of their own, in the kernels for any operands where these differ;
    dg and db each without the other are the same bit for bit. Bounds as in test_backward_of_rows_far_from_zero."""
    import torch
    gen = torch.Generator().manual_seed(width)
    views = []
    for extra, off in zip(lds, offs):
        ld = width + extra
        store = torch.full((off + rows * ld + 8,), float("nan"), dtype=torch.bfloat16, device="cuda")
        views.append((torch.as_strided(store, (rows, width), (ld, 1), off), ld))
        views[-1][0].copy_(torch.randn(rows, width, generator=gen).cuda())
    (dy, ld_dy), (x, ld_x), (dres, ld_dres), (dx, ld_dx) = views
    g = torch.randn(width, generator=gen).bfloat16().cuda()
    mean, rstd = torch.randn(rows, generator=gen).cuda(), (0.5 + torch.rand(rows, generator=gen)).cuda()
    n = L.mt_layernorm_bwd_workspace_bytes(rows, width)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    outs = [(H.empty_f32(width), H.empty_f32(width)), (H.empty_f32(width), None), (None, H.empty_f32(width))]
    got = []
    for dg, db in outs:
        dx.fill_(float("nan"))
        L.mt_layernorm_bwd(dy, ld_dy, x, ld_x, g, mean, rstd, dres, ld_dres, dx, ld_dx, dg, db, rows, width, ws, n)
        torch.cuda.synchronize()
        got.append(dx.clone())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[2][1])
    dy64, x64, r64, g64 = (H.host_f64(t.contiguous()) for t in (dy, x, dres, g))
    m, r = H.host_f64(mean)[:, None], H.host_f64(rstd)[:, None]
    xh, w = (x64 - m) * r, dy64 * g64
    c1, c2 = w.mean(1, keepdims=True), (w * xh).mean(1, keepdims=True)
    ref = r * (w - c1 - xh * c2) + r64
    e1, e2 = 70 * U * np.abs(w).mean(1, keepdims=True), 74 * U * np.abs(w * xh).mean(1, keepdims=True)
    err = r * (5 * U * (np.abs(w) + np.abs(c1) + np.abs(xh * c2)) + e1 + np.abs(xh) * e2 + 3 * U * np.abs(xh * c2))
    assert np.all(np.abs(H.host_f64(got[0]) - ref) <= (UB + 2 * U) * np.abs(ref) + 1.01 * err)
    chain = rows / 32 + 64 + 4 * 148 / 8
    assert np.all(np.abs(H.host_f64(outs[0][0]) - (dy64 * xh).sum(0)) <= (chain + 3) * U * np.abs(dy64 * xh).sum(0))
    assert np.all(np.abs(H.host_f64(outs[0][1]) - dy64.sum(0)) <= chain * U * np.abs(dy64).sum(0))
    assert L.mt_device_error(clear=True) == 0
