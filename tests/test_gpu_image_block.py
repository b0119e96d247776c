"""LayerNorm, projection, multi-axis rotary positions and attention, their backward and the Muon update of the
projection's weight, as one attention block of image tokens would run them: the library's calls in a row
against float64 autograd over the same bf16 inputs.

Every intermediate is rounded to bf16 (2^-8 of its value at most, about 2^-9 rms) and the chain has six such
roundings forward and five back, each passed on by maps of norm about one: 2e-2 per tensor, the bound that the
layer's parity tests use, holds them with room.
"""
import numpy as np
import pytest

import helpers as H
from host_offloaded_layer_b200 import _lib as L

pytestmark = pytest.mark.gpu

EPS, THETA = 1e-6, 1e4


def _turn(x, ang):
    """Rotate-half in float64: x [B, T, heads, d], ang [B * T, d/2]."""
    import torch
    B, T, n, d = x.shape
    a, b = x[..., :d // 2], x[..., d // 2:]
    c, s = torch.cos(ang).reshape(B, T, 1, d // 2), torch.sin(ang).reshape(B, T, 1, d // 2)
    return torch.cat([a * c - b * s, b * c + a * s], -1)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_block_of_image_tokens_trains(d):
    import torch
    B, T, nq, nkv = 2, 200, 4, 2
    hid, sections = 4 * d, [d // 8, d // 8, d // 4]
    M, Nqk, N = B * T, (nq + nkv) * d, (nq + 2 * nkv) * d
    gen = torch.Generator().manual_seed(d)

    def bf(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen) * std + mean).bfloat16().cuda()

    x, g, b, w, bias = bf(M, hid), bf(hid, std=0.1, mean=1.0), bf(hid, std=0.1), bf(N, hid, std=hid ** -0.5), bf(N, std=0.1)
    d_o = bf(M, nq * d, std=0.1)
    t = torch.arange(T, dtype=torch.int32)
    pos = torch.stack([t // 40, (t // 8) % 5, t % 8]).repeat(1, B).contiguous().cuda()  # frames of 5 x 8 patches

    # the library
    h, mean, rstd = H.empty_bf16(M, hid), H.empty_f32(M), H.empty_f32(M)
    qkv, o, lse = H.empty_bf16(M, N), H.empty_bf16(M, nq * d), H.empty_f32(B, nq, T)
    L.mt_layernorm_fwd(x, hid, g, b, h, hid, mean, rstd, M, hid, EPS)
    L.mt_gemm_bf16(h, hid, 0, w, hid, 0, qkv, N, 0, 0, M, N, hid, bias)
    L.mt_mrope(qkv, N, qkv, N, pos, M, sections, M, nq + nkv, d, THETA)
    L.mt_attention_fwd(qkv, N, o, nq * d, lse, B, T, nq, nkv, d)
    dqkv, dh, dw = H.empty_bf16(M, N), H.empty_bf16(M, hid), H.empty_f32(N, hid)
    n = L.mt_attention_bwd_workspace_bytes(B, T, nq)
    L.mt_attention_bwd(qkv, N, o, d_o, nq * d, lse, dqkv, B, T, nq, nkv, d, H.workspace(n), n)
    L.mt_mrope(dqkv, N, dqkv, N, pos, M, sections, M, nq + nkv, d, THETA, inverse=True)
    L.mt_gemm_bf16(dqkv, N, 0, w, hid, 1, dh, hid, 0, 0, M, hid, N)
    L.mt_gemm_bf16(dqkv, N, 1, h, hid, 1, dw, hid, 1, 0, N, hid, M)
    dx, dg, db = H.empty_bf16(M, hid), H.empty_f32(hid), H.empty_f32(hid)
    n = L.mt_layernorm_bwd_workspace_bytes(M, hid)
    L.mt_layernorm_bwd(dh, hid, x, hid, g, mean, rstd, None, 0, dx, hid, dg, db, M, hid, H.workspace(n), n)
    mom = torch.zeros(N, hid, device="cuda")
    upd, cfg = H.empty_bf16(N, hid), L.make_muon_cfg()
    n = L.mt_muon_workspace_bytes(N, hid)
    L.mt_muon_update(dw, hid, mom, mom, hid, upd, hid, N, hid, cfg, H.workspace(n), n)
    torch.cuda.synchronize()
    assert L.mt_device_error(clear=True) == 0

    # float64
    x6, g6, b6, w6, bias6 = (v.double().requires_grad_() for v in (x, g, b, w, bias))
    c = x6 - x6.mean(1, keepdim=True)
    h6 = c / torch.sqrt((c * c).mean(1, keepdim=True) + EPS) * g6 + b6
    y = (h6 @ w6.T + bias6).reshape(B, T, nq + 2 * nkv, d)
    axis = torch.tensor([a for a, s in enumerate(sections) for _ in range(s)], device="cuda")
    freq = THETA ** (-torch.arange(d // 2, device="cuda").double() / (d // 2))
    ang = pos.index_select(0, axis).T.double() * freq
    q, k, v = _turn(y[:, :, :nq], ang), _turn(y[:, :, nq:nq + nkv], ang), y[:, :, nq + nkv:]
    k, v = (u.repeat_interleave(nq // nkv, dim=2) for u in (k, v))
    s = torch.einsum("bthd,bshd->bhts", q, k) / d ** 0.5
    s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
    o6 = torch.einsum("bhts,bshd->bthd", s.softmax(-1), v).reshape(M, nq * d)
    o6.backward(d_o.double())
    for name, got, ref in (("o", o, o6), ("dw", dw, w6.grad), ("dx", dx, x6.grad), ("dg", dg, g6.grad), ("db", db, b6.grad)):
        assert H.rel(H.host_f64(got), ref.detach().cpu().numpy()) < H.TOL, name

    # the update of the gradient that the block left: u = g + 0.95 m', m' = g
    u = dw.double() * (1 + float(np.float32(0.95)))
    z = (u / (u.norm() + cfg.eps)).T if N > hid else u / (u.norm() + cfg.eps)
    for _ in range(5):
        a = z @ z.T
        z = 3.4445 * z + (-4.7750 * a + 2.0315 * a @ a) @ z
    assert torch.equal(mom, dw)
    assert H.rel(H.host_f64(upd), (z.T if N > hid else z).cpu().numpy()) < 2.0 ** -8 + 4e-3
