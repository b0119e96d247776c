"""Argument checks of LayerNorm and multi-axis rotary positions (nothing is enqueued: no GPU needed)."""
import numpy as np
import pytest

from host_offloaded_layer_b200 import _lib as L

BUF = np.zeros(4096, dtype=np.float32)
P = (BUF.ctypes.data + 63) // 64 * 64  # an aligned address that a refused call never reads


def _refused(name, fn, *args):
    with pytest.raises(L.MTError) as e:
        fn(*args)
    assert e.value.name == name
    assert L.last_error()


@pytest.mark.parametrize("bad,name", [
    (dict(x=None), "MT_ERR_INVALID_ARG"), (dict(y=None), "MT_ERR_INVALID_ARG"), (dict(rows=-1), "MT_ERR_INVALID_ARG"),
    (dict(H=0), "MT_ERR_INVALID_ARG"), (dict(ld_x=15), "MT_ERR_INVALID_ARG"), (dict(ld_y=15), "MT_ERR_INVALID_ARG"),
    (dict(eps=-1.0), "MT_ERR_INVALID_ARG"), (dict(eps=float("nan")), "MT_ERR_INVALID_ARG"),
    (dict(y=P, ld_y=24), "MT_ERR_INVALID_ARG"), (dict(x=P + 1), "MT_ERR_ALIGNMENT"), (dict(mean=P + 2), "MT_ERR_ALIGNMENT"),
    (dict(H=(1 << 28) + 1, ld_x=1 << 29, ld_y=1 << 29), "MT_ERR_UNSUPPORTED")])
def test_layernorm_forward_refuses(bad, name):
    a = dict(x=P, ld_x=16, g=P, b=P, y=P + 1024, ld_y=16, mean=P, rstd=P, rows=2, H=16, eps=1e-5)
    a.update(bad)
    _refused(name, L.mt_layernorm_fwd, *a.values())


@pytest.mark.parametrize("bad,name", [
    (dict(dy=None), "MT_ERR_INVALID_ARG"), (dict(x=None), "MT_ERR_INVALID_ARG"), (dict(mean=None), "MT_ERR_INVALID_ARG"),
    (dict(rstd=None), "MT_ERR_INVALID_ARG"), (dict(dx=None), "MT_ERR_INVALID_ARG"), (dict(ws=None), "MT_ERR_INVALID_ARG"),
    (dict(rows=-1), "MT_ERR_INVALID_ARG"), (dict(H=0), "MT_ERR_INVALID_ARG"), (dict(ld_dx=8), "MT_ERR_INVALID_ARG"),
    (dict(dres=P + 512, ld_dres=8), "MT_ERR_INVALID_ARG"), (dict(dx=P, ld_dx=24), "MT_ERR_INVALID_ARG"),
    (dict(dx=P + 256), "MT_ERR_INVALID_ARG"), (dict(ws_bytes=16), "MT_ERR_WORKSPACE"), (dict(dg=P + 2), "MT_ERR_ALIGNMENT"),
    (dict(ws=P + 8), "MT_ERR_ALIGNMENT")])
def test_layernorm_backward_refuses(bad, name):
    a = dict(dy=P, ld_dy=16, x=P + 256, ld_x=16, g=P, mean=P, rstd=P, dres=None, ld_dres=0, dx=P + 1024, ld_dx=16, dg=P, db=P,
             rows=2, H=16, ws=P, ws_bytes=1 << 20)
    a.update(bad)
    _refused(name, L.mt_layernorm_bwd, *a.values())


def test_layernorm_backward_workspace():
    assert L.mt_layernorm_bwd_workspace_bytes(-1, 8) == 0 and L.mt_layernorm_bwd_workspace_bytes(8, 0) == 0
    for rows in (0, 1, 100, 98304, 1 << 40):
        for width in (1, 7, 256, 3584, 8192, 8193, 1 << 20):
            n = L.mt_layernorm_bwd_workspace_bytes(rows, width)
            assert 2 * width * 4 <= n <= 4 * 148 * 2 * width * 4 + 256


@pytest.mark.parametrize("bad,name", [
    (dict(x=None), "MT_ERR_INVALID_ARG"), (dict(pos=None), "MT_ERR_INVALID_ARG"), (dict(sections=[]), "MT_ERR_INVALID_ARG"),
    (dict(sections=[1] * 9), "MT_ERR_INVALID_ARG"), (dict(sections=[-1, 4]), "MT_ERR_INVALID_ARG"),
    (dict(sections=[0, 0]), "MT_ERR_INVALID_ARG"), (dict(sections=[5, 4]), "MT_ERR_INVALID_ARG"),
    (dict(sections=[129], d=512, ld_x=2048, ld_y=2048), "MT_ERR_UNSUPPORTED"), (dict(rows=-1), "MT_ERR_INVALID_ARG"),
    (dict(heads=-1), "MT_ERR_INVALID_ARG"), (dict(d=0), "MT_ERR_INVALID_ARG"), (dict(theta=0.0), "MT_ERR_INVALID_ARG"),
    (dict(theta=float("inf")), "MT_ERR_INVALID_ARG"), (dict(ld_x=31), "MT_ERR_INVALID_ARG"),
    (dict(ld_y=31), "MT_ERR_INVALID_ARG"), (dict(ld_pos=3), "MT_ERR_INVALID_ARG"), (dict(y=P, ld_y=40), "MT_ERR_INVALID_ARG"),
    (dict(x=P + 1), "MT_ERR_ALIGNMENT"), (dict(pos=P + 2), "MT_ERR_ALIGNMENT")])
def test_mrope_refuses(bad, name):
    a = dict(x=P, ld_x=32, y=P + 1024, ld_y=32, pos=P, ld_pos=4, sections=[4, 4], rows=4, heads=2, d=16, theta=1e4)
    a.update(bad)
    _refused(name, L.mt_mrope, *a.values())


def test_layernorm_backward_workspace_is_nothing_for_a_width_that_the_call_refuses():
    for rows in (0, 1, 98304):
        assert L.mt_layernorm_bwd_workspace_bytes(rows, 1 << 28) >= 2 * (1 << 28) * 4
        assert L.mt_layernorm_bwd_workspace_bytes(rows, (1 << 28) + 1) == 0
        assert L.mt_layernorm_bwd_workspace_bytes(rows, 2 ** 31 - 1) == 0
    _refused("MT_ERR_UNSUPPORTED", L.mt_layernorm_bwd, P, 1 << 29, P + 256, 1 << 29, P, P, P, None, 0, P + 1024, 1 << 29, P, P, 2,
             (1 << 28) + 1, P, 1 << 62)
