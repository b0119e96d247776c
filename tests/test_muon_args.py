"""Argument checks and workspace sizes of the Muon update (nothing is enqueued: no GPU needed)."""
import numpy as np
import pytest

from host_offloaded_layer_b200 import _lib as L

BUF = np.zeros(4096, dtype=np.float32)
P = (BUF.ctypes.data + 255) // 256 * 256  # an aligned address that a refused call never reads


@pytest.mark.parametrize("bad,name", [
    (dict(g=None), "MT_ERR_INVALID_ARG"), (dict(o=None), "MT_ERR_INVALID_ARG"), (dict(m_in=None), "MT_ERR_INVALID_ARG"),
    (dict(m_out=None), "MT_ERR_INVALID_ARG"), (dict(ws=None), "MT_ERR_INVALID_ARG"), (dict(rows=-1), "MT_ERR_INVALID_ARG"),
    (dict(rows=1 << 20, cols=(1 << 16) + 1, ld_g=1 << 17, ld_m=1 << 17, ld_o=1 << 17), "MT_ERR_UNSUPPORTED"),
    (dict(cols=1 << 31, ld_g=1 << 32, ld_m=1 << 32, ld_o=1 << 32), "MT_ERR_INVALID_ARG"), (dict(ld_g=7), "MT_ERR_INVALID_ARG"),
    (dict(ld_m=7), "MT_ERR_INVALID_ARG"), (dict(ld_o=7), "MT_ERR_INVALID_ARG"), (dict(cfg=dict(steps=0)), "MT_ERR_INVALID_ARG"),
    (dict(cfg=dict(steps=101)), "MT_ERR_INVALID_ARG"), (dict(cfg=dict(eps=0.0)), "MT_ERR_INVALID_ARG"),
    (dict(cfg=dict(momentum=float("nan"))), "MT_ERR_INVALID_ARG"), (dict(cfg=dict(scale=float("inf"))), "MT_ERR_INVALID_ARG"),
    (dict(ws_bytes=255), "MT_ERR_WORKSPACE"), (dict(g=P + 2), "MT_ERR_ALIGNMENT"), (dict(o=P + 1), "MT_ERR_ALIGNMENT"),
    (dict(ws=P + 128), "MT_ERR_ALIGNMENT")])
def test_muon_refuses(bad, name):
    a = dict(g=P, ld_g=8, m_in=P, m_out=P, ld_m=8, o=P, ld_o=8, rows=8, cols=8, cfg={}, ws=P, ws_bytes=1 << 30)
    a.update(bad)
    a["cfg"] = L.make_muon_cfg(**a["cfg"])
    with pytest.raises(L.MTError) as e:
        L.mt_muon_update(*a.values())
    assert e.value.name == name and L.last_error()


def test_empty_matrices_are_nothing_to_do():
    cfg = L.make_muon_cfg()
    assert L.mt_muon_workspace_bytes(0, 5) == 0 and L.mt_muon_workspace_bytes(5, -1) == 0
    L.mt_muon_update(None, 5, None, None, 0, None, 5, 0, 5, cfg, None, 0)
    L.mt_muon_update(None, 0, None, None, 0, None, 0, 5, 0, cfg, None, 0)


def test_workspace_holds_three_copies_of_x_and_its_square_matrices():
    """Two square matrices, three where the long side is at least twice the short one; in small matrices, parts of one
    product (fp32 tiles of 128 x 128) for 148 SMs at most."""
    for rows, cols in ((65, 65), (512, 3584), (18944, 3584), (1000, 70), (40000, 300), (688, 256)):
        m = min(rows, cols)
        n = L.mt_muon_workspace_bytes(rows, cols)
        up = lambda v: -(-v // 64) * 64  # noqa: E731
        need = 2 * (3 * rows * up(cols) + 2 * m * up(m)) + 592 * 8
        assert need <= n <= need + 2 * m * up(m) + 148 * 128 * 128 * 4 + 9 * 256
    for rows, cols in ((1, 1), (64, 100000), (100000, 3)):
        assert 0 < L.mt_muon_workspace_bytes(rows, cols) <= 148 * 64 * 64 * 8 + 64 * 64 * 4 + 512


def test_the_order_of_sums_is_chosen_by_the_matrix_alone():
    """No function that chooses a path, a split of K or the parts of a workspace asks for the device's SMs (read from the
    source: there is one kind of device to run on)."""
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "host_offloaded_layer_b200", "csrc", "muon.cu")
    with open(path) as f:
        code = f.read()
    for name in ("int pick_split(", "bool pick_fused(", "int fused_split(", "bool pair_first_steps(", "Plan plan("):
        at = code.index("\n" + name)
        assert "num_sms" not in code[at:code.index("\n}", at)], name
