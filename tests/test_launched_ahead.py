"""Kernels that start before the one in front of them has ended: what they read of it is neither declared read-only
for their whole run (in the source), nor left over from a call before (on the GPU)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "host_offloaded_layer_b200", "csrc")


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith(".cu")))
def test_kernels_launched_ahead_promise_nothing_about_what_they_wait_for(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"\n(?:template[^\n]*\n)?__(?:global|device)__[^;{]*?(\w+)\(([^{;]*)\)\s*\{", code):
        body = code[m.end():code.index("\n}\n", m.end())]
        waits = "griddepcontrol.wait" in body or "wait_for_last()" in body or m.group(1) == "scale_pass"
        if waits:
            assert not re.search(r"const\s+\w+\s*\*\s*__restrict__", m.group(2)), m.group(1)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,width", [(300, 256), (4000, 3584), (2000, 1153), (40, 8200)])
def test_layernorm_backward_takes_nothing_from_the_workspace_of_a_call_before(rows, width):
    import torch

    import helpers as H
    from host_offloaded_layer_b200 import _lib as L
    gen = torch.Generator().manual_seed(width)
    x = torch.randn(rows, width, generator=gen).bfloat16().cuda()
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    n = L.mt_layernorm_bwd_workspace_bytes(rows, width)
    dx, shared = torch.empty_like(x), H.workspace(n)
    dys = [(torch.randn(rows, width, generator=gen) * 2.0 ** i).bfloat16().cuda() for i in range(6)]

    def go(dy, ws):
        dg, db = H.empty_f32(width), H.empty_f32(width)
        L.mt_layernorm_bwd(dy, width, x, width, None, mean, rstd, None, 0, dx, width, dg, db, rows, width, ws, n)
        return dg, db

    want = [go(dy, H.workspace(n)) for dy in dys]
    torch.cuda.synchronize()
    got = [go(dy, shared) for dy in dys]  # one behind the other in the stream
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for w, g in zip(want, got) for a, b in zip(w, g))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(50, 3000), (300, 700), (1300, 1200), (1200, 2600)])
def test_muon_takes_nothing_from_the_workspace_of_a_call_before(rows, cols):
    import torch

    import helpers as H
    from host_offloaded_layer_b200 import _lib as L
    gen = torch.Generator().manual_seed(rows)
    n, cfg, shared = L.mt_muon_workspace_bytes(rows, cols), L.make_muon_cfg(), H.workspace(L.mt_muon_workspace_bytes(rows, cols))
    gs = [(torch.randn(rows, cols, generator=gen) * 10.0 ** i).cuda() for i in range(4)]

    def go(g, ws):
        o = H.empty_bf16(rows, cols)
        L.mt_muon_update(g, cols, None, None, 0, o, cols, rows, cols, cfg, ws, n)
        return o

    want = [go(g, H.workspace(n)) for g in gs]
    torch.cuda.synchronize()
    got = [go(g, shared) for g in gs]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert L.mt_device_error(clear=True) == 0
