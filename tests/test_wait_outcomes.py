"""What the kernels that wait for copies of their own do when a wait runs out, read from their source (a wait that
runs out is not provoked on a GPU): its outcome is used, and the copies in flight are waited for before the CTA leaves."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "host_offloaded_layer_b200", "csrc")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _bodies(code):
    """{name: body} of the __global__ functions."""
    out = {}
    for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\(", code):
        start = code.index("{", m.end())
        depth, i = 1, start + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(code[i], 0)
            i += 1
        out[m.group(1)] = code[start:i]
    return out


@pytest.mark.parametrize("name,kernels", [("layernorm.cu", 1), ("muon.cu", 3)])
def test_a_wait_that_runs_out_leaves_no_copies_in_flight(name, kernels):
    code = _code(name)
    bodies = {k: b for k, b in _bodies(code).items() if re.search(r"\b(bulk_copy|load_atom\w*|fused_product)\b", b)}
    assert len(bodies) == kernels, sorted(bodies)
    for kernel, body in bodies.items():
        if "give_up<" in body:  # a function of its own, which ends the thread
            body = code[code.index(" give_up("):code.index("exit;")]
        assert "drain_ring(" in body, kernel


@pytest.mark.parametrize("name", ["layernorm.cu", "muon.cu"])
def test_every_outcome_of_a_wait_is_used(name):
    code = _code(name)
    waits = list(re.finditer(r"\b(?:tc::)?(?:mbar_wait|warp_wait|wait_one)\(", code))
    assert waits
    for m in waits:
        before = code[:m.start()].rstrip()
        assert before.endswith(("!", "=", "return", "if (", "bool")), code[m.start() - 80:m.end() + 40]
