"""Outputs that share memory with an input, with the workspace or with one
another are refused by the delta rule's and the norms' entry points, on the CPU.

Every call gets fake pointers (never dereferenced) and is refused: where an
alias is allowed, the refusal must name the next one.
"""
import ctypes

import pytest

from test_regression_amd import mesa
from tests.test_abi_delta import ENTRIES, FAKE, INVALID, OTHER

OUTS = {
    "mesa_delta_forward": "out final_state workspace",
    "mesa_delta_backward": "grad_q grad_k grad_v grad_gamma grad_beta grad_state workspace",
    "mesa_delta_step": "out state",
    "mesa_gate_norm": "y",
    "mesa_gate_norm_backward": "grad_x grad_gate grad_w workspace",
    "mesa_residual_norm": "h_out n",
    "mesa_residual_norm_backward": "grad_h grad_y grad_w grad_scale workspace",
}
ALLOWED = {("mesa_delta_forward", "final_state", "state0"), ("mesa_delta_backward", "grad_state", "grad_final"),
           ("mesa_residual_norm", "h_out", "h")}


def apart(name):
    """The entry's arguments with every tensor in 64 MiB of its own."""
    a = dict(ENTRIES[name])
    for i, n in enumerate(n for n, v in ENTRIES[name].items() if v in (FAKE, OTHER, FAKE + 4096)):
        a[n] = (i + 1) << 26
    return a


def message(name, a):
    L = mesa.lib()
    st = getattr(L, name)(*(ctypes.c_float(v) if n == "eps" else v for n, v in a.items()))
    assert st == INVALID, (name, a)
    return L.mesa_last_error_message().decode()


PAIRS = [(n, o, t) for n, outs in OUTS.items() for o in outs.split()
         for t in ENTRIES[n] if t != o and ENTRIES[n][t] in (FAKE, OTHER, FAKE + 4096)]


@pytest.mark.parametrize("name,out,other", PAIRS)
@pytest.mark.parametrize("by", [0, 16, -16])
def test_shared_memory_is_refused(name, out, other, by):
    if (name, out, other) in ALLOWED or (name, other, out) in ALLOWED:
        if by == 0:
            pytest.skip("allowed")
    a = apart(name)
    a[out] = a[other] + by
    msg = message(name, a)
    assert "alias" in msg and out in msg and other in msg, msg


@pytest.mark.parametrize("name,out,over", sorted(ALLOWED))
def test_allowed_aliases(name, out, over):
    a = apart(name)
    a[out] = a[over]
    last = OUTS[name].split()[-1]
    some = "y" if name == "mesa_residual_norm" else "q"
    a[last] = a[some]
    assert message(name, a) == f"{last} must not alias {some}"


def test_neighbours_are_not_aliases():
    """A tensor that begins where another ends."""
    for name, first, size, then in (("mesa_delta_forward", "q", 2 * 100 * 64 * 4, "out"),
                                    ("mesa_delta_backward", "gamma", 4 * 100 * 4, "grad_gamma"),
                                    ("mesa_residual_norm", "h", 5 * 100 * 4, "h_out")):
        a = apart(name)
        a[then] = a[first] + size
        last, some = OUTS[name].split()[-1], "y" if name == "mesa_residual_norm" else "k"
        a[last] = a[some]
        assert message(name, a) == f"{last} must not alias {some}"
        a[then] -= 16
        assert message(name, a) == f"{then} must not alias {first}"
