"""What moe_gate takes and refuses of its arguments, beyond the bad values:
without a GPU (nothing here is launched)."""
import ctypes

import pytest

import expert_ffn_router_b200 as M

L = M.lib
FAKE = 1 << 20  # 16-byte aligned, never dereferenced
B = ctypes.byref


def gate(c, T=0):
    return L.moe_gate(B(c), B(M.gate_rule()), FAKE, 0, 24, T, FAKE, FAKE, FAKE, None)


def test_a_configuration_of_the_selection_alone():
    """Of the configuration only n_experts, top_k, routed_scale and topp are
    used, so the others may be anything: a zero-initialised one will do."""
    c = M.MoeConfig(0, 0, 24, 5, 0, 0, 2.5, 0, 0.0)
    assert gate(c) == M.MOE_OK
    c.d, c.f, c.wbits, c.has_shared = 100000, -3, 7, 9
    assert gate(c) == M.MOE_OK


@pytest.mark.parametrize("field,value", [("n_experts", 0), ("n_experts", 1025), ("top_k", 0), ("top_k", 25),
                                         ("top_k", 33), ("routed_scale", float("nan")), ("topp", -0.1), ("topp", 1.1)])
def test_the_fields_it_uses_are_checked(field, value):
    c = M.MoeConfig(0, 0, 24, 5, 0, 0, 2.5, 0, 0.0)
    setattr(c, field, value)
    assert gate(c, T=4) == M.MOE_EINVAL
    assert L.moe_last_error()
