"""Sizes at which a workspace's layout ends are refused on the host."""
import ctypes

import expert_ffn_router_b200 as M

L = M.lib
FAKE = 1 << 20  # 16-byte aligned, never dereferenced
B = ctypes.byref
MOST = 1 << 20  # tokens a workspace is laid out for


def test_more_tokens_than_a_workspace_layout_holds():
    """The layout is carved for at most 2^20 tokens, however large the
    workspace: a call of more would write beyond its arrays."""
    c = M.config(128, 64, 8, 2)
    pool = M.MoePool(FAKE, FAKE)
    huge = 1 << 50
    T = MOST + 1
    assert M.moe_workspace_bytes(c, MOST) > 0
    assert L.moe_workspace_bytes(B(c), T) == 0 and L.moe_last_error()
    none = None
    calls = {
        "moe_route": lambda: L.moe_route(B(c), FAKE, 0, T, FAKE, FAKE, FAKE, FAKE, FAKE, huge, none),
        "moe_route_gated": lambda: L.moe_route_gated(B(c), B(M.gate_rule()), FAKE, 0, T, FAKE, none, FAKE, FAKE, FAKE,
                                                     huge, none),
        "moe_layer": lambda: L.moe_layer(B(c), B(pool), FAKE, FAKE, FAKE, 0, T, FAKE, 0, none, none, FAKE, huge, none),
        "moe_layer_routed": lambda: L.moe_layer_routed(B(c), B(pool), FAKE, FAKE, FAKE, 0, T, FAKE, 0, FAKE, huge, none),
        "moe_expert_ffn": lambda: L.moe_expert_ffn(B(c), B(pool), 0, FAKE, FAKE, T, FAKE, none, none, none, none, FAKE,
                                                   huge, none),
        "moe_expert_down": lambda: L.moe_expert_down(B(c), B(pool), 0, FAKE, FAKE, T, FAKE, none, FAKE, huge, none),
    }
    assert {n: f() for n, f in calls.items()} == {n: M.MOE_EINVAL for n in calls}
