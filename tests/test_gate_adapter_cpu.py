"""moe_gate, moe_route_gated, moe_layer_routed and the adapter calls without a
GPU: their arguments are refused on the host before anything is launched."""
import ctypes

import pytest
import torch

import expert_ffn_router_b200 as M

L = M.lib
FAKE = 1 << 20  # 16-byte aligned, never dereferenced
B = ctypes.byref


def cfg(**kw):
    c = M.config(128, 64, 24, 5, 1, 4, 2.5)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def gate(c=None, r=None, logits=FAKE, dtype=0, ld=24, T=4, bias=FAKE, idx=FAKE, w=FAKE):
    return L.moe_gate(B(c if c is not None else cfg()), B(r if r is not None else M.gate_rule()), logits, dtype, ld, T,
                      bias, idx, w, None)


@pytest.mark.parametrize("field,value", [
    ("score", 2), ("score", -1), ("n_groups", -1), ("n_groups", 33), ("n_groups", 5), ("raw_weights", 2)])
def test_gate_refuses_a_bad_rule(field, value):
    r = M.gate_rule()
    setattr(r, field, value)
    assert gate(r=r) == M.MOE_EINVAL
    assert L.moe_last_error()


@pytest.mark.parametrize("groups,keep,value", [(3, 0, 0), (3, 4, 0), (3, 1, 2), (8, 1, 0)])
def test_gate_refuses_bad_groups(groups, keep, value):
    """(8, 1): three experts of one group cannot fill five slots."""
    r = M.MoeGateRule(0, groups, keep, value, 0)
    assert gate(r=r) == M.MOE_EINVAL


def test_gate_does_not_read_the_group_fields_without_groups():
    for n in (0, 1):
        assert gate(r=M.MoeGateRule(0, n, -7, 99, 0), T=0) == M.MOE_OK


def test_gate_refuses_bad_arguments():
    assert L.moe_gate(B(cfg()), None, FAKE, 0, 24, 4, FAKE, FAKE, FAKE, None) == M.MOE_EINVAL
    assert L.moe_gate(None, B(M.gate_rule()), FAKE, 0, 24, 4, FAKE, FAKE, FAKE, None) == M.MOE_EINVAL
    assert gate(dtype=2) == M.MOE_EINVAL  # codes are adapters' inputs only
    assert gate(T=-1) == M.MOE_EINVAL
    assert gate(ld=23) == M.MOE_EINVAL
    assert gate(logits=None) == M.MOE_EINVAL
    assert gate(idx=None) == M.MOE_EINVAL
    assert gate(w=None) == M.MOE_EINVAL
    assert gate(logits=FAKE + 2) == M.MOE_EALIGN
    assert gate(bias=FAKE + 4) == M.MOE_EALIGN
    assert gate(c=cfg(top_k=25)) == M.MOE_EINVAL
    assert gate(T=0) == M.MOE_OK


def test_gate_rule_names():
    r = M.gate_rule("softmax", 8, 4, "max", renorm=False)
    assert (r.score, r.n_groups, r.topk_groups, r.group_value, r.raw_weights) == (1, 8, 4, 1, 1)
    with pytest.raises(KeyError):
        M.gate_rule("relu")


def test_route_gated_refuses_bad_arguments():
    def call(c=None, r=None, x=FAKE, dtype=0, T=4, wr=FAKE, bias=FAKE, ws=FAKE, wsb=1 << 40):
        return L.moe_route_gated(B(c or cfg()), B(r or M.gate_rule()), x, dtype, T, wr, bias, FAKE, FAKE, ws, wsb, None)

    assert call(r=M.gate_rule("sigmoid", 5, 1)) == M.MOE_EINVAL
    assert call(dtype=2) == M.MOE_EINVAL
    assert call(x=None) == M.MOE_EINVAL
    assert call(wr=FAKE + 8) == M.MOE_EALIGN
    assert call(wsb=100) == M.MOE_ENOSPACE
    assert call(T=-1) == M.MOE_EINVAL
    assert call(T=0) == M.MOE_OK


def test_layer_routed_refuses_bad_arguments():
    pool = M.MoePool(FAKE, FAKE)

    def call(c=None, pl=pool, idx=FAKE, w=FAKE, x=FAKE, dtype=0, T=4, out=FAKE, ws=FAKE, wsb=1 << 40):
        return L.moe_layer_routed(B(c or cfg()), B(pl) if pl is not None else None, idx, w, x, dtype, T, out, 0, ws, wsb,
                                  None)

    assert call(pl=None) == M.MOE_EINVAL
    assert call(pl=M.MoePool(None, FAKE)) == M.MOE_EINVAL
    assert call(pl=M.MoePool(FAKE, FAKE, FAKE, 0)) == M.MOE_EINVAL
    assert call(idx=None) == M.MOE_EINVAL
    assert call(w=FAKE + 4) == M.MOE_EALIGN
    assert call(out=None) == M.MOE_EINVAL
    assert call(dtype=2) == M.MOE_EINVAL
    assert call(wsb=1000) == M.MOE_ENOSPACE
    assert call(T=0) == M.MOE_OK


def test_plan_refuses_bad_arguments():
    assert L.moe_adapter_plan_bytes(0, 4) == 0
    assert L.moe_adapter_plan_bytes(1025, 4) == 0
    assert L.moe_adapter_plan_bytes(4, -1) == 0
    n = M.moe_adapter_plan_bytes(4, 100)
    assert n >= 64 + 100 * 4 + 5 * 16
    assert M.moe_adapter_plan_bytes(1024, 1 << 20) > (1 << 22)

    def call(n_ad=4, of=FAKE, T=100, plan=FAKE, nb=n):
        return L.moe_adapter_plan(n_ad, of, T, plan, nb, None)

    assert call(n_ad=0) == M.MOE_EINVAL
    assert call(of=None) == M.MOE_EINVAL
    assert call(T=-1) == M.MOE_EINVAL
    assert call(plan=None) == M.MOE_EINVAL
    assert call(plan=FAKE + 8) == M.MOE_EALIGN
    assert call(nb=n - 1) == M.MOE_ENOSPACE
    with pytest.raises(M.MoeError):
        M.moe_adapter_plan_bytes(0, 1)


MB = 1 << 20


def adapters(**kw):
    f = dict(n_adapters=4, r_max=16, d_in=128, d_out=64, a=10 * MB, b=11 * MB, rank=12 * MB, scale=13 * MB)
    f.update(kw)
    return M.MoeAdapters(*[f[n] for n, _ in M.MoeAdapters._fields_])


def adapt(ad=None, plan=20 * MB, nb=1 << 20, x=30 * MB, dtype=0, sx=None, ldx=128, T=8, base=40 * MB, ldb=64,
          y=50 * MB, ldy=64):
    return L.moe_adapter(B(ad if ad is not None else adapters()), plan, nb, x, dtype, sx, ldx, T, base, ldb, y, ldy, None)


@pytest.mark.parametrize("field,value,status", [
    ("n_adapters", 0, -1), ("n_adapters", 1025, -1), ("r_max", 4, -1), ("r_max", 20, -1), ("r_max", 136, -1),
    ("d_in", 120, -1), ("d_in", 0, -1), ("d_out", 8, -1), ("d_out", 40000, -1), ("a", None, -1), ("b", None, -1),
    ("a", 10 * MB + 8, -2), ("rank", 12 * MB + 4, -2)])
def test_adapter_refuses_a_bad_set(field, value, status):
    assert adapt(adapters(**{field: value})) == status


def test_adapter_refuses_bad_arguments():
    assert L.moe_adapter(None, FAKE, MB, FAKE, 0, None, 128, 8, None, 0, FAKE, 64, None) == M.MOE_EINVAL
    assert adapt(dtype=3) == M.MOE_EINVAL
    assert adapt(dtype=2) == M.MOE_EINVAL  # codes without their scales
    assert adapt(sx=60 * MB) == M.MOE_EINVAL  # scales without codes
    assert adapt(ldx=112) == M.MOE_EINVAL
    assert adapt(ldx=130) == M.MOE_EINVAL  # rows off 16 bytes
    assert adapt(dtype=1, ldx=132) == M.MOE_EINVAL
    assert adapt(ldy=60) == M.MOE_EINVAL
    assert adapt(ldy=66) == M.MOE_EINVAL
    assert adapt(ldb=66) == M.MOE_EINVAL
    assert adapt(nb=64) == M.MOE_ENOSPACE
    assert adapt(plan=None) == M.MOE_EINVAL
    assert adapt(x=None) == M.MOE_EINVAL
    assert adapt(y=None) == M.MOE_EINVAL
    assert adapt(y=50 * MB + 4) == M.MOE_EALIGN
    assert adapt(T=-1) == M.MOE_EINVAL
    assert adapt(T=0) == M.MOE_OK


def test_adapter_refuses_an_output_over_an_input():
    row = 64 * 4
    assert adapt(base=50 * MB, y=50 * MB, ldb=64, ldy=128) == M.MOE_EINVAL  # in place, rows elsewhere
    assert adapt(base=50 * MB + row, y=50 * MB) == M.MOE_EINVAL
    assert adapt(base=50 * MB - 7 * row, y=50 * MB) == M.MOE_EINVAL
    assert adapt(x=50 * MB + 7 * row, y=50 * MB) == M.MOE_EINVAL
    assert adapt(y=10 * MB) == M.MOE_EINVAL
    assert adapt(y=11 * MB - row) == M.MOE_EINVAL
    assert adapt(y=12 * MB) == M.MOE_EINVAL
    assert adapt(y=13 * MB) == M.MOE_EINVAL
    assert adapt(y=20 * MB) == M.MOE_EINVAL
    assert adapt(dtype=2, sx=50 * MB, ldx=128, y=50 * MB) == M.MOE_EINVAL


def test_binding_refuses_bad_tensors():
    c, r = cfg(), M.gate_rule()
    with pytest.raises(ValueError):  # host logits
        M.moe_gate(c, r, torch.zeros(2, 24), None, torch.zeros(2, 5), torch.zeros(2, 5))
    with pytest.raises(ValueError):
        M.make_adapters(torch.zeros(2, 8, 16), torch.zeros(2, 16, 16))
    with pytest.raises(ValueError):
        M.make_adapters(torch.zeros(2, 8, 16, dtype=torch.bfloat16), torch.zeros(2, 16, 8, dtype=torch.bfloat16))
