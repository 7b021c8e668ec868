"""Calls of several host threads at once."""
import threading

import pytest
import torch

import expert_ffn_router_b200 as M

pytestmark = pytest.mark.gpu


def test_plans_and_selections_of_two_threads():
    """Plans whose kernel needs 54 and 136 KB of shared memory, selections of
    256 and 1024 experts: every call launches, and gives what it gives alone."""
    g = torch.Generator(device="cuda").manual_seed(1)
    T = 700
    of = {n: torch.randint(-1, n, (T,), generator=g, device="cuda").to(torch.int32) for n in (400, 1000)}
    lg = {E: torch.randn(T, E, generator=g, device="cuda") for E in (256, 1024)}
    cfg = {E: M.config(128, 64, E, 32) for E in lg}
    got, errors = {}, []

    def work(n, E, stream):
        try:
            with torch.cuda.stream(stream):
                for i in range(50):
                    plan = M.adapter_plan(n, of[n])
                    idx = torch.empty(T, 32, dtype=torch.int32, device="cuda")
                    w = torch.empty(T, 32, device="cuda")
                    M.moe_gate(cfg[E], M.gate_rule("softmax"), lg[E], None, idx, w)
                stream.synchronize()
                got[n] = (plan.clone(), idx, w)
                stream.synchronize()
        except Exception as e:  # noqa: BLE001 (the assertion below shows it)
            errors.append(e)

    torch.cuda.synchronize()
    ts = [threading.Thread(target=work, args=(n, E, torch.cuda.Stream())) for n, E in ((400, 256), (1000, 1024))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors
    for n, E in ((400, 256), (1000, 1024)):
        plan, idx, w = got[n]
        order = plan[64:64 + 4 * T].view(torch.int32)
        key = torch.where(of[n] < 0, n, of[n])
        assert torch.equal(order.long(), torch.sort(key, stable=True)[1])
        assert torch.equal(idx.long(), torch.sort(lg[E], dim=1, descending=True, stable=True)[1][:, :32])
        assert M.moe_poll_status(plan) == M.MOE_OK
