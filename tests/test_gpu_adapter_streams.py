"""Plans made on one stream and read on another: their memory is neither
written while an earlier plan in it is read nor handed out while it is
written."""
import pytest
import torch

import expert_ffn_router_b200 as M

pytestmark = pytest.mark.gpu
T, N, D = 5000, 7, 64


def setup():
    g = torch.Generator(device="cuda").manual_seed(5)
    a = torch.randn(N, 16, D, generator=g, device="cuda").bfloat16()
    b = torch.randn(N, D, 16, generator=g, device="cuda").bfloat16()
    x = torch.randn(T, D, generator=g, device="cuda")
    of = [torch.randint(-1, N, (T,), generator=g, device="cuda").to(torch.int32) for _ in range(2)]
    return M.make_adapters(a, b), x, of


def test_plan_in_memory_that_is_still_read():
    ad, x, of = setup()
    want = torch.empty(T, D, device="cuda")
    M.moe_adapter(ad, M.adapter_plan(N, of[0]), x, want)
    y, z, ref = torch.empty_like(want), torch.empty_like(want), torch.empty_like(want)
    M.moe_adapter(ad, M.adapter_plan(N, of[1]), x, ref)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    plan = M.adapter_plan(N, of[0])
    at = plan.data_ptr()
    torch.cuda._sleep(50_000_000)  # (some 25 ms)
    M.moe_adapter(ad, plan, x, y)
    del plan
    plan = M.adapter_plan(N, of[1], stream=side)
    assert plan.data_ptr() == at  # the case in question
    M.moe_adapter(ad, plan, x, z, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(z, ref)


def test_plan_dropped_before_it_is_written():
    ad, x, of = setup()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    plan = M.adapter_plan(N, of[0], stream=side)
    n = plan.numel()
    del plan
    z = torch.zeros(n, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert (z == 0).all()
