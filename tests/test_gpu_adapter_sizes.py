"""moe_adapter at the ends of its range: the smallest rows through the kernel of
many rows, tables and rows whose offsets pass 2^31 elements through both."""
import pytest
import torch

import expert_ffn_router_b200 as M
from gate_reference import adapter

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.int8])
@pytest.mark.parametrize("r_max,d_in,d_out", [(40, 16, 16), (64, 16, 2048), (128, 2048, 16), (48, 32, 48)])
def test_many_rows_of_the_smallest_widths(dtype, r_max, d_in, d_out):
    T, n = 2050, 2
    g = torch.Generator(device="cuda").manual_seed(d_in + d_out)
    a = torch.randn(n, r_max, d_in, generator=g, device="cuda").bfloat16()
    b = torch.randn(n, d_out, r_max, generator=g, device="cuda").bfloat16()
    rank = [r_max, r_max - 7]
    x, sx = torch.randn(T, d_in, generator=g, device="cuda"), None
    if dtype is torch.int8:
        sx = x.abs().amax(1) / 127
        x = torch.clamp(torch.round(x / sx[:, None]), -127, 127)
    x = x.to(dtype)
    of = torch.randint(-1, n, (T,), generator=g, device="cuda").to(torch.int32)
    ad = M.make_adapters(a, b, torch.tensor(rank, dtype=torch.int32, device="cuda"))
    for owners in (of, of.sort()[0]):
        wide = torch.full((T + 1, d_out), 7.0, device="cuda")
        plan = M.adapter_plan(n, owners)
        M.moe_adapter(ad, plan, x, wide[:T], sx=sx)
        assert M.moe_poll_status(plan) == M.MOE_OK
        ref, err = adapter(x, sx, owners, a, b, rank, None, None)
        assert bool(((wide[:T].double() - ref).abs() <= err + 1e-30).all())
        assert (wide[T] == 7.0).all()


# 520 adapters of 128 x 32768: the last one starts at 2.18e9 elements.  133120
# rows are the least that go to the kernel of many rows with 520 adapters; of
# 32768 elements each, the last row starts at 4.36e9.
N, R, W = 520, 128, 32768
ROWS = [3, 256 * N]


def owners(T):
    of = torch.full((T,), -1, dtype=torch.int32)
    of[0] = of[T - 1] = N - 1
    of[T // 2 - 100:T // 2 + 1] = N - 1
    return of.cuda()


@pytest.mark.parametrize("T", ROWS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.int8])
def test_a_and_x_beyond_32_bits(T, dtype):
    a = torch.zeros(N, R, W, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(N, 16, R, dtype=torch.bfloat16, device="cuda")
    a[-1], b[-1] = 0.25, 2.0  # (all sums are exact)
    of = owners(T)
    x = torch.ones(T, W, dtype=dtype, device="cuda")
    x[:, 7] = 3
    x[T - 1, W - 1] = 5
    sx = torch.ones(T, device="cuda") if dtype is torch.int8 else None
    y = torch.full((T, 16), 9.0, device="cuda")
    plan = M.adapter_plan(N, of)
    M.moe_adapter(M.make_adapters(a, b), plan, x, y, sx=sx)
    assert M.moe_poll_status(plan) == M.MOE_OK
    want = torch.where(of >= 0, 0.25 * 2 * R * (W + 2.0), 0.0)
    want[T - 1] += 0.25 * 2 * R * 4
    assert torch.equal(y, want[:, None].expand(T, 16))


@pytest.mark.parametrize("T", ROWS)
@pytest.mark.parametrize("in_place", [False, True])
def test_b_base_and_y_beyond_32_bits(T, in_place):
    a = torch.zeros(N, R, 16, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(N, W, R, dtype=torch.bfloat16, device="cuda")
    a[-1] = 1.0
    b[-1] = 2.0
    b[-1, W - 1] = 4.0
    of = owners(T)
    x = torch.ones(T, 16, dtype=torch.bfloat16, device="cuda")
    base = torch.empty(T, W, device="cuda")
    base[:] = torch.arange(T, device="cuda").float()[:, None]
    y = base if in_place else torch.empty(T, W, device="cuda")
    plan = M.adapter_plan(N, of)
    M.moe_adapter(M.make_adapters(a, b), plan, x, y, base=base)
    assert M.moe_poll_status(plan) == M.MOE_OK
    step = torch.where(of >= 0, 2.0 * R * 16, 0.0)
    want = torch.arange(T, device="cuda").float() + step
    assert torch.equal(y[:, :W - 1], want[:, None].expand(T, W - 1))
    assert torch.equal(y[:, W - 1], want + step)
