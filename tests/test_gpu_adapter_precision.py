"""moe_adapter keeps all the bits it says it keeps, in both of its kernels.

Two kinds of check beside the worst-case bound of the other tests:
values that 24 bits hold exactly, whose differences are a few units of the
last one (a product on fewer bits gives another number), and the relative L2
error, against what float32 sums of that depth can be off by."""
import pytest
import torch

import expert_ffn_router_b200 as M
from gate_reference import adapter

pytestmark = pytest.mark.gpu

# rows and rank of a call that k_adapter_few takes, of one that k_adapter takes
FEW = [(1, 16), (9, 64), (70, 32), (130, 128)]
MANY = [(2048, 64), (2300, 128)]


def run(x, a, b, sx=None):
    T = x.shape[0]
    ad = M.make_adapters(a, b)
    of = torch.zeros(T, dtype=torch.int32, device="cuda")
    y = torch.empty(T, b.shape[1], device="cuda")
    M.moe_adapter(ad, M.adapter_plan(1, of), x, y, sx=sx)
    return y


@pytest.mark.parametrize("T,r", FEW + MANY)
def test_first_product_keeps_24_bits_of_float32_rows(T, r):
    """A x = x_i - x_j, integers of 24 bits that differ by less than 256: every
    product and sum is exact if the parts hold all bits, so the result is."""
    g = torch.Generator(device="cuda").manual_seed(T + r)
    d_in, d_out = 1040, 2 * r
    x = torch.randint(1 << 23, 1 << 24, (T, d_in), generator=g, device="cuda")
    at = torch.randperm(d_in, generator=g, device="cuda")[:2 * r].view(2, r)
    x[:, at[1]] = x[:, at[0]] - torch.randint(-255, 256, (T, r), generator=g, device="cuda")
    x = x.clamp(1 << 23, (1 << 24) - 1)
    a = torch.zeros(1, r, d_in, device="cuda")
    a[0, torch.arange(r, device="cuda"), at[0]] = 1
    a[0, torch.arange(r, device="cuda"), at[1]] = -1
    b = torch.cat([torch.eye(r, device="cuda"), -2 * torch.eye(r, device="cuda").flip(0)])[None]
    y = run(x.float(), a.bfloat16(), b.bfloat16().contiguous())
    h = x[:, at[0]] - x[:, at[1]]
    assert torch.equal(y.double(), torch.cat([h, -2 * h.flip(1)], 1).double())
    assert int(h.abs().max()) > 100


@pytest.mark.parametrize("T,r", FEW + MANY)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "i8"])
def test_second_product_keeps_24_bits_of_the_first(T, r, dtype):
    """Components of A x that are integers of 22 to 24 bits, in pairs whose
    difference B takes: exact, as above."""
    g = torch.Generator(device="cuda").manual_seed(T + r + 7)
    d_in, d_out, p = 1040, r // 2, r // 2
    at = torch.randperm(d_in, generator=g, device="cuda")[:3 * r].view(3, r)  # three columns a component
    bits = 7 if dtype == "i8" else 8
    lo = torch.randint(0, 1 << bits, (3, T, p), generator=g, device="cuda")
    lo[0] |= 1 << (bits - 1)
    twin = lo.clone()
    twin[2] = torch.randint(0, 1 << bits, (T, p), generator=g, device="cuda")  # the last 7 or 8 bits differ
    digits = torch.cat([lo, -twin], 2)  # [3][T][r]: component c < p, and minus its twin
    a = torch.zeros(1, r, d_in, device="cuda")
    c = torch.arange(r, device="cuda")
    x = torch.randint(-100, 100, (T, d_in), generator=g, device="cuda")
    if dtype == "f32":  # one column holds all of it
        x[:, at[0]] = (digits[0] << 16) + (digits[1] << 8) + digits[2]
        a[0, c, at[0]] = 1
    else:
        for i in range(3):
            x[:, at[i]] = digits[i]
            a[0, c, at[i]] = float(1 << (bits * (2 - i)))
    b = torch.cat([torch.eye(p, device="cuda"), torch.eye(p, device="cuda")], 1)[None]
    if d_out % 16:  # (sizes are multiples of 16)
        b = torch.cat([b, torch.zeros(1, 16 - d_out % 16, r, device="cuda")], 1)
    kind = {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8}[dtype]
    sx = torch.ones(T, device="cuda") if dtype == "i8" else None
    y = run(x.to(kind), a.bfloat16(), b.bfloat16().contiguous(), sx)[:, :p]
    want = lo[2] - twin[2]
    assert torch.equal(y.double(), want.double())
    assert int(want.abs().max()) > 50 or T * p < 100


def cut(v, bits):
    """v (float32) with the last of its 24 bits cut off."""
    i = v.contiguous().view(torch.int32)
    return (i & ~((1 << (24 - bits)) - 1)).view(torch.float32)


@pytest.mark.parametrize("T,r,d", [(64, 16, 6144), (200, 64, 2048), (2100, 64, 6144), (2100, 128, 6144)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "i8"])
def test_relative_error_is_that_of_float32_sums(T, r, d, dtype):
    """Adders that truncate are off by up to 2^-23 of the sum so far, by 0.75 *
    2^-24 on the mean, all towards 0; a sum of random terms grows with the root
    of their number, so n additions in a row are off by at most 2 / 3 n of
    those, relative to the result (all errors taken to add up).  n is at most 48
    in the first product (then it is read out), 3 r / 16 in the second; some 20
    rounded additions join the parts of the first (counted as 8 of those).
    Without the reading out, or with the last 8 bits of x or A x cut off (0.72 *
    2^-16 on the mean, all towards 0), the result is off by more."""
    g = torch.Generator(device="cuda").manual_seed(T + r)
    x = torch.randn(T, d, generator=g, device="cuda")
    sx = None
    if dtype == "i8":
        sx = x.abs().amax(1) / 127
        x = torch.clamp(torch.round(x / sx[:, None]), -127, 127).to(torch.int8)
    elif dtype == "bf16":
        x = x.bfloat16()
    a = (torch.randn(1, r, d, generator=g, device="cuda") / d ** 0.5).bfloat16()
    b = torch.randn(1, 512, r, generator=g, device="cuda").bfloat16()
    y = run(x, a, b, sx).double()
    of = torch.zeros(T, dtype=torch.int32, device="cuda")
    ref, _ = adapter(x, sx, of, a, b, [r], None, None)
    off = float((y - ref).norm() / ref.norm())
    limit = (2 / 3 * 48 + 2 / 3 * 3 * r / 16 + 8) * 0.75 * 2.0 ** -24
    assert off < limit, f"{off:.2e} of {limit:.2e}"
    # the limit tells 24 bits from 16, of x and of A x
    h = (x.double() * (1 if sx is None else sx.double()[:, None])) @ a[0].double().T
    worse = cut(h.float(), 16).double() @ b[0].double().T
    assert float((worse - ref).norm() / ref.norm()) > limit
    if dtype == "f32":
        worse = (cut(x, 16).double() @ a[0].double().T) @ b[0].double().T
        assert float((worse - ref).norm() / ref.norm()) > limit
