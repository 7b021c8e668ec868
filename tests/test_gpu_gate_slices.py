"""moe_gate on logits that are columns of a wider matrix, from any column on."""
import ctypes

import numpy as np
import pytest
import torch

import expert_ffn_router_b200 as M
from gate_reference import gate, gate_weight_rtol

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k,G", [(8, 2, 1), (60, 6, 4), (256, 8, 8), (512, 32, 1), (1023, 5, 1)])
def test_logits_from_any_column_on(dtype, E, k, G):
    g = torch.Generator().manual_seed(E)
    for wide in (E + 8, E + 11):
        x = torch.randn(19, wide, generator=g).to(dtype).cuda()
        bias = (0.02 * torch.rand(E, generator=g)).cuda()
        c = M.config(128, 64, E, k, routed_scale=1.0)
        for at in range(9):
            lg = x[:, at:at + E]
            idx = torch.full((19, k), -9, dtype=torch.int32, device="cuda")
            w = torch.full((19, k), -9.0, device="cuda")
            M.moe_gate(c, M.gate_rule("softmax", G, max(1, G // 2)), lg, bias, idx, w)
            r_idx, r_w = gate(lg, bias, k, score="softmax", groups=G, keep=max(1, G // 2), scale=1.0)
            np.testing.assert_array_equal(idx.cpu().numpy(), r_idx)
            widest = float(lg.double().max() - lg.double().min())
            np.testing.assert_allclose(w.cpu().numpy().astype(np.float64), r_w, rtol=gate_weight_rtol(E, k, widest))


def test_logits_off_their_own_size_are_refused():
    raw = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    c, r = M.config(128, 64, 8, 2), M.gate_rule()
    idx = torch.empty(3, 2, dtype=torch.int32, device="cuda")
    w = torch.empty(3, 2, device="cuda")
    at = raw.data_ptr()
    for dtype, off, want in ((0, 2, M.MOE_EALIGN), (0, 1, M.MOE_EALIGN), (0, 4, M.MOE_OK), (1, 1, M.MOE_EALIGN),
                             (1, 2, M.MOE_OK), (0, 12, M.MOE_OK)):
        st = M.lib.moe_gate(ctypes.byref(c), ctypes.byref(r), at + off, dtype, 8, 3, None, idx.data_ptr(), w.data_ptr(),
                            torch.cuda.current_stream().cuda_stream)
        assert st == want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_beyond_32_bits(dtype):
    """The last row starts 2^32 elements behind the first."""
    E, k, ld = 64, 6, 1 << 31
    wide = torch.empty(2 * ld + E, dtype=dtype, device="cuda")
    lg = torch.as_strided(wide, (3, E), (ld, 1))
    lg.copy_(torch.randn(3, E, generator=torch.Generator().manual_seed(3)).to(dtype))
    idx = torch.empty(3, k, dtype=torch.int32, device="cuda")
    w = torch.empty(3, k, device="cuda")
    M.moe_gate(M.config(128, 64, E, k), M.gate_rule("sigmoid", 8, 4), lg, None, idx, w)
    r_idx, _ = gate(lg, None, k, groups=8, keep=4)
    np.testing.assert_array_equal(idx.cpu().numpy(), r_idx)


def test_many_rows():
    """More outputs than 2^31 bytes, more rows than any grid."""
    T, E, k = (1 << 24) + 5, 40, 32
    lg = torch.randint(-20, 20, (T, E), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    lg[:, ::5] = -float("inf")
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    M.moe_gate(M.config(128, 64, E, k, routed_scale=1.0), M.gate_rule("softmax"), lg, None, idx[:T], w[:T])
    key = lg.to(torch.int32).masked_fill(lg == -float("inf"), -100) * 64 + (63 - torch.arange(E, device="cuda")).int()
    want = torch.sort(key, dim=1, descending=True)[1][:, :k].to(torch.int32)
    assert torch.equal(idx[:T], want)  # 32 of 40 can be selected
    assert (w[:T].sum(1) - 1).abs().max() < 40 * 2.0 ** -24
    assert (idx[T] == -7).all() and (w[T] == -7.0).all()
