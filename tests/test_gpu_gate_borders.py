"""moe_gate where the border between the selected and the others is as narrow
as the types allow: the order is the double-precision one."""
import pytest
import torch

import expert_ffn_router_b200 as M

pytestmark = pytest.mark.gpu


def select(lg, bias, k, scale=1.0, **kw):
    T, E = lg.shape
    c = M.config(128, 64, E, k, routed_scale=scale)
    idx = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -9.0, device="cuda")
    M.moe_gate(c, M.gate_rule(**kw), lg, bias, idx, w)
    torch.cuda.synchronize()
    return idx, w


def values(lg, bias, score):
    p = torch.softmax(lg, 1) if score == "softmax" else torch.sigmoid(lg)
    return p + bias


def border_rows(T, E, k, score, bias, seed):
    """float32 logits whose k-th and (k + 1)-th selection values differ by what
    rounding one logit to float32 leaves."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    lg = (1.5 * torch.randn(T, E, generator=g, device="cuda")).double()
    order = values(lg, bias, score).sort(1, descending=True)[1]
    a, c = order[:, k - 1:k], order[:, k:k + 1]
    swap = torch.rand(T, 1, generator=g, device="cuda") < 0.5
    a, c = torch.where(swap, c, a), torch.where(swap, a, c)
    for _ in range(30):  # the logit that gives c the value of a (the softmax's sum moves with it)
        want = values(lg, bias, score).gather(1, a) - bias[c]
        if score == "softmax":
            top = lg.amax(1, keepdim=True)
            new = top + torch.log(want * torch.exp(lg - top).sum(1, keepdim=True))
        else:
            new = torch.log(want / (1 - want))
        lg = lg.scatter(1, c, torch.where(torch.isfinite(new), new, lg.gather(1, c)))
    lg = lg.float()
    v = values(lg.double(), bias, score)
    near = (v.gather(1, a) - v.gather(1, c)).abs() < 2.0 ** -24
    return lg, v, float(near.double().mean())


@pytest.mark.parametrize("E,k", [(32, 4), (64, 6), (256, 8), (512, 32), (1024, 8)])
@pytest.mark.parametrize("score,renorm", [("softmax", True), ("softmax", False), ("sigmoid", True)])
def test_borders_within_a_float32_rounding(E, k, score, renorm):
    """Scores stand within 2^-23 of each other (their own rounding is 2^-25 to
    2^-30), the logits and biases do not tie: the set and its order are
    decided in double."""
    T = 30000
    g = torch.Generator(device="cuda").manual_seed(E)
    bias = (0.02 if score == "sigmoid" else 0.2 / E) * torch.rand(E, generator=g, device="cuda")
    lg, v, near = border_rows(T, E, k, score, bias.double(), E + k)
    assert near > 0.9
    idx, _ = select(lg, bias, k, score=score, renorm=renorm)
    want = torch.sort(v, dim=1, descending=True, stable=True)[1][:, :k].to(torch.int32)
    wrong = (idx != want).any(1)
    assert not wrong.any(), f"{int(wrong.sum())} of {T} rows"
