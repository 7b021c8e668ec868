"""moe_gate where the border between the selected and the others is as narrow
as the types allow, or where sums leave float32's range: the order is the
double-precision one."""
import numpy as np
import pytest
import torch

import expert_ffn_router_b200 as M
from gate_reference import gate

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


LOW = torch.finfo(torch.float32).min


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("value", ["top2", "max"])
@pytest.mark.parametrize("E,G,keep,k", [(24, 3, 2, 5), (64, 8, 3, 8), (256, 8, 4, 8), (1024, 32, 3, 32)])
def test_groups_whose_sums_leave_float32(score, value, E, G, keep, k):
    """Biases of the type's lowest value (a mask, to some callers) are values
    like others: the sum of two of them is not -inf."""
    g = torch.Generator().manual_seed(E)
    lg = torch.randn(9, E, generator=g).cuda()
    lg[3, ::2] = -float("inf")
    lg[4] = -float("inf")
    gs = E // G
    for fill in (LOW, LOW / 1.5, -1.0e38, 2.5e38, torch.finfo(torch.float32).max):
        b = torch.full((E,), fill)
        spread = b.clone()
        spread[gs:2 * gs] *= 0.75
        some = b.clone()
        some[[0, gs, E - 1]] = 0.25
        one = b.clone()
        one[gs:2 * gs] = 0.0
        for bias in (b, spread, some, one):
            bias = bias.cuda()
            idx, w = select(lg, bias, k, score=score, n_groups=G, topk_groups=keep, group_value=value)
            r_idx, r_w = gate(lg, bias, k, score=score, groups=G, keep=keep, value=value, scale=1.0)
            np.testing.assert_array_equal(idx.cpu().numpy(), r_idx)
            # roundings of float32 weights: twice an exponential (4, and the argument, up to 8 wide), a sum over 1024
            # experts (37 deep) and one over 32, the quotient and the scale
            np.testing.assert_allclose(w.cpu().numpy().astype(np.float64), r_w, rtol=(2 * (8 + 4) + 37 + 32 + 3) * 2.0 ** -24)


@pytest.mark.parametrize("renorm", [True, False])
def test_slots_without_an_expert_weigh_nothing_whatever_the_scale(renorm):
    """An infinite routed_scale too; rows of both forms (the second one's
    infinite logit sends it through the double-precision one)."""
    lg = torch.full((3, 64), -float("inf"), device="cuda")
    lg[0, 3] = 1.0
    lg[1, 3], lg[1, 9] = float("inf"), 2.0
    idx, w = select(lg, None, 6, scale=float("inf"), score="sigmoid", renorm=renorm)
    assert idx.tolist() == [[3] + [-1] * 5, [3, 9] + [-1] * 4, [-1] * 6]
    assert (w[idx < 0] == 0).all() and (w[idx >= 0] == float("inf")).all()
