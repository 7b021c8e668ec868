"""moe_gate against its rule in 64 bits: indices equal, weights within the
roundings of float32 (gate_reference.gate_weight_rtol)."""
import numpy as np
import pytest
import torch

import expert_ffn_router_b200 as M
import oracle as O
import workloads as W
from gate_reference import gate, gate_weight_rtol

pytestmark = pytest.mark.gpu


def select(lg, bias, k, score="sigmoid", groups=0, keep=0, value="top2", renorm=True, scale=2.5, topp=0.0):
    T, E = lg.shape
    c = M.config(128, 64, E, k, routed_scale=scale, topp=topp)
    idx = torch.full((T, k), -9, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -9.0, device="cuda")
    M.moe_gate(c, M.gate_rule(score, groups, keep, value, renorm), lg, bias, idx, w)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy().astype(np.float64)


def check(lg, bias, k, **kw):
    idx, w = select(lg, bias, k, **kw)
    r_idx, r_w = gate(lg, bias, k, **kw)
    np.testing.assert_array_equal(idx, r_idx)
    l64 = lg.double()
    fin = l64[torch.isfinite(l64)]
    widest = float(fin.max() - fin.min()) if fin.numel() else 0.0
    np.testing.assert_allclose(w, r_w, rtol=gate_weight_rtol(lg.shape[1], k, widest), atol=1e-37)
    return idx, w


def logits(T, E, seed, dtype=torch.float32, sigma=1.5, ld=None):
    g = torch.Generator().manual_seed(seed)
    x = sigma * torch.randn(T, ld or E, generator=g)
    return x.to(dtype).cuda()[:, :E]


def bias_of(E, seed, width=0.02):
    g = torch.Generator().manual_seed(seed + 77)
    return (width * (torch.rand(E, generator=g) - 0.5)).cuda()


SHAPES = [(1, 1, 1), (1, 8, 2), (5, 8, 8), (33, 24, 5), (3, 31, 31), (7, 32, 32), (2, 33, 4), (9, 60, 6), (70, 64, 8),
          (4, 96, 7), (3, 160, 32), (1, 256, 8), (129, 256, 8), (5, 257, 9), (6, 384, 6), (3, 512, 32), (2, 1023, 17),
          (11, 1024, 32), (2500, 256, 8)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [True, False])
def test_shapes(T, E, k, score, with_bias):
    for dtype in (torch.float32, torch.bfloat16):
        check(logits(T, E, T + E, dtype), bias_of(E, k) if with_bias else None, k, score=score)


GROUPS = [(24, 3, 2, 5), (24, 24, 7, 5), (24, 2, 2, 12), (60, 4, 1, 6), (64, 8, 4, 8), (96, 32, 5, 15), (96, 3, 3, 32),
          (160, 8, 3, 6), (256, 8, 4, 8), (256, 32, 1, 8), (256, 16, 16, 32), (384, 2, 1, 9), (512, 8, 4, 32),
          (1024, 32, 6, 32), (1020, 30, 11, 8), (32, 8, 4, 8), (16, 4, 2, 6)]


@pytest.mark.parametrize("E,G,keep,k", GROUPS)
@pytest.mark.parametrize("value", ["top2", "max"])
def test_groups(E, G, keep, k, value):
    for T, score, dtype, b in ((3, "sigmoid", torch.float32, True), (41, "softmax", torch.float32, True),
                               (40, "sigmoid", torch.bfloat16, False), (1, "softmax", torch.bfloat16, False),
                               (300, "sigmoid", torch.bfloat16, True)):
        check(logits(T, E, E + G, dtype), bias_of(E, G) if b else None, k, score=score, groups=G, keep=keep,
              value=value)


@pytest.mark.parametrize("E,k", [(8, 2), (24, 5), (256, 8), (512, 32)])
@pytest.mark.parametrize("ld", [0, 1, 3, 4, 8])
def test_rows_of_a_wider_matrix(E, k, ld):
    for dtype in (torch.float32, torch.bfloat16):
        check(logits(37, E, ld, dtype, ld=E + ld), bias_of(E, 1), k)


@pytest.mark.parametrize("topp", [0.1, 0.5, 0.7, 0.95, 1.0])
@pytest.mark.parametrize("renorm", [True, False])
def test_truncation(topp, renorm):
    for score in ("sigmoid", "softmax"):
        check(logits(65, 256, 3), bias_of(256, 2), 8, score=score, topp=topp, renorm=renorm)
        check(logits(9, 24, 3, torch.bfloat16), None, 5, score=score, topp=topp, renorm=renorm, groups=3, keep=2)


@pytest.mark.parametrize("share", [0.3, 0.8, 0.97, 1.0])
@pytest.mark.parametrize("E,G,keep,k", [(8, 1, 1, 4), (24, 3, 2, 5), (256, 8, 4, 8), (512, 1, 1, 32)])
def test_masked_experts(share, E, G, keep, k):
    """Masks that leave fewer than k experts, one group of several, or none."""
    g = torch.Generator().manual_seed(E)
    lg = torch.randn(150, E, generator=g).masked_fill(torch.rand(150, E, generator=g) < share, -float("inf"))
    lg[17] = -float("inf")
    lg[18, 1:] = -float("inf")
    for dtype in (torch.float32, torch.bfloat16):
        for score, b in (("sigmoid", True), ("softmax", True), ("softmax", False), ("sigmoid", False)):
            idx, w = check(lg.to(dtype).cuda(), bias_of(E, 5) if b else None, k, score=score, groups=G, keep=keep)
            assert (idx[17] == -1).all() and (w[17] == 0).all()
            assert (w[idx == -1] == 0).all()


def test_not_a_number_and_infinities():
    nan, inf = float("nan"), float("inf")
    lg = logits(12, 64, 1).clone()
    lg[0, 5] = nan
    lg[1, :] = nan
    lg[2, 7] = inf
    lg[3, 7] = lg[3, 9] = inf  # two that share all the mass
    lg[4, 3] = -inf
    lg[5, 0], lg[5, 1], lg[5, 2] = nan, inf, -inf
    lg[6] = torch.finfo(torch.float32).min  # the type's lowest value is a logit like another
    lg[7, ::2] = torch.finfo(torch.float32).min
    lg[8] = torch.finfo(torch.float32).max
    lg[9] = 0.0
    for b in (None, bias_of(64, 3)):
        for score in ("sigmoid", "softmax"):
            for kw in ({}, {"groups": 8, "keep": 3}, {"groups": 4, "keep": 2, "value": "max"}):
                check(lg, b, 6, score=score, renorm=False, **kw)
                check(lg, b, 6, score=score, **kw)
    b = bias_of(64, 4)
    b[1], b[2], b[3], b[60] = nan, -inf, inf, inf
    for score in ("sigmoid", "softmax"):
        check(lg, b, 6, score=score)
        check(lg, b, 6, score=score, groups=8, keep=3)
        check(lg, torch.full_like(b, -inf), 6, score=score)


@pytest.mark.parametrize("E,k,G,keep", [(8, 3, 1, 1), (24, 5, 3, 2), (64, 8, 8, 4), (256, 8, 1, 1), (256, 8, 8, 4),
                                        (1024, 32, 1, 1)])
def test_ties_take_the_lower_index(E, k, G, keep):
    lg = torch.zeros(20, E, device="cuda")
    lg[1] = 3.25
    lg[2, E // 2:] = 1.0
    lg[3, ::3] = 2.0
    lg[4] = torch.randint(0, 3, (E,), generator=torch.Generator().manual_seed(1)).float().cuda()
    lg[5:] = torch.randint(0, 2, (15, E), generator=torch.Generator().manual_seed(2)).float().cuda()
    flat = torch.full((E,), 0.125, device="cuda")
    levels = (torch.randint(-2, 3, (E,), generator=torch.Generator().manual_seed(3)).float() * 0.125).cuda()
    for b in (None, flat, levels):
        for score in ("sigmoid", "softmax"):
            for value in ("top2", "max"):
                check(lg, b, k, score=score, groups=G, keep=keep, value=value)


def test_scores_that_float32_cannot_tell_apart():
    """Sigmoids near 1 (or far below 1 against a bias) differ in double only;
    the order, of experts and of groups, is the double one."""
    E = 256
    g = torch.Generator().manual_seed(8)
    lg = torch.full((40, E), -4.0)
    for t in range(40):
        at = torch.randperm(E, generator=g)[:20]
        lg[t, at] = 14.0 + 4e-6 * torch.randperm(20, generator=g).float() * (1 + t % 5)
    lg = lg.cuda()
    assert (torch.sigmoid(lg).sort(1, descending=True)[0][:, :20].diff(dim=1) == 0).any()
    for b in (torch.zeros(E, device="cuda"), torch.full((E,), 0.5, device="cuda"), None):
        for G, keep in ((1, 1), (8, 4), (32, 6)):
            for value in ("top2", "max"):
                check(lg, b, 8, groups=G, keep=keep, value=value)
    small = (-30.0 + 8.0 * torch.rand(40, E, generator=g)).cuda()
    check(small, torch.full((E,), 1.0, device="cuda"), 8)
    check(small, torch.full((E,), 100.0, device="cuda"), 8, groups=16, keep=5)
    check(small, bias_of(E, 1, 1e-6), 8, score="softmax")


def test_biases_far_apart():
    """One bias that dwarfs the scores leaves the rest of the row in order."""
    lg = logits(33, 256, 9)
    b = bias_of(256, 9)
    b[100] = -1e30
    check(lg, b, 8)
    b[7] = 1e6
    check(lg, b, 8)
    check(lg, b, 8, score="softmax", groups=8, keep=2)
    b[9] = 3e38
    check(lg, b, 8)


def test_weights_of_scores_that_underflow():
    lg = -torch.linspace(60, 700, 64).repeat(3, 1).cuda()
    check(lg, None, 8)  # float32 sigmoids are 0 from 104 on, double ones are not
    check(lg - 100, torch.linspace(1, 0, 64).cuda(), 8)
    idx, w = select(torch.full((2, 64), -1e4, device="cuda"), None, 8)
    assert (w == 0).all() and (idx == np.arange(8)).all()


def test_repeated_calls_agree_and_rows_behind_the_last_stay():
    lg, b = logits(777, 256, 4, torch.bfloat16), bias_of(256, 4)
    c, r = M.config(128, 64, 256, 8), M.gate_rule("sigmoid", 8, 4)
    idx = torch.full((780, 8), -7, dtype=torch.int32, device="cuda")
    w = torch.full((780, 8), -7.0, device="cuda")
    M.moe_gate(c, r, lg, b, idx[:777], w[:777])
    first = idx.clone(), w.clone()
    for _ in range(3):
        M.moe_gate(c, r, lg, b, idx[:777], w[:777])
    assert torch.equal(idx, first[0]) and torch.equal(w, first[1])
    assert (idx[777:] == -7).all() and (w[777:] == -7.0).all()


def test_other_stream_and_captured_graph():
    lg, b = logits(64, 256, 6), bias_of(256, 6)
    c, r = M.config(128, 64, 256, 8), M.gate_rule("sigmoid", 8, 4)
    outs = [(torch.zeros(64, 8, dtype=torch.int32, device="cuda"), torch.zeros(64, 8, device="cuda")) for _ in range(2)]
    M.moe_gate(c, r, lg, b, *outs[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    M.moe_gate(c, r, lg, b, *outs[1], stream=s)
    s.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.moe_gate(c, r, lg, b, *outs[1])
    lg.copy_(logits(64, 256, 60))
    g.replay()
    torch.cuda.synchronize()
    r_idx, _ = gate(lg, b, 8, groups=8, keep=4)
    np.testing.assert_array_equal(outs[1][0].cpu().numpy(), r_idx)


@pytest.mark.parametrize("T", [1, 4, 8, 9, 70])
def test_route_gated_is_the_projection_and_the_gate(T):
    """With the zero rule it selects as moe_route; with a rule, as the rule on
    the projection's logits (their error: 2e-6 of the logits' spread, so rows
    whose border is nearer than that are left out)."""
    wl = W.workload(1)
    d, E, k = 512, 256, 8
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, d, generator=g)
    wr = 0.05 * torch.randn(E, d, generator=g)
    b = bias_of(E, T)
    c = M.config(d, 128, E, k)
    ws = M.workspace(c, T)
    out = [(torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")) for _ in range(2)]
    M.moe_route(c, x.cuda(), wr.cuda(), b, *out[0], ws)
    M.moe_route_gated(c, M.gate_rule(), x.cuda(), wr.cuda(), b, *out[1], ws)
    lg = x.double() @ wr.double().T
    sel = torch.sigmoid(lg) + b.cpu().double()
    top = sel.sort(1, descending=True)[0][:, :k + 1]
    clear = (top.diff(dim=1).abs().min(1)[0] > 2e-5).numpy()
    assert clear.sum() > 0.8 * T
    np.testing.assert_array_equal(out[0][0].cpu().numpy()[clear], out[1][0].cpu().numpy()[clear])
    np.testing.assert_allclose(out[0][1].cpu().numpy()[clear], out[1][1].cpu().numpy()[clear], rtol=4e-6)
    M.moe_route_gated(c, M.gate_rule("softmax", 8, 3, "max"), x.bfloat16().cuda(), wr.cuda(), None, *out[1], ws)
    assert M.moe_poll_status(ws) == M.MOE_OK
    lg = x.bfloat16().double() @ wr.double().T
    r_idx, r_w = gate(lg, None, k, score="softmax", groups=8, keep=3, value="max")
    p = torch.softmax(lg, 1)
    gv = p.view(T, 8, 32).amax(2).sort(1, descending=True)[0]
    top = lg.sort(1, descending=True)[0][:, :64].diff(dim=1).abs()
    kept = [np.sort(lg[t, torch.as_tensor(sorted(set(e // 32 for e in range(E) if gv[t, 2] <= p[t].view(8, 32).amax(1)[e // 32])))
                       .repeat_interleave(32) * 32 + torch.arange(32).repeat(3)].numpy())[::-1][:k + 1] for t in range(T)]
    clear = np.array([(gv[t, 2] - gv[t, 3] > 1e-5 * gv[t, 2]).item() and np.abs(np.diff(kept[t])).min() > 2e-5
                      for t in range(T)])
    assert clear.sum() > 0.7 * T
    np.testing.assert_array_equal(out[1][0].cpu().numpy()[clear], r_idx[clear])
    np.testing.assert_allclose(out[1][1].cpu().numpy()[clear], r_w[clear], rtol=3e-5)


def rel_l2(a, b):
    return float(np.linalg.norm(np.asarray(a, np.float64) - b) / np.linalg.norm(b))


@pytest.mark.parametrize("T,tc", [(1, 0), (2, 0), (5, -1), (5, 0), (32, 0), (32, -1)])
def test_layer_routed_equals_the_layer_on_its_own_routing(T, tc):
    """Fed with the routing that moe_layer itself reports, the routed layer
    gives the layer's output: the same integer products on either path."""
    wl = W.workload(0).replace(T=T)
    dl = W.device_layer(wl, 0, 0, "cuda:0")
    c = M.config(wl.d, wl.f, wl.n_experts, wl.top_k, 1, wl.wbits, wl.routed_scale, tc_min_tokens=tc)
    ws = M.workspace(c, T)
    x = W.tokens(wl, 0, 0, T).cuda()
    pool = M.make_pool(dl.pool_w, dl.pool_s)
    out, out2 = torch.empty(T, wl.d, device="cuda"), torch.empty(T, wl.d, device="cuda")
    idx = torch.empty(T, wl.top_k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, wl.top_k, device="cuda")
    M.moe_layer(c, pool, dl.w_router, dl.bias, x, out, ws, topk_idx_out=idx, topk_w_out=w)
    M.moe_layer_routed(c, pool, idx, w, x, out2, ws)
    assert M.moe_poll_status(ws) == M.MOE_OK
    assert rel_l2(out2.cpu().numpy(), out.cpu().numpy()) < 2e-3  # the layer's own tolerance (a code may flip)
    out3 = torch.ones(T, wl.d, device="cuda")
    M.moe_layer_routed(c, pool, idx, w, x, out3, ws, accumulate=True)
    torch.testing.assert_close(out3, out2 + 1, rtol=1e-6, atol=1e-6)


def expert_out(c, pool, e, x, ws):
    T = x.shape[0]
    xq, sx = torch.empty(T, c.d, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    y = torch.empty(T, c.d, device="cuda")
    M.moe_quantize(c, x, xq, sx)
    M.moe_expert_ffn(c, pool, e, xq, sx, y, ws)
    return y.double()


@pytest.mark.parametrize("tc", [0, -1])
@pytest.mark.parametrize("shared", [0, 1])
def test_layer_routed_takes_any_routing(tc, shared):
    """Empty slots, empty rows, one expert in every slot of a row, an index
    that is no expert's: the output is the sum over the slots, expert by
    expert, and the bad index is recorded."""
    wl = W.workload(0).replace(has_shared=shared)
    T, k = 7, 4
    dl = W.device_layer(wl, 0, 0, "cuda:0")
    c = M.config(wl.d, wl.f, wl.n_experts, k, shared, wl.wbits, 1.0, tc_min_tokens=tc)
    pool = M.make_pool(dl.pool_w, dl.pool_s)
    ws = M.workspace(c, T)
    x = W.tokens(wl, 0, 0, T).cuda()
    rows = [[3, 3, 3, 3], [-1, -1, -1, -1], [0, -1, 7, -1], [7, 6, 5, 4], [-1, 2, 2, 1], [3, 3, 3, 3], [3, 3, 3, 3]]
    idx = torch.tensor(rows, dtype=torch.int32, device="cuda")
    w = torch.rand(T, k, generator=torch.Generator().manual_seed(1)).cuda() + 0.1
    ys = [expert_out(c, pool, e, x, ws) for e in range(wl.n_experts)]
    want = expert_out(c, pool, -1, x, ws) if shared else torch.zeros(T, wl.d, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            if rows[t][j] >= 0:
                want[t] += w[t, j].double() * ys[rows[t][j]][t]
    out = torch.full((T, wl.d), 9.0, device="cuda")
    M.moe_layer_routed(c, pool, idx, w, x, out, ws)
    assert M.moe_poll_status(ws) == M.MOE_OK
    assert rel_l2(out.cpu().numpy(), want.cpu().numpy()) < 2e-3
    if not shared:
        assert (out[1] == 0).all()
    none = torch.full_like(idx, -1)
    M.moe_layer_routed(c, pool, none, w, x, out, ws)
    assert M.moe_poll_status(ws) == M.MOE_OK
    want = expert_out(c, pool, -1, x, ws) if shared else torch.zeros(T, wl.d, dtype=torch.float64, device="cuda")
    assert float((out.double() - want).norm()) <= 2e-3 * float(want.norm())
    kept = out.clone()
    M.moe_layer_routed(c, pool, none, w, x, out, ws, accumulate=True)
    torch.testing.assert_close(out, 2 * kept, rtol=1e-6, atol=0)
    bad = none.clone()
    bad[2, 1] = wl.n_experts
    M.moe_layer_routed(c, pool, bad, w, x, out, ws)
    assert M.moe_poll_status(ws) == M.MOE_EDEVICE
    assert torch.equal(out, kept)  # the slot is dropped
    M.moe_workspace_init(ws)
    bad[2, 1] = -2
    M.moe_layer_routed(c, pool, bad, w, x, out, ws)
    assert M.moe_poll_status(ws) == M.MOE_EDEVICE


def test_layer_routed_one_expert_for_all_slots_of_a_batch():
    """64 tokens that name one expert in each of their 8 slots: 512 rows of one
    expert, tasks fuller than a call of distinct experts has."""
    wl = W.workload(0).replace(T=64)
    dl = W.device_layer(wl, 0, 0, "cuda:0")
    for T, tc in ((64, 0), (3, 0), (3, -1), (1, -1)):
        c = M.config(wl.d, wl.f, wl.n_experts, 8, 1, wl.wbits, 1.0, tc_min_tokens=tc)
        pool = M.make_pool(dl.pool_w, dl.pool_s)
        ws = M.workspace(c, T)
        x = W.tokens(wl, 0, 0, T).cuda()
        idx = torch.full((T, 8), 5, dtype=torch.int32, device="cuda")
        w = torch.full((T, 8), 0.25, device="cuda")
        out = torch.empty(T, wl.d, device="cuda")
        M.moe_layer_routed(c, pool, idx, w, x, out, ws)
        assert M.moe_poll_status(ws) == M.MOE_OK
        want = expert_out(c, pool, -1, x, ws) + 2 * expert_out(c, pool, 5, x, ws)
        assert rel_l2(out.cpu().numpy(), want.cpu().numpy()) < 2e-3
