"""The selection, the routed layer and the adapters as a serving step runs them:
captured and replayed on new inputs, on one workspace in turn with moe_layer,
and the projection with the selection beside moe_route's."""
import numpy as np
import pytest
import torch

import expert_ffn_router_b200 as M
import workloads as W

pytestmark = pytest.mark.gpu


def parts(T, shared=1, tc=0):
    wl = W.workload(0).replace(T=T, has_shared=shared)
    dl = W.device_layer(wl, 0, 0, "cuda:0")
    c = M.config(wl.d, wl.f, wl.n_experts, wl.top_k, shared, wl.wbits, wl.routed_scale, tc_min_tokens=tc)
    return wl, dl, c, M.make_pool(dl.pool_w, dl.pool_s)


@pytest.mark.parametrize("T,tc", [(1, 0), (2, -1), (7, 0), (40, 0), (40, -1)])
def test_a_step_in_a_graph(T, tc):
    wl, dl, c, pool = parts(T, tc=tc)
    d, E, k, n = wl.d, wl.n_experts, wl.top_k, 3
    g = torch.Generator(device="cuda").manual_seed(T)
    ad = M.make_adapters((torch.randn(n, 16, d, generator=g, device="cuda") / d ** 0.5).bfloat16(),
                         torch.randn(n, d, 16, generator=g, device="cuda").bfloat16())
    rule = M.gate_rule("softmax", 4, 2)
    ws = M.workspace(c, T)
    plan = torch.empty(M.moe_adapter_plan_bytes(n, T), dtype=torch.uint8, device="cuda")
    x, out = torch.empty(T, d, device="cuda"), torch.empty(T, d, device="cuda")
    of = torch.empty(T, dtype=torch.int32, device="cuda")
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")

    def inputs(seed):
        x.copy_(W.tokens(wl, seed, 0, T))
        of.copy_(torch.randint(-1, n, (T,), generator=torch.Generator().manual_seed(seed)))

    def step():
        M.moe_route_gated(c, rule, x, dl.w_router, dl.bias, idx, w, ws)
        M.moe_layer_routed(c, pool, idx, w, x, out, ws)
        M.moe_adapter_plan(n, of, plan)
        M.moe_adapter(ad, plan, x, out, base=out)

    want = {}
    for seed in (0, 1, 2):
        inputs(seed)
        step()
        want[seed] = (idx.clone(), w.clone(), out.clone())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 0, 2, 1):
        inputs(seed)
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((idx, w, out), want[seed]):
            assert torch.equal(got, ref)
    assert M.moe_poll_status(ws) == M.MOE_OK and M.moe_poll_status(plan) == M.MOE_OK


@pytest.mark.parametrize("shared", [0, 1])
def test_in_turn_with_the_layer_on_one_workspace(shared):
    """Each call leaves the workspace as the others need it: the decode kernel,
    both expert paths, batches of several sizes, rows without experts."""
    wl, dl, c, pool = parts(40, shared)
    dp4a = M.config(wl.d, wl.f, wl.n_experts, wl.top_k, shared, wl.wbits, wl.routed_scale, tc_min_tokens=-1)
    x = W.tokens(wl, 0, 0, 40).cuda()
    idx = torch.empty(40, wl.top_k, dtype=torch.int32, device="cuda")
    w = torch.empty(40, wl.top_k, device="cuda")
    M.moe_gate(c, M.gate_rule(), x @ dl.w_router.T, dl.bias, idx, w)
    idx[::3, 0] = -1
    idx[4] = -1

    def call(kind, T, ws):
        out = torch.full((T, wl.d), 3.0, device="cuda")
        if kind == "layer":
            M.moe_layer(c, pool, dl.w_router, dl.bias, x[:T], out, ws)
        elif kind == "gated":
            i, v = torch.empty_like(idx[:T]), torch.empty_like(w[:T])
            M.moe_route_gated(c, M.gate_rule("softmax"), x[:T], dl.w_router, None, i, v, ws)
            return v
        else:
            M.moe_layer_routed(c if kind == "tc" else dp4a, pool, idx[:T], w[:T], x[:T], out, ws)
        return out

    steps = [("layer", 1), ("dp4a", 1), ("layer", 1), ("tc", 5), ("layer", 1), ("layer", 2), ("gated", 3), ("tc", 40),
             ("dp4a", 40), ("layer", 8), ("dp4a", 2), ("layer", 40), ("gated", 40), ("dp4a", 7), ("layer", 1)]
    ws = M.workspace(c, 40)
    for kind, T in steps:
        got = call(kind, T, ws)
        ref = call(kind, T, M.workspace(c, 40))
        assert torch.equal(got, ref), (kind, T)
    assert M.moe_poll_status(ws) == M.MOE_OK


@pytest.mark.parametrize("topp", [0.3, 0.7])
@pytest.mark.parametrize("T", [3, 50])
def test_truncated_selection_beside_the_routers(T, topp):
    """With the zero rule and topp, as moe_route where no value is nearer to
    another, and no sum nearer to the border, than float32 logits and sums are
    off by (2e-5 of scores of order 1; eight scores' sum: 1e-4)."""
    d, E, k = 512, 256, 8
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, d, generator=g)
    wr = 0.05 * torch.randn(E, d, generator=g)
    b = 0.02 * (torch.rand(E, generator=g) - 0.5)
    c = M.config(d, 128, E, k, topp=topp)
    ws = M.workspace(c, T)
    out = [(torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")) for _ in range(2)]
    M.moe_route(c, x.cuda(), wr.cuda(), b.cuda(), *out[0], ws)
    M.moe_route_gated(c, M.gate_rule(), x.cuda(), wr.cuda(), b.cuda(), *out[1], ws)
    s = torch.sigmoid(x.double() @ wr.double().T)
    top, at = torch.sort(s + b.double(), dim=1, descending=True)
    apart = top[:, :k + 1].diff(dim=1).abs().min(1)[0] > 2e-5
    kept = s.gather(1, at[:, :k])
    border = (torch.cumsum(kept, 1) - topp * kept.sum(1, keepdim=True)).abs().min(1)[0] > 1e-4
    clear = (apart & border).numpy()
    assert clear.sum() > 0.8 * T
    np.testing.assert_array_equal(out[0][0].cpu().numpy()[clear], out[1][0].cpu().numpy()[clear])
    np.testing.assert_allclose(out[0][1].cpu().numpy()[clear], out[1][1].cpu().numpy()[clear], rtol=4e-6)
    assert (out[1][0][:, -1] == -1).any()
