"""moe_adapter against its sum in 64 bits, within the bound that
gate_reference.adapter derives for float32 sums."""
import pytest
import torch

import expert_ffn_router_b200 as M
import workloads as W
from gate_reference import adapter, gate

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8}


class Set:
    def __init__(self, n, r_max, d_in, d_out, ranks=None, seed=0, scale=True, junk=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.a = (torch.randn(n, r_max, d_in, generator=g, device="cuda") / d_in ** 0.5).bfloat16()
        self.b = torch.randn(n, d_out, r_max, generator=g, device="cuda").bfloat16()
        self.ranks = ranks if ranks is not None else [r_max] * n
        if junk:  # what lies beyond a rank takes no part
            for i, r in enumerate(self.ranks):
                self.a[i, r:] = float("nan")
                self.b[i, :, r:] = float("inf")
        self.rank = torch.tensor(self.ranks, dtype=torch.int32, device="cuda") if ranks is not None else None
        self.scale = 0.5 + torch.rand(n, generator=g, device="cuda") if scale else None
        self.c = M.make_adapters(self.a, self.b, self.rank, self.scale)

    def want(self, x, sx, of, base):
        return adapter(x, sx, of, self.a, self.b, self.ranks, self.scale, base)


def rows(T, d, dtype, seed=1, ld=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, ld or d, generator=g, device="cuda")
    if dtype == "i8":
        sx = x[:, :d].abs().amax(1) / 127
        return torch.clamp(torch.round(x / sx[:, None]), -127, 127).to(torch.int8)[:, :d], sx
    return x.to(DT[dtype])[:, :d], None


def owners(T, n, kind, seed=2):
    g = torch.Generator().manual_seed(seed)
    of = torch.randint(-1, n, (T,), generator=g)
    if kind == "runs":
        of = of.sort(descending=True)[0]
    if kind == "one":
        of[:] = n - 1
    if kind == "none":
        of[:] = -1
    return of.to(torch.int32).cuda()


def close(y, want):
    ref, err = want
    off = (y.double() - ref).abs()
    assert torch.isfinite(ref).all()
    assert bool((off <= err + 1e-30).all()), f"{float((off / (err + 1e-30)).max()):.3g} of the bound"


def check(s, T, dtype, of, base=True, ldx=None, ldy=None, in_place=False):
    x, sx = rows(T, s.c.d_in, dtype, ld=ldx)
    wide = torch.full((T + 2, ldy or s.c.d_out), 7.0, device="cuda")
    y = wide[:T, :s.c.d_out]
    b = torch.randn(T, s.c.d_out, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    plan = M.adapter_plan(s.c.n_adapters, of)
    want = s.want(x, sx, of, b if base else None)
    if in_place:
        y.copy_(b)
        M.moe_adapter(s.c, plan, x, y, base=y, sx=sx)
    else:
        M.moe_adapter(s.c, plan, x, y, base=b if base else None, sx=sx)
    assert M.moe_poll_status(plan) == M.MOE_OK
    close(y, want)
    assert (wide[T:] == 7.0).all() and (wide[:, s.c.d_out:] == 7.0).all()
    return y


SHAPES = [  # T, n, r_max, ranks, d_in, d_out
    (1, 1, 8, None, 16, 16), (1, 4, 16, None, 128, 128), (2, 3, 16, [1, 16, 5], 256, 64), (7, 5, 8, [0, 8, 3, 1, 7], 48, 80),
    (16, 2, 32, None, 128, 48), (17, 2, 64, [33, 64], 1040, 208), (33, 9, 24, None, 400, 1008),
    (63, 1, 64, None, 128, 128), (64, 1, 128, None, 256, 256), (65, 2, 128, [127, 97], 272, 144),
    (130, 40, 40, [(7 * i) % 41 for i in range(40)], 512, 96), (200, 3, 16, None, 2048, 512),
    (9, 1024, 8, None, 32, 32), (300, 2, 48, [17, 48], 96, 2064), (128, 3, 104, [104, 1, 56], 160, 176)]


@pytest.mark.parametrize("T,n,r_max,ranks,d_in,d_out", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "i8"])
def test_shapes(T, n, r_max, ranks, d_in, d_out, dtype):
    s = Set(n, r_max, d_in, d_out, ranks)
    check(s, T, dtype, owners(T, n, "mixed"))
    check(s, T, dtype, owners(T, n, "runs"), base=False)
    check(s, T, dtype, owners(T, n, "one"), in_place=True)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("T,n,r_max,d_in,d_out", [(1, 4, 16, 6144, 6144), (40, 24, 64, 2048, 6144),
                                                  (520, 3, 64, 6144, 2048), (1500, 5, 32, 1024, 1024),
                                                  (3, 2, 128, 32768, 64), (3, 2, 128, 64, 32768)])
def test_large_shapes(T, n, r_max, d_in, d_out, dtype):
    ranks = [r_max - (5 * i) % (r_max // 2) for i in range(n)]
    s = Set(n, r_max, d_in, d_out, ranks)
    check(s, T, dtype, owners(T, n, "mixed"))
    check(s, T, dtype, owners(T, n, "runs"), base=False)


MANY = [  # rows enough for the kernel of many rows (rank above 32, 2048 rows, 256 an adapter)
    (2048, 1, 40, None, 64, 80), (2111, 3, 64, [64, 33, 0], 272, 528), (2600, 4, 128, [127, 97, 128, 5], 144, 96),
    (2050, 8, 64, [17, 64, 8, 48, 40, 1, 63, 32], 1040, 272), (4097, 2, 48, [16, 24], 512, 2064)]


@pytest.mark.parametrize("T,n,r_max,ranks,d_in,d_out", MANY)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "i8"])
def test_many_rows(T, n, r_max, ranks, d_in, d_out, dtype):
    s = Set(n, r_max, d_in, d_out, ranks)
    check(s, T, dtype, owners(T, n, "mixed"))
    check(s, T, dtype, owners(T, n, "runs"), base=False)
    check(s, T, dtype, owners(T, n, "runs"), in_place=True)
    check(s, T, dtype, owners(T, n, "one"), ldx=d_in + 48, ldy=d_out + 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "i8"])
@pytest.mark.parametrize("kind", ["mixed", "runs"])
def test_many_rows_large(dtype, kind):
    s = Set(4, 64, 6144, 2048, [64, 50, 9, 33])
    check(s, 3000, dtype, owners(3000, 4, kind))
    s = Set(2, 64, 1024, 6144, [61, 64])
    check(s, 2500, dtype, owners(2500, 2, kind))


def test_many_rows_in_graphs_and_on_two_streams():
    s = Set(4, 64, 512, 512, [64, 7, 40, 16])
    of = owners(2304, 4, "runs")
    plan = M.adapter_plan(4, of)
    x, _ = rows(2304, 512, "bf16")
    y = [torch.empty(2304, 512, device="cuda") for _ in range(3)]
    M.moe_adapter(s.c, plan, x, y[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    few = M.adapter_plan(4, of[:100].contiguous())
    z = torch.empty(100, 512, device="cuda")
    for _ in range(5):  # both kernels at once, too
        M.moe_adapter(s.c, plan, x, y[1])
        M.moe_adapter(s.c, plan, x, y[2], stream=side)
        M.moe_adapter(s.c, few, x[:100], z, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.moe_adapter_plan(4, of, plan)
        M.moe_adapter(s.c, plan, x, y[1])
    of.copy_(owners(2304, 4, "mixed", seed=9))
    x.copy_(rows(2304, 512, "bf16", seed=10)[0])
    g.replay()
    torch.cuda.synchronize()
    close(y[1], s.want(x, None, of, None))


def test_many_rows_that_are_not_finite_stay_alone():
    s = Set(2, 64, 128, 64)
    for dtype in ("f32", "bf16"):
        of = owners(2100, 2, "mixed")
        of[:4] = torch.tensor([0, 1, 0, -1])
        x, _ = rows(2100, 128, dtype)
        clean = x.clone()
        x[0, 3], x[1, 5], x[3, 0] = float("nan"), float("inf"), float("nan")
        plan = M.adapter_plan(2, of)
        y, z = torch.zeros(2100, 64, device="cuda"), torch.zeros(2100, 64, device="cuda")
        M.moe_adapter(s.c, plan, x, y)
        M.moe_adapter(s.c, plan, clean, z)
        assert not torch.isfinite(y[0]).any() and not torch.isfinite(y[1]).any()
        assert torch.equal(y[2:], z[2:])


@pytest.mark.parametrize("dtype,ldx", [("f32", 4), ("f32", 60), ("bf16", 8), ("i8", 16)])
def test_rows_that_lie_apart(dtype, ldx):
    s = Set(3, 16, 112, 80, [16, 9, 2])
    for T in (1, 5, 70):
        check(s, T, dtype, owners(T, 3, "mixed"), ldx=112 + ldx, ldy=84)
        check(s, T, dtype, owners(T, 3, "mixed"), ldx=112 + ldx, ldy=128, in_place=True)


def test_rows_without_an_adapter():
    s = Set(2, 16, 64, 64)
    x, _ = rows(70, 64, "bf16")
    of = owners(70, 2, "none")
    plan = M.adapter_plan(2, of)
    y = torch.full((70, 64), 3.0, device="cuda")
    M.moe_adapter(s.c, plan, x, y, base=y)
    assert (y == 3.0).all()
    b = torch.randn(70, 64, device="cuda")
    M.moe_adapter(s.c, plan, x, y, base=b)
    assert torch.equal(y, b)
    M.moe_adapter(s.c, plan, x, y)
    assert (y == 0).all()


def test_no_scale_no_rank_and_rank_out_of_range():
    s = Set(2, 16, 64, 64, scale=False)
    check(s, 20, "f32", owners(20, 2, "mixed"))
    s = Set(3, 16, 64, 64, [16, 0, 16], junk=False)
    s.rank.copy_(torch.tensor([99, -5, 16], dtype=torch.int32))
    check(s, 20, "bf16", owners(20, 3, "mixed"))


def test_float32_rows_keep_all_their_bits():
    """Products that cancel to what the last of a float32's 24 bits leave: an
    evaluation on fewer bits of x, or of A x, is off by far more."""
    s = Set(1, 16, 256, 64)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(6, 128, generator=g, device="cuda")
    fine = x * (1 + 2.0 ** -20)
    x = torch.cat([x, -fine], 1).contiguous()
    s.a[0, :, 128:] = s.a[0, :, :128]
    of = owners(6, 1, "one")
    y = torch.empty(6, 64, device="cuda")
    M.moe_adapter(s.c, M.adapter_plan(1, of), x, y)
    ref, _ = s.want(x, None, of, None)
    # each half's sum is 2^20 times the difference; a float32 sum of it is off by 2^-23 of that at each of at most
    # 256 / 8 + 16 additions, and in fact by about their square root of a half of it
    assert float((y.double() - ref).norm() / ref.norm()) < 2.0 ** -23 * 2.0 ** 20 * 7


def test_values_that_are_not_finite_stay_in_their_row():
    s = Set(2, 16, 128, 64)
    for T in (5, 70):
        of = owners(T, 2, "mixed")
        of[:4] = torch.tensor([0, 1, 0, -1])
        x, _ = rows(T, 128, "f32")
        clean = x.clone()
        x[0, 3], x[1, 5], x[3, 0] = float("nan"), float("inf"), float("nan")
        plan = M.adapter_plan(2, of)
        y, z = torch.zeros(T, 64, device="cuda"), torch.zeros(T, 64, device="cuda")
        M.moe_adapter(s.c, plan, x, y)
        M.moe_adapter(s.c, plan, clean, z)
        assert not torch.isfinite(y[0]).any() and not torch.isfinite(y[1]).any()
        assert torch.equal(y[2:], z[2:])


def test_large_and_tiny_values():
    s = Set(1, 16, 64, 64)
    of = owners(3, 1, "one")
    x, _ = rows(3, 64, "f32")
    for f in (1e-30, 1e30):
        xs = x * f
        y = torch.empty(3, 64, device="cuda")
        M.moe_adapter(s.c, M.adapter_plan(1, of), xs, y)
        close(y, s.want(xs, None, of, None))


def test_plan():
    """Rows grouped by adapter in their order, tasks of at most 8 and of at most 64."""
    for T, n in ((1, 1), (64, 2), (65, 1), (1000, 7), (5000, 300), (3000, 1024), (0, 3)):
        of = owners(T, n, "mixed") if T else torch.empty(0, dtype=torch.int32, device="cuda")
        plan = M.adapter_plan(n, of).cpu()
        head = plan[:64].view(torch.int32)
        order = plan[64:64 + 4 * T].view(torch.int32)
        assert head[0] == 0 and head[3] == T and head[4] == n
        key = of.cpu().clone()
        key[key < 0] = n
        assert order.tolist() == key.sort(stable=True)[1].tolist()
        at = (64 + 4 * T + 15) // 16 * 16
        for i, most in enumerate((8, 64)):
            tasks = plan[at:at + 16 * int(head[5 + i])].view(torch.int32).view(-1, 4).tolist()
            at += 16 * (min(T, n + 1) + T // most)
            seen = 0
            for a, first, cnt, together in tasks:
                assert first == seen and 1 <= cnt <= most
                assert (of.cpu()[order[first:first + cnt].long()] == a).all()
                assert together == int(bool((order[first:first + cnt].diff() == 1).all()))
                seen += cnt
            assert seen == T
        assert plan.numel() == at


def test_bad_owner_is_recorded_and_counts_as_none():
    s = Set(3, 8, 32, 32)
    of = torch.tensor([0, 3, -2, 1, 2], dtype=torch.int32, device="cuda")
    plan = M.adapter_plan(3, of)
    assert M.moe_poll_status(plan) == M.MOE_EDEVICE
    x, _ = rows(5, 32, "bf16")
    y = torch.empty(5, 32, device="cuda")
    M.moe_adapter(s.c, plan, x, y)
    fixed = torch.tensor([0, -1, -1, 1, 2], dtype=torch.int32, device="cuda")
    close(y, s.want(x, None, fixed, None))
    M.moe_adapter_plan(3, fixed, plan)
    assert M.moe_poll_status(plan) == M.MOE_OK  # a plan made anew starts clean


def test_plan_of_another_batch_is_refused():
    s = Set(3, 8, 32, 32)
    plan = M.adapter_plan(3, owners(9, 3, "mixed"))
    x, _ = rows(8, 32, "bf16")
    y = torch.full((8, 32), 5.0, device="cuda")
    M.moe_adapter(s.c, plan, x, y)
    assert M.moe_poll_status(plan) == M.MOE_EDEVICE
    assert (y == 5.0).all()
    plan = M.adapter_plan(4, owners(8, 3, "mixed"))
    M.moe_adapter(s.c, plan, x, y)
    assert M.moe_poll_status(plan) == M.MOE_EDEVICE
    plan = torch.zeros(M.moe_adapter_plan_bytes(3, 8), dtype=torch.uint8, device="cuda")  # never made
    M.moe_adapter(s.c, plan, x, y)
    assert M.moe_poll_status(plan) == M.MOE_EDEVICE
    assert (y == 5.0).all()


def test_repeated_calls_two_streams_and_graph():
    s = Set(6, 32, 512, 256, [32, 7, 16, 1, 30, 8])
    of = owners(90, 6, "mixed")
    plan = M.adapter_plan(6, of)
    x, _ = rows(90, 512, "f32")
    y = [torch.empty(90, 256, device="cuda") for _ in range(3)]
    M.moe_adapter(s.c, plan, x, y[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):  # two calls on one plan at once
        M.moe_adapter(s.c, plan, x, y[1])
        M.moe_adapter(s.c, plan, x, y[2], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.moe_adapter_plan(6, of, plan)
        M.moe_adapter(s.c, plan, x, y[1])
    of.copy_(owners(90, 6, "runs", seed=9))
    x.copy_(rows(90, 512, "f32", seed=10)[0])
    g.replay()
    torch.cuda.synchronize()
    close(y[1], s.want(x, None, of, None))


def test_offsets_beyond_32_bits():
    """Tables and rows whose offsets pass 2^31 elements."""
    n, r, d = 130, 128, 32768  # 545 M elements a table, 1.1 GB; the last adapter's offset is 2^29
    a = torch.zeros(n, r, d, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(n, 64, r, dtype=torch.bfloat16, device="cuda")
    a[-1] = 0.01
    b[-1] = 1.0
    ad = M.make_adapters(a, b)
    T, ld = 3, 1 << 30
    wide = torch.empty((T - 1) * ld + d, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(wide, (T, d), (ld, 1))
    x.fill_(0.5)
    yw = torch.empty((T - 1) * ld + 64, dtype=torch.float32, device="cuda")
    y = torch.as_strided(yw, (T, 64), (ld, 1))
    of = torch.tensor([n - 1, -1, n - 1], dtype=torch.int32, device="cuda")
    M.moe_adapter(ad, M.adapter_plan(n, of), x, y)
    want = 128 * 32768 * 0.5 * float(torch.tensor(0.01).bfloat16())
    assert torch.allclose(y[0], torch.full_like(y[0], want), rtol=1e-4)
    assert (y[1] == 0).all()
    assert torch.equal(y[2], y[0])


def test_binding_refuses():
    s = Set(2, 8, 32, 32)
    plan = M.adapter_plan(2, owners(4, 2, "mixed"))
    x, sx = rows(4, 32, "i8")
    y = torch.empty(4, 32, device="cuda")
    for bad in (lambda: M.moe_adapter(s.c, plan, x[:, :16], y, sx=sx),
                lambda: M.moe_adapter(s.c, plan, x, y[:3], sx=sx),
                lambda: M.moe_adapter(s.c, plan, x, y, base=y[:2], sx=sx),
                lambda: M.moe_adapter(s.c, plan, x, y.double(), sx=sx),
                lambda: M.moe_adapter(s.c, plan, x, y.t(), sx=sx),
                lambda: M.moe_adapter(s.c, plan, x.half(), y)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(M.MoeError):
        M.moe_adapter(s.c, plan, x, y)  # codes without scales


def test_gate_layer_and_adapters_together():
    """A step as a serving program runs it: logits -> gate -> the layer's
    experts -> each request's adapter on the layer's output, and the down
    projection of the shared expert with its adapter on the same codes."""
    wl = W.workload(0)
    T, d, f, E, k = 32, wl.d, wl.f, wl.n_experts, 3
    dl = W.device_layer(wl, 0, 0, "cuda:0")
    c = M.config(d, f, E, k, 1, wl.wbits, wl.routed_scale)
    pool = M.make_pool(dl.pool_w, dl.pool_s)
    ws = M.workspace(c, T)
    x = W.tokens(wl, 0, 0, T).cuda()
    lg = x @ dl.w_router.T
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    rule = M.gate_rule("sigmoid", 4, 2)
    of = owners(T, 5, "mixed")
    s, sd = Set(5, 16, d, d, [16, 3, 8, 9, 1]), Set(5, 8, f, d)
    plan = M.adapter_plan(5, of)
    out = torch.empty(T, d, device="cuda")
    M.moe_gate(c, rule, lg, dl.bias, idx, w)
    M.moe_layer_routed(c, pool, idx, w, x, out, ws)
    layer = out.clone()
    M.moe_adapter(s.c, plan, x, out, base=out)
    r_idx, _ = gate(lg, dl.bias, k, groups=4, keep=2)
    assert (idx.cpu().numpy() == r_idx).all()
    close(out, s.want(x, None, of, layer))
    hq = torch.randint(-127, 128, (T, f), dtype=torch.int8, device="cuda")
    sh = torch.rand(T, device="cuda")
    y = torch.empty(T, d, device="cuda")
    M.moe_expert_down(c, pool, -1, hq, sh, y, ws)
    shared = y.clone()
    M.moe_adapter(sd.c, plan, hq, y, base=y, sx=sh)
    close(y, sd.want(hq, sh, of, shared))
    assert M.moe_poll_status(ws) == M.MOE_OK and M.moe_poll_status(plan) == M.MOE_OK
