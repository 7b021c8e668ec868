"""Measured cases of the routing and adapter operators.

Each case is one call as a serving program makes it: ``moe_gate`` picks the
experts of a batch from its router logits, ``moe_adapter`` adds the low-rank
adapters of many requests to a projection that all of them share.  ``run``
computes a case in plain torch operations, or, with ``own`` true, through the
library.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _gate(name, T, E, k, dtype, score, bias, groups=1, keep=1, group="top2", renorm=True, scale=2.5, topp=0.0,
          masked=0.0, pad=0):
    return {"name": name, "op": "gate", "T": T, "E": E, "k": k, "dtype": dtype, "score": score, "bias": bias,
            "groups": groups, "keep": keep, "group": group, "renorm": renorm, "scale": scale, "topp": topp,
            "masked": masked, "pad": pad}


def _adapter(name, T, n, r_max, ranks, d_in, d_out, dtype, spread, none=0.0, base=True):
    return {"name": name, "op": "adapter", "T": T, "n": n, "r_max": r_max, "ranks": ranks, "d_in": d_in,
            "d_out": d_out, "dtype": dtype, "spread": spread, "none": none, "base": base}


def listed():
    return [
        # one decoded token at the 256-expert layer: latency alone counts
        _gate("gate_decode_1", 1, 256, 8, "f32", "sigmoid", True),
        # a small softmax router without a bias, bf16 logits as a bf16 projection leaves them
        _gate("gate_tiny_32", 32, 8, 2, "bf16", "softmax", False, scale=1.0),
        # a decode batch with group-limited routing, every token's choice cut to half of the groups
        _gate("gate_decode_64", 64, 256, 8, "f32", "sigmoid", True, groups=8, keep=4),
        # odd sizes: rows that are a slice of a wider projection, experts masked out (some rows keep fewer than k),
        # the best expert standing for its group, weights left as they are
        _gate("gate_masked_1001", 1001, 24, 5, "bf16", "softmax", True, groups=3, keep=2, group="max", renorm=False,
              scale=1.0, masked=0.6, pad=8),
        # a prefill chunk of the 256-expert layer, truncated to 70% of the selected mass
        _gate("gate_prefill_512", 512, 256, 8, "f32", "sigmoid", True, groups=8, keep=4, topp=0.7),
        # the widest router: 32 of 1024 experts by softmax, no bias
        _gate("gate_wide_4096", 4096, 1024, 32, "f32", "softmax", False, scale=1.0),
        # the prefill of many prompts at once
        _gate("gate_prefill_65536", 65536, 256, 8, "f32", "sigmoid", True, groups=8, keep=4),
        # one decoded token of one request: one adapter of rank 16 is read, latency counts
        _adapter("adapter_decode_1", 1, 4, 16, "max", 6144, 6144, "bf16", "mixed"),
        # a decode batch of 64 requests with adapters of their own, ranks 4 to 64, some requests without;
        # the activations are the normalised residual stream in fp32
        _adapter("adapter_decode_64", 64, 64, 64, "ragged", 6144, 6144, "f32", "mixed", none=0.1),
        # the down projection's adapter on the int8 codes of h, four requests of a verify batch
        _adapter("adapter_down_256", 256, 24, 32, "ragged", 2048, 6144, "i8", "mixed", none=0.05),
        # a prefill chunk: a few prompts of unequal length, each with its adapter
        _adapter("adapter_prefill_509", 509, 5, 64, "ragged", 6144, 6144, "bf16", "runs"),
        # the prefill of many prompts, the residual stream read and written whole
        _adapter("adapter_prefill_8192", 8192, 16, 64, "ragged", 6144, 6144, "bf16", "runs", none=0.02),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _drawn(rng)
    del case["name"]
    return case


def _drawn(rng):
    if rng.random() < 0.5:
        E = rng.choice([8, 24, 60, 64, 96, 128, 160, 256, 256, 384, 512, 1024])
        groups = rng.choice([g for g in (1, 1, 2, 3, 4, 8, 16, 32) if E % g == 0])
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(32, keep * (E // groups)))
        score = rng.choice(["sigmoid", "softmax"])
        return _gate("", _log_int(rng, 1, (1 << 24) // E), E, k, rng.choice(["f32", "bf16"]), score,
                     rng.random() < 0.7, groups, keep, rng.choice(["top2", "max"]), rng.random() < 0.8,
                     rng.choice([1.0, 2.5]), rng.choice([0.0, 0.0, 0.7]), rng.choice([0.0, 0.0, 0.3, 0.8]),
                     rng.choice([0, 0, 1, 8]))
    T = _log_int(rng, 1, 8192)
    n = _log_int(rng, 1, max(2, min(64, 2 * T, 131072 // T)))
    r_max = rng.choice([8, 16, 32, 64, 64])
    d_in, d_out = 16 * _log_int(rng, 8, 384), 16 * _log_int(rng, 8, 384)
    return _adapter("", T, n, r_max, rng.choice(["max", "ragged"]), d_in, d_out, rng.choice(["f32", "bf16", "i8"]),
                    rng.choice(["mixed", "runs"]), rng.choice([0.0, 0.1, 0.5]), rng.random() < 0.7)


def work(case):
    T = case["T"]
    if case["op"] == "gate":
        E, k, size = case["E"], case["k"], 4 if case["dtype"] == "f32" else 2
        # a score is an exponential, an addition and a division; a bias another addition
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": T * E * 4 + T * k * 2}
    size = {"f32": 4, "bf16": 2, "i8": 1}[case["dtype"]]
    ranks, of = _ranks(case), _adapter_of(case, 0)
    used = sorted(set(of) - {-1})
    rank_rows = sum(ranks[a] for a in of if a >= 0)
    with_adapter = sum(1 for a in of if a >= 0)
    bytes_ = (with_adapter * case["d_in"] * size + T * case["d_out"] * 4 * (2 if case["base"] else 1) +
              2 * sum(ranks[a] for a in used) * (case["d_in"] + case["d_out"]) + 4 * T)
    return {"bytes": bytes_, "flops": 2 * rank_rows * (case["d_in"] + case["d_out"])}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _ranks(case):
    """Rank of each adapter: all r_max, or spread from 4 (or r_max / 2) up to it, odd ones among them."""
    n, r = case["n"], case["r_max"]
    if case["ranks"] == "max":
        return [r] * n
    lo = min(4, r // 2)
    return [r - (a * 7) % (r - lo + 1) for a in range(n)]


def _adapter_of(case, seed):
    """Adapter of each row (-1: none): one request after the other ("runs", as prompts are packed), or every
    row a request's of its own ("mixed", as a decode batch is)."""
    T, n = case["T"], case["n"]
    rng = random.Random(1000003 * seed + T * 31 + n)
    if case["spread"] == "runs":
        cuts = sorted(rng.randint(0, T) for _ in range(n - 1))
        of = [a for a, (b, e) in enumerate(zip([0] + cuts, cuts + [T])) for _ in range(b, e)]
        bare = int(T * case["none"])
        return of[:T - bare] + [-1] * bare
    return [-1 if T > 1 and rng.random() < case["none"] else rng.randrange(n) for _ in range(T)]


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 7919 + case["T"])

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE)

    T, s = case["T"], dict(case)
    if case["op"] == "gate":
        E, k = case["E"], case["k"]
        dtype = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        rows = 1.5 * normal(T, E + case["pad"])
        if case["masked"]:
            rows = rows.masked_fill(torch.rand(T, E + case["pad"], generator=g, device=DEVICE) < case["masked"],
                                    -math.inf)
        s["logits"] = rows.to(dtype)[:, :E]
        s["b"] = 0.02 * (torch.rand(E, generator=g, device=DEVICE) - 0.5) if case["bias"] else None
        if own:
            import expert_ffn_router_b200 as M
            s["cfg"] = M.config(6144, 2048, E, k, routed_scale=case["scale"], topp=case["topp"])
            s["rule"] = M.gate_rule(case["score"], case["groups"], case["keep"], case["group"], case["renorm"])
            s["idx"] = torch.empty(T, k, dtype=torch.int32, device=DEVICE)
            s["w"] = torch.empty(T, k, device=DEVICE)
        return s
    n, r, d_in, d_out = case["n"], case["r_max"], case["d_in"], case["d_out"]
    of = _adapter_of(case, seed)
    s["of"] = torch.tensor(of, dtype=torch.int32, device=DEVICE)
    s["A"] = (normal(n, r, d_in) / math.sqrt(d_in)).to(torch.bfloat16)
    s["B"] = (0.05 * normal(n, d_out, r)).to(torch.bfloat16)
    s["rank"] = torch.tensor(_ranks(case), dtype=torch.int32, device=DEVICE)
    s["scale"] = 0.5 + 1.5 * torch.rand(n, generator=g, device=DEVICE)
    s["base"] = normal(T, d_out) if case["base"] else None
    s["sx"] = None
    if case["dtype"] == "i8":
        x = normal(T, d_in)
        s["sx"] = x.abs().amax(1) / 127
        s["x"] = torch.clamp(torch.round(x / s["sx"][:, None]), -127, 127).to(torch.int8)
    else:
        s["x"] = normal(T, d_in).to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
    if own:
        import expert_ffn_router_b200 as M
        s["adapters"] = M.make_adapters(s["A"], s["B"], s["rank"], s["scale"])
        s["plan"] = M.adapter_plan(n, s["of"])
        s["y"] = torch.empty(T, d_out, device=DEVICE)
    else:
        # each adapter's rows side by side, padded with row T to the longest list (the batch's own plan: a
        # program keeps it for all projections of all layers of a step)
        count = [0] * n
        place = []
        for a in of:
            place.append(count[a] if a >= 0 else 0)
            count[a] += a >= 0
        lists = torch.full((n, max(1, max(count))), T, dtype=torch.int64)
        on = [t for t in range(T) if of[t] >= 0]
        if on:
            lists[torch.tensor([of[t] for t in on]), torch.tensor([place[t] for t in on])] = torch.tensor(on)
        s["lists"] = lists.to(DEVICE)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _plain_gate(s):
    """In 64 bits: selection values lie next to one another, and the order has to be right."""
    lg = s["logits"].double()
    T, E = lg.shape
    k, G, b = s["k"], s["groups"], s["b"]
    fit = ~torch.isnan(lg) & (lg > -math.inf)
    if b is not None:
        fit = fit & (~torch.isnan(b) & (b > -math.inf))
    lg = torch.where(fit, lg, -math.inf)
    if s["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-lg))
    else:
        top = lg.amax(1, keepdim=True)
        e = torch.where(fit, torch.exp(lg - top), 0.0)
        score = torch.where(fit, e / e.sum(1, keepdim=True), 0.0)
    val = torch.where(fit, score + b.double(), -math.inf) if b is not None else lg
    if G > 1:
        by = (score if b is None else score + b.double()).masked_fill(~fit, -math.inf).view(T, G, E // G)
        two = torch.sort(by, dim=2, descending=True)[0][:, :, :2 if s["group"] == "top2" else 1]
        gval = torch.where(two[:, :, 0] > -math.inf, torch.where(two > -math.inf, two, 0.0).sum(2), -math.inf)
        order = torch.sort(gval, dim=1, descending=True, stable=True)[1][:, :s["keep"]]
        stays = torch.zeros(T, G, dtype=torch.bool, device=lg.device).scatter_(1, order, True)
        val = torch.where(stays.repeat_interleave(E // G, 1), val, -math.inf)
    val, idx = torch.sort(val, dim=1, descending=True, stable=True)
    val, idx = val[:, :k], idx[:, :k]
    on = val > -math.inf
    w = torch.where(on, score.gather(1, idx), 0.0)
    if s["topp"]:
        before = torch.cumsum(w, 1) - w
        on = on & ((before < float(torch.tensor(s["topp"])) * w.sum(1, keepdim=True)) |
                   (torch.arange(k, device=w.device) == 0))
        w = torch.where(on, w, 0.0)
    if s["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(on, idx, -1).to(torch.int32), (w * s["scale"]).float()


def _plain_adapter(s):
    """The rows of each adapter gathered, two batched products in 32 bits, and the sums put back in place."""
    x, lists = s["x"].float(), s["lists"]
    T = x.shape[0]
    if s["sx"] is not None:
        x = x * s["sx"][:, None]
    live = torch.arange(s["r_max"], device=x.device) < s["rank"][:, None]
    a = torch.where(live[:, :, None], s["A"].float(), 0.0)
    b = torch.where(live[:, None, :], s["B"].float(), 0.0)
    x = torch.cat([x, torch.zeros_like(x[:1])])
    h = torch.matmul(x[lists], a.transpose(1, 2))
    delta = torch.matmul(h, b.transpose(1, 2)) * s["scale"][:, None, None]
    y = torch.zeros(T + 1, s["d_out"], device=x.device)
    y[lists.reshape(-1)] = delta.reshape(-1, s["d_out"])
    return y[:T] if s["base"] is None else s["base"] + y[:T]


def run(s):
    if own:
        import expert_ffn_router_b200 as M
        if s["op"] == "gate":
            M.moe_gate(s["cfg"], s["rule"], s["logits"], s["b"], s["idx"], s["w"])
            return s["idx"], s["w"]
        M.moe_adapter(s["adapters"], s["plan"], s["x"], s["y"], base=s["base"], sx=s["sx"])
        return s["y"]
    return _plain_gate(s) if s["op"] == "gate" else _plain_adapter(s)


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _exact_gate(s):
    l64, b, k, G = s["logits"].double(), s["b"], s["k"], s["groups"]
    T, E = l64.shape
    out = (l64 != l64) | (l64 == -math.inf)
    if b is not None:
        out |= ((b != b) | (b == -math.inf))[None]
    if s["score"] == "sigmoid":
        p = torch.sigmoid(l64).masked_fill(out, 0.0)
    else:
        p = torch.nan_to_num(torch.softmax(l64.masked_fill(out, -math.inf), 1)).masked_fill(out, 0.0)
    sel = p + b.double()[None] if b is not None else p
    if G > 1:
        part = sel.masked_fill(out, -math.inf).reshape(T, G, -1)
        best, at = part.max(2)
        if s["group"] == "top2":
            second = part.scatter(2, at[:, :, None], -math.inf).amax(2)
            value = best + second.masked_fill(second == -math.inf, 0.0)
        else:
            value = best
        closed = torch.ones(T, G, dtype=torch.bool, device=sel.device)
        for _ in range(s["keep"]):
            g = value.argmax(1, keepdim=True)
            closed.scatter_(1, g, value.gather(1, g) == -math.inf)
            value.scatter_(1, g, -math.inf)
        out = out | closed[:, :, None].expand(T, G, E // G).reshape(T, E)
    sel = (sel if b is not None else l64).masked_fill(out, -math.inf)
    idx = torch.full((T, k), -1, dtype=torch.int64, device=sel.device)
    w = torch.zeros(T, k, dtype=torch.float64, device=sel.device)
    for j in range(k):
        e = sel.argmax(1, keepdim=True)
        there = sel.gather(1, e) > -math.inf
        idx[:, j:j + 1] = torch.where(there, e, -1)
        w[:, j:j + 1] = torch.where(there, p.gather(1, e), 0.0)
        sel.scatter_(1, e, -math.inf)
    if s["topp"]:
        whole, run_sum = w.sum(1) * float(torch.tensor(s["topp"], dtype=torch.float32)), w[:, 0].clone()
        for j in range(1, k):
            drop = ~(run_sum < whole)
            run_sum += w[:, j]
            idx[drop, j] = -1
            w[drop, j] = 0.0
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    return idx.to(torch.int32), w * s["scale"]


def _exact_adapter(s):
    T, d_out = s["x"].shape[0], s["d_out"]
    y = torch.zeros(T, d_out, dtype=torch.float64, device=DEVICE)
    if s["base"] is not None:
        y += s["base"]
    for a, r in enumerate(s["rank"].tolist()):
        rows = torch.nonzero(s["of"] == a)[:, 0]
        if len(rows):
            x = s["x"][rows].double()
            if s["sx"] is not None:
                x *= s["sx"][rows].double()[:, None]
            y[rows] += s["scale"][a].double() * (x @ s["A"][a, :r].double().T) @ s["B"][a, :, :r].double().T
    return y


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_gate(s) if case["op"] == "gate" else _exact_adapter(s)
