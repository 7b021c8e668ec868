"""The selection rule of moe_gate and the adapters' sum of moe_adapter, in 64
bits on the host, row after row: what the GPU tests compare with."""
import numpy as np


def gate_row(lg, bias, k, score="sigmoid", groups=0, keep=0, value="top2", renorm=True, scale=2.5, topp=0.0):
    """lg [E] float64 -> (idx int32 [k], w float64 [k])."""
    E = len(lg)
    fit = [e for e in range(E) if lg[e] > -np.inf and (bias is None or bias[e] > -np.inf)]
    s = np.zeros(E)
    with np.errstate(over="ignore"):
        if score == "sigmoid":
            for e in fit:
                s[e] = 1.0 / (1.0 + np.exp(-lg[e]))
        elif fit:
            m = max(lg[e] for e in fit)
            ex = {e: 1.0 if lg[e] == m else np.exp(lg[e] - m) for e in fit}
            z = sum(ex.values())
            for e in fit:
                s[e] = ex[e] / z
    val = {e: (s[e] + float(bias[e]) if bias is not None else lg[e]) for e in fit}
    if groups > 1:
        gs = E // groups
        gval = {}
        for g in range(groups):
            best = sorted((s[e] + (float(bias[e]) if bias is not None else 0.0) for e in fit if e // gs == g),
                          reverse=True)
            if best:
                gval[g] = best[0] + (best[1] if value == "top2" and len(best) > 1 else 0.0)
        stay = set(sorted(gval, key=lambda g: (-gval[g], g))[:keep])
        val = {e: v for e, v in val.items() if e // gs in stay}
    order = sorted(val, key=lambda e: (-val[e], e))[:k]
    idx, w = np.full(k, -1, np.int32), np.zeros(k)
    whole, before = float(np.float32(topp)) * sum(s[e] for e in order), 0.0
    for j, e in enumerate(order):
        if 0.0 < topp < 1.0 and j > 0 and not before < whole:
            break
        idx[j], w[j] = e, s[e]
        before += s[e]
    total = w.sum()
    if renorm:
        w = w / total if total > 0 else np.zeros(k)
    return idx, w * float(np.float32(scale))


def gate(logits, bias, k, **kw):
    """logits: torch tensor [T][E]; bias torch tensor or None."""
    lg = logits.detach().double().cpu().numpy()
    b = None if bias is None else bias.detach().double().cpu().numpy()
    rows = [gate_row(r, b, k, **kw) for r in lg]
    return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])


def gate_weight_rtol(E, k, widest):
    """Relative error of a float32 weight, counted in roundings of 2^-24 (a
    correctly rounded operation: 1; expf: 4, its documented 2 ulp).  Sigmoid:
    expf 4, the addition and the division 1 each.  Softmax: the subtraction
    l - m moves the exponent by half an ulp of at most `widest`, that is
    `widest` roundings of the result; expf 4; its sum over E experts at most
    E / 32 + 5 additions deep; the division 1.  Then k additions of the
    normaliser, a division and the scale."""
    return (max(6, 2 * (widest + 4) + E / 32 + 5 + 1) + k + 2) * 2.0 ** -24


def adapter(x, sx, of, a, b, rank, scale, base):
    """All torch tensors (rank a list): y in float64 [T][d_out], and a bound of
    a float32 evaluation's error, element by element.

    The bound: products of bf16 values (and of the parts of a float32 one) are
    exact, so only additions round.  A sum of n terms taken at most n / 8 + 16
    additions deep (groups of 8 or more added at once, the groups' sums one
    after the other), each off by at most 2^-23 (a truncating adder), is off by
    (n / 8 + 16) * 2^-23 times the sum of the terms' magnitudes.  It holds for
    h = A x, then for B h (with the error that h carries in), and the scale,
    the code's scale and the base add a rounding each."""
    T, d_out = x.shape[0], b.shape[1]
    xd, ad, bd = x.double(), a.double(), b.double()
    if sx is not None:
        xd = xd * sx.double()[:, None]
    import torch
    y = torch.zeros(T, d_out, dtype=torch.float64, device=x.device)
    err = torch.zeros_like(y)
    u = 2.0 ** -23
    for i, r in enumerate(rank):
        rows = torch.nonzero(of == i)[:, 0]
        if len(rows) == 0 or r == 0:
            continue
        A, B = ad[i, :r], bd[i, :, :r]
        s = float(scale[i]) if scale is not None else 1.0
        h, hm = xd[rows] @ A.T, xd[rows].abs() @ A.abs().T
        h_err = (x.shape[1] / 8 + 16 + 2) * u * hm
        y[rows] += s * (h @ B.T)
        err[rows] += abs(s) * (h_err @ B.abs().T + (r / 8 + 16 + 2) * u * (h.abs() @ B.abs().T))
    if base is not None:
        y += base.double()
    err += 2 * u * y.abs()
    return y, err
