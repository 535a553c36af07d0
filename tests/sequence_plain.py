"""The sequence operators in 64 bits on the CPU, from their definitions, and
how far a result that holds its sums in 32 bits may be from them.

The bounds are worst-case rounding bounds, computed from the inputs before a
kernel is looked at: U32 is float32's unit roundoff, a sum of n terms is within
n * U32 times the sum of their magnitudes, and a value that is rounded to the
output's type moves by at most that type's unit roundoff.  Nothing here is
shared with the library or with perf/operators.py.
"""
import math

import torch

U32 = 2.0**-24
U = {torch.float32: U32, torch.bfloat16: 2.0**-8}  # half an ulp, relative, and the tie
TINY = 1e-30


def within(got, want, bound, what=""):
    """Every element of `got` is within `bound` of `want`; infinities and NaN sit in the same places."""
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    finite = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    assert torch.equal(got[~finite & ~torch.isnan(want)], want[~finite & ~torch.isnan(want)]), what
    off = (got - want).abs()[finite] - bound.expand_as(want)[finite]
    assert off.numel() == 0 or off.max() <= 0, (what, "over the bound by", off.max().item(),
                                                "bound", bound.max().item())


# ---------------------------------------------------------------- embedding
def embed(tokens, weight, scale):
    rows = weight.shape[0]
    t = tokens.reshape(-1)
    ok = (t >= 0) & (t < rows)
    out = weight.double()[t.clamp(0, rows - 1)] * scale
    out[~ok] = 0
    return out.reshape(*tokens.shape, weight.shape[1])


def embed_backward(tokens, grad, rows, scale, out_dtype):
    """(dW, bound)."""
    t = tokens.reshape(-1)
    ok = (t >= 0) & (t < rows)
    g = grad.double().reshape(-1, grad.shape[-1])[ok]
    t = t[ok]
    dw = torch.zeros(rows, grad.shape[-1], dtype=torch.float64).index_add_(0, t, g) * scale
    mag = torch.zeros(rows, grad.shape[-1], dtype=torch.float64).index_add_(0, t, g.abs()) * abs(scale)
    count = torch.zeros(rows, dtype=torch.float64).index_add_(0, t, torch.ones_like(t, dtype=torch.float64))
    return dw, (count[:, None] + 2) * U32 * mag + U[out_dtype] * dw.abs() + TINY


# --------------------------------------------------------------- layer norm
def layer_norm(x, w, b, eps, dtype):
    """y, mean, rstd and their bounds."""
    x, d = x.double(), x.shape[-1]
    w = torch.ones(d, dtype=torch.float64) if w is None else w.double()
    b = torch.zeros(d, dtype=torch.float64) if b is None else b.double()
    mean = x.mean(-1, keepdim=True)
    xc = x - mean
    var = (xc * xc).mean(-1, keepdim=True)
    rstd = 1 / (var + eps).sqrt()
    n = d + 4
    e_mean = n * U32 * x.abs().mean(-1, keepdim=True)
    e_xc = e_mean + U32 * (xc.abs() + e_mean)
    e_var = (2 * xc.abs() * e_xc + e_xc * e_xc).mean(-1, keepdim=True) + n * U32 * var
    rel = e_var / (var + eps) / 2 * 1.1 + 4 * U32      # of rstd, to first order and a margin for the second
    xh = xc * rstd
    e_xh = e_xc * rstd * (1 + rel) + xh.abs() * (rel + 2 * U32)
    y = xh * w + b
    e_y = e_xh * w.abs() + 2 * U32 * ((xh * w).abs() + b.abs()) + U[dtype] * y.abs() + TINY
    return {"y": (y, e_y), "mean": (mean[..., 0], e_mean[..., 0] + TINY),
            "rstd": (rstd[..., 0], rstd[..., 0] * rel[..., 0]), "xh": (xh, e_xh), "w": w}


def layer_norm_backward(g, x, w, eps, dtype, w_dtype):
    f = layer_norm(x, w, None, eps, dtype)
    (xh, e_xh), (rstd, e_rstd), w, d = f["xh"], f["rstd"], f["w"], x.shape[-1]
    rstd, rel = rstd[..., None], (e_rstd / f["rstd"][0])[..., None]
    g, n = g.double(), d + 4
    a = g * w
    m1, m2 = a.mean(-1, keepdim=True), (a * xh).mean(-1, keepdim=True)
    e_m1 = (n + 1) * U32 * a.abs().mean(-1, keepdim=True)
    e_m2 = (n + 2) * U32 * (a * xh).abs().mean(-1, keepdim=True) + (a.abs() * e_xh).mean(-1, keepdim=True)
    inner = a - m1 - xh * m2
    mags = a.abs() + m1.abs() + (xh * m2).abs()
    e_inner = e_m1 + xh.abs() * e_m2 + e_xh * (m2.abs() + e_m2) + 4 * U32 * mags
    dx = rstd * inner
    e_dx = rstd * e_inner * (1 + rel) + dx.abs() * (rel + 2 * U32) + U[dtype] * dx.abs() + TINY
    rows = x.numel() // d
    flat = lambda t: t.reshape(-1, d).sum(0)  # noqa: E731
    dw, db = flat(g * xh), flat(g)
    e_dw = (rows + 4) * U32 * flat((g * xh).abs()) + flat(g.abs() * e_xh) + U[w_dtype] * dw.abs() + TINY
    e_db = (rows + 4) * U32 * flat(g.abs()) + U[w_dtype] * db.abs() + TINY
    return {"dx": (dx, e_dx), "dw": (dw, e_dw), "db": (db, e_db)}


# ---------------------------------------------------------- cross attention
def kept_keys(k, lens=None, offsets=None, mask=None):
    """Per batch entry, the row numbers (into k[b] or packed k) of its keys that count."""
    out = []
    batch = k.shape[0] if offsets is None else len(offsets) - 1
    for b in range(batch):
        if offsets is None:
            n = k.shape[1] if lens is None else int(lens[b])
            rows = torch.arange(n)
            ok = mask[b, :n].bool() if mask is not None else torch.ones(n, dtype=torch.bool)
        else:
            rows = torch.arange(int(offsets[b]), int(offsets[b + 1]))
            ok = mask[rows].bool() if mask is not None else torch.ones(len(rows), dtype=torch.bool)
        out.append(rows[ok])
    return out


def attention(q, k, v, scale, kept, packed, grad=None):
    """Values and bounds of o, lse (and dq, dk, dv with grad): {name: (value, bound)}."""
    dtype = q.dtype
    up = U[dtype] if dtype == torch.bfloat16 else 0.0   # P and dS on their way into a product
    q, k, v = q.double(), k.double(), v.double()
    batch, lq, hq, d = q.shape
    hkv = k.shape[-2]
    group = hq // hkv
    val = {"o": torch.zeros_like(q), "lse": torch.full((batch, lq, hq), -math.inf, dtype=torch.float64)}
    err = {"o": torch.full_like(q, TINY), "lse": torch.zeros(batch, lq, hq, dtype=torch.float64)}
    if grad is not None:
        grad = grad.double()
        for name, like in (("dq", q), ("dk", k), ("dv", v)):
            val[name], err[name] = torch.zeros_like(like), torch.full_like(like, TINY)
    for b in range(batch):
        rows = kept[b]
        n = len(rows)
        if n == 0:
            continue
        kb, vb = (k, v) if packed else (k[b], v[b])
        for h in range(hq):
            at = (rows, h // group)
            K, V, Q = kb[at], vb[at], q[b, :, h]
            S = scale * Q @ K.T
            eS = (d + 6) * U32 * scale * (Q.abs() @ K.abs().T) + 4 * U32 * S.abs()
            L = torch.logsumexp(S, -1, keepdim=True)
            P = torch.exp(S - L)
            # every weight's relative error: its score's, the largest's, the exponential's, the sum's
            eP = 2 * eS.amax(-1, keepdim=True) + eS + (n + 12) * U32
            val["lse"][b, :, h] = L[:, 0]
            err["lse"][b, :, h] = eP.amax(-1) * 1.1 + 4 * U32 * (L[:, 0].abs() + S.abs().amax(-1) + 1)
            O = P @ V
            val["o"][b, :, h] = O
            eO = (P * (eP * 1.1 + up + n * U32)) @ V.abs()
            err["o"][b, :, h] += eO + U[dtype] * (O.abs() + eO)
            if grad is None:
                continue
            G = grad[b, :, h]
            # the backward pass has L from the forward's rounded result
            eP = eP + err["lse"][b, :, h][:, None] + 4 * U32
            dP = G @ V.T
            edP = (d + 2) * U32 * (G.abs() @ V.abs().T)
            delta = (G * O).sum(-1, keepdim=True)
            edelta = (G.abs() * (err["o"][b, :, h] + (d + 2) * U32 * O.abs())).sum(-1, keepdim=True)
            dS = P * (dP - delta)
            edS = dS.abs() * (eP * 1.1 + up + 4 * U32) + P * (1 + eP) * (edP + edelta + 2 * U32 * (dP.abs() + delta.abs()))
            val["dq"][b, :, h] = scale * dS @ K
            err["dq"][b, :, h] += scale * ((edS + (n + 2) * U32 * dS.abs()) @ K.abs())
            r = lq * group
            for name, value, bound in (
                    ("dk", scale * dS.T @ Q, scale * ((edS + (r + 2) * U32 * dS.abs()).T @ Q.abs())),
                    ("dv", P.T @ G, (P * (eP * 1.1 + up + (r + 2) * U32)).T @ G.abs())):
                into, ei = (val[name], err[name]) if packed else (val[name][b], err[name][b])
                into[at] += value
                ei[at] += bound
    if grad is not None:
        for name in ("dq", "dk", "dv"):
            err[name] += U[dtype] * (val[name].abs() + err[name])
    return {name: (val[name], err[name]) for name in val}
