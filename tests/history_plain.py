"""The operators of a growing history in 64 bits, from their definitions, and how far a result that holds its sums
in 32 bits may be from them (worst-case rounding bounds, computed from the inputs: see sequence_plain).

Positions: the kernel's argument of cosine and sine is a float32 number of half turns of magnitude 1 at most, rounded
(pi * 2^-25 radians), of a product of three 64-bit factors (3 * 2^-53 of the angle); cosine and sine are within 2
units of the last place of numbers below 1 (2^-22), and scaling, products and sum round four times more.
"""
import math

import torch

from sequence_plain import TINY, U, U32


# ---------------------------------------------------------------- positions
def rotary(x, freqs, positions, interleaved, amplitude, back=False):
    """(y, bound) of x [..., heads, dim] at positions [...]."""
    dtype, half = x.dtype, freqs.numel()
    x = x.double()
    angle = positions.double().unsqueeze(-1) * freqs.double()
    c, s = (angle.cos() * amplitude).unsqueeze(-2), (angle.sin() * (-amplitude if back else amplitude)).unsqueeze(-2)
    at = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    a, b = x[..., at[0]], x[..., at[1]]
    y, err = x.clone(), torch.zeros_like(x)
    y[..., at[0]], y[..., at[1]] = a * c - b * s, b * c + a * s
    unit = math.pi * 2.0**-25 + 2.0**-22 + 6 * U32 + angle.abs().unsqueeze(-2) * 3 * 2.0**-53
    e = abs(amplitude) * (a.abs() + b.abs()) * unit
    err[..., at[0]] = err[..., at[1]] = e
    err[..., : 2 * half] += U[dtype] * y[..., : 2 * half].abs() + TINY
    return y, err


# -------------------------------------------------------------- paged cache
def slots(table_row, page_size, positions):
    """(page, slot) of positions of one entry."""
    return table_row.long()[positions // page_size], positions % page_size


def new_rows(batch, new_len, offsets):
    """Each entry's rows, into packed rows or its own of a padded batch."""
    if offsets is None:
        return [torch.arange(new_len) for _ in range(batch)]
    return [torch.arange(int(offsets[b]), int(offsets[b + 1])) for b in range(batch)]


def keys_of(cache, table_row, page_size, n):
    """The first n keys of an entry, [n, heads, dim]."""
    page, slot = slots(table_row, page_size, torch.arange(n, device=cache.device))
    return cache[page, slot]


# ---------------------------------------------------------------- attention
def seen(queries, keys, window=None, sinks=0):
    """[queries, keys]: which positions see which."""
    q, k = queries[:, None], keys[None]
    ok = k <= q
    if window is not None:
        ok &= (q - k < window) | (k < sinks)
    return ok


def attention(q, k, v, ok, scale, grad=None):
    """One entry: q [lq, hq, d], k and v [lk, hkv, d], ok [lq, lk].  {name: (value, bound)} of o, lse and with grad dq,
    dk, dv."""
    dtype = q.dtype
    up = U[dtype] if dtype == torch.bfloat16 else 0.0   # P and dS on their way into a product
    q, k, v = q.double(), k.double(), v.double()
    lq, hq, d = q.shape
    lk, hkv = k.shape[0], k.shape[1]
    group = hq // hkv
    val = {"o": torch.zeros_like(q), "lse": torch.full((lq, hq), -math.inf, dtype=torch.float64, device=q.device)}
    err = {"o": torch.full_like(q, TINY), "lse": torch.zeros((lq, hq), dtype=torch.float64, device=q.device)}
    if grad is not None:
        grad = grad.double()
        for name, like in (("dq", q), ("dk", k), ("dv", v)):
            val[name], err[name] = torch.zeros_like(like), torch.full_like(like, TINY)
    some = ok.any(1)
    if some.any():
        n = int(ok.sum(1).max())
        for h in range(hq):
            K, V, Q = k[:, h // group], v[:, h // group], q[:, h]
            # what no row sees does not count, whatever it holds
            live = ok.any(0)
            K, V = torch.where(live[:, None], K, 0.0), torch.where(live[:, None], V, 0.0)
            S = scale * Q @ K.T
            eS = (d + 6) * U32 * scale * (Q.abs() @ K.abs().T) + 4 * U32 * S.abs()
            S, eS = S.masked_fill(~ok, -math.inf), eS.masked_fill(~ok, 0.0)
            L = torch.logsumexp(S, -1, keepdim=True)
            P = torch.where(ok, torch.exp(S - torch.where(some[:, None], L, 0.0)), 0.0)
            eP = 2 * eS.amax(-1, keepdim=True) + eS + (n + 12) * U32
            top = S.masked_fill(~ok, 0.0).abs().amax(-1)
            val["lse"][:, h] = L[:, 0]
            err["lse"][:, h] = torch.where(some, eP.amax(-1) * 1.1 + 4 * U32 * (L[:, 0].abs() + top + 1), 0.0)
            O = P @ V
            val["o"][:, h] = O
            eO = (P * (eP * 1.1 + up + n * U32)) @ V.abs()
            err["o"][:, h] += eO + U.get(dtype, 0.0) * (O.abs() + eO)
            if grad is None:
                continue
            G = torch.where(some[:, None], grad[:, h], 0.0)
            Q = torch.where(some[:, None], Q, 0.0)
            eL = torch.where(some, err["lse"][:, h], 0.0)[:, None]
            eP = eP + eL + 4 * U32   # the backward pass has L from the forward's rounded result
            dP = G @ V.T
            edP = (d + 2) * U32 * (G.abs() @ V.abs().T)
            delta = (G * O).sum(-1, keepdim=True)
            edelta = (G.abs() * (err["o"][:, h] + (d + 2) * U32 * O.abs())).sum(-1, keepdim=True)
            dS = P * (dP - delta)
            edS = dS.abs() * (eP * 1.1 + up + 4 * U32) + P * (1 + eP) * (
                edP + edelta + 2 * U32 * (dP.abs() + delta.abs()))
            val["dq"][:, h] = scale * dS @ K
            err["dq"][:, h] += scale * ((edS + (n + 2) * U32 * dS.abs()) @ K.abs())
            r = lq * group
            val["dk"][:, h // group] += scale * dS.T @ Q
            err["dk"][:, h // group] += scale * ((edS + (r + 2) * U32 * dS.abs()).T @ Q.abs())
            val["dv"][:, h // group] += P.T @ G
            err["dv"][:, h // group] += (P * (eP * 1.1 + up + (r + 2) * U32)).T @ G.abs()
    if grad is not None:
        for name in ("dq", "dk", "dv"):
            err[name] += U.get(dtype, 0.0) * (val[name].abs() + err[name])
    return {name: (val[name], err[name]) for name in val}


def self_attention(q, k, v, scale, lens=None, offsets=None, mask=None, window=None, sinks=0, grad=None):
    """{name: (value, bound)} over a batch; positions of no entry and past the lengths give 0 (lse -inf)."""
    names = ("o", "lse") if grad is None else ("o", "lse", "dq", "dk", "dv")
    like = {"o": q, "lse": q[..., 0], "dq": q, "dk": k, "dv": v}
    val = {n: torch.full(like[n].shape, -math.inf if n == "lse" else 0.0, dtype=torch.float64, device=q.device)
           for n in names}
    err = {n: torch.full(like[n].shape, TINY, dtype=torch.float64, device=q.device) for n in names}
    batch = q.shape[0] if offsets is None else len(offsets) - 1
    for b in range(batch):
        if offsets is None:
            at = (b, slice(0, q.shape[1] if lens is None else int(lens[b])))
        else:
            at = (slice(int(offsets[b]), int(offsets[b + 1])),)
        n = q[at].shape[0]
        pos = torch.arange(n, device=q.device)
        ok = seen(pos, pos, window, sinks)
        if mask is not None:
            ok = ok & mask[at].bool()[None]
        if n:
            for name, (x, e) in attention(q[at], k[at], v[at], ok, scale, None if grad is None else grad[at]).items():
                val[name][at], err[name][at] = x, e
    return {n: (val[n], err[n]) for n in names}


def paged_attention(q, k_cache, v_cache, table, lens, scale, offsets=None, causal=True, window=None, sinks=0):
    """{o, lse: (value, bound)}; rows of no entry 0 and -inf."""
    val = {"o": torch.zeros_like(q, dtype=torch.float64),
           "lse": torch.full(q.shape[:-1], -math.inf, dtype=torch.float64, device=q.device)}
    err = {n: torch.full_like(x, TINY) for n, x in val.items()}
    batch, page_size = table.shape[0], k_cache.shape[1]
    for b, rows in enumerate(new_rows(batch, q.shape[1], offsets)):
        at = (b, rows) if offsets is None else (rows,)
        n, total = len(rows), int(lens[b])
        if not n or not total:
            continue
        keys = torch.arange(total, device=q.device)
        queries = total - n + torch.arange(n, device=q.device)
        ok = seen(queries, keys, window, sinks) if causal else torch.ones(n, total, dtype=torch.bool, device=q.device)
        got = attention(q[at], keys_of(k_cache, table[b], page_size, total),
                        keys_of(v_cache, table[b], page_size, total), ok, scale)
        for name, (x, e) in got.items():
            val[name][at], err[name][at] = x, e
    return {n: (val[n], err[n]) for n in val}
