"""What is measured of the operators of a growing history: positions by rotation, the paged cache of keys and
values with its append, attention of new events over that cache, and causal self attention with a sliding window
and first events that stay visible, with its backward pass.

``run`` is one pass as a user's program makes it: with ``own`` false in plain torch operations held in 32 bits (the
angles in 64), with ``own`` true through ``dynamic_embedding_tables_amd.sequence``.  ``exact`` gives the same
outputs from the definitions in 64 bits.  Sizes follow the behaviour-sequence workload of this repository (2048
samples of 1000 ids, dim 128 as 4 heads of 32, bfloat16), its lifelong histories of 8192, and go down to single
events.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the newest event of 32 users, far into their histories
        {"name": "rotary_serve_f32", "op": "rotary_fwd", "b": 32, "l": 1, "heads": 4, "d": 32, "rot": 32,
         "pairs": "halves", "far": 1000000, "factor": 1.0, "dtype": "f32"},
        # a dense model's odd heads, neighbours as pairs, part of the head, scaled for longer histories; both passes
        {"name": "rotary_train_odd_f32", "op": "rotary_train", "b": 61, "l": 777, "heads": 6, "d": 40, "rot": 24,
         "pairs": "neighbours", "far": 0, "factor": 8.0, "dtype": "f32"},
        # every position of the training batch, both passes
        {"name": "rotary_train_batch_bf16", "op": "rotary_train", "b": 2048, "l": 1000, "heads": 4, "d": 32,
         "rot": 32, "pairs": "halves", "far": 0, "factor": 1.0, "dtype": "bf16"},
        # serving: one new event for each of 64 users with lifelong histories
        {"name": "append_one_bf16", "op": "append", "b": 64, "new": 1, "lk": 8192, "page": 64, "hq": 16, "hkv": 4,
         "d": 128, "rot": 128, "pairs": "halves", "factor": 1.0, "dtype": "bf16", "packed": False},
        # filling the cache: whole histories of 2048 users, packed as the table's gather returns them
        {"name": "append_fill_bf16", "op": "append", "b": 2048, "new": 1000, "lk": 1000, "page": 64, "hq": 4,
         "hkv": 4, "d": 32, "rot": 32, "pairs": "halves", "factor": 1.0, "dtype": "bf16", "packed": True},
        # serving: one event a user over short histories
        {"name": "paged_one_short_f32", "op": "paged", "b": 4, "new": 1, "lk": 200, "page": 16, "hq": 4, "hkv": 4,
         "d": 32, "causal": True, "window": 0, "sinks": 0, "dtype": "f32", "packed": False},
        # serving: one event a user over lifelong histories, four query heads to a key head
        {"name": "paged_one_long_bf16", "op": "paged", "b": 64, "new": 1, "lk": 8192, "page": 64, "hq": 16, "hkv": 4,
         "d": 128, "causal": True, "window": 0, "sinks": 0, "dtype": "bf16", "packed": False},
        # catching up: up to 512 new events a user join a lifelong history in one pass
        {"name": "paged_chunk_bf16", "op": "paged", "b": 32, "new": 512, "lk": 8192, "page": 64, "hq": 16, "hkv": 4,
         "d": 128, "causal": True, "window": 0, "sinks": 0, "dtype": "bf16", "packed": True},
        # ranking in 32 bits: candidates read the cached history, odd pages and head size
        {"name": "paged_rank_odd_f32", "op": "paged", "b": 33, "new": 50, "lk": 999, "page": 24, "hq": 6, "hkv": 2,
         "d": 40, "causal": False, "window": 0, "sinks": 0, "dtype": "f32", "packed": False},
        # the whole batch's histories forward, as the table's gather packs them
        {"name": "window_fwd_packed_bf16", "op": "window_fwd", "b": 512, "l": 1000, "hq": 4, "hkv": 4, "d": 32,
         "window": 128, "sinks": 4, "dtype": "bf16", "kv": "packed"},
        # training on long histories, both passes
        {"name": "window_train_bf16", "op": "window_train", "b": 32, "l": 4096, "hq": 8, "hkv": 8, "d": 64,
         "window": 512, "sinks": 4, "dtype": "bf16", "kv": "lens"},
        # training in 32 bits: odd lengths and head size, shared key heads, a mask with holes
        {"name": "window_train_odd_f32", "op": "window_train", "b": 9, "l": 777, "hq": 6, "hkv": 2, "d": 40,
         "window": 100, "sinks": 3, "dtype": "f32", "kv": "mask"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary_fwd", "rotary_train", "append_one", "append", "paged_one", "paged", "window_fwd",
                     "window_train"])
    dtype = rng.choice(["f32", "bf16"])
    d = rng.choice([16, 32, 64, 128, 2 * rng.randint(9, 60)])
    rot = {"rot": rng.choice([d, d, 2 * rng.randint(1, d // 2)]), "pairs": rng.choice(["halves", "neighbours"]),
           "factor": rng.choice([1.0, 4.0])}
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 1, 2, 4])
    if op.startswith("rotary"):
        heads = rng.choice([1, 4, 6, 20])
        n = _log(rng, 1, 120_000_000 // (heads * d))
        l = min(n, _log(rng, 1, 2000))
        return {"op": op, "b": max(1, n // l), "l": l, "heads": heads, "d": d, **rot, "far": rng.choice([0, 1000000]),
                "dtype": dtype}
    if op.startswith("append"):
        new, lk = (rng.choice([1, 1, 3]), _log(rng, 20, 8192)) if op == "append_one" else (_log(rng, 4, 1000), 0)
        lk = max(lk, new + _log(rng, 1, 1000))
        b = _log(rng, 1, max(1, min(1024, 2**27 // (lk * hkv * d))))
        return {"op": "append", "b": b, "new": new, "lk": lk, "page": rng.choice([16, 64, 128, rng.randint(5, 70)]),
                "hq": hq, "hkv": hkv, "d": d, **rot, "dtype": dtype, "packed": rng.random() < 0.5}
    if op.startswith("paged"):
        window, sinks = rng.choice([(0, 0), (0, 0), (_log(rng, 1, 1000), rng.choice([0, 4]))])
        new = rng.choice([1, 1, 2, 5]) if op == "paged_one" else _log(rng, 6, 600)
        lk = new + (_log(rng, 20, 8000) if op == "paged_one" else _log(rng, 16, 4000))
        most = (2**33 if dtype == "bf16" else 2**31) // (new * lk * hq * d)
        b = _log(rng, 1, max(1, min(512 if op == "paged_one" else 128, most, 2**27 // (lk * hkv * d))))
        causal = rng.random() < 0.75 or window > 0
        return {"op": "paged", "b": b, "new": new, "lk": lk, "page": rng.choice([16, 64, 128, rng.randint(5, 70)]),
                "hq": hq, "hkv": hkv, "d": d, "causal": causal, "window": window, "sinks": sinks, "dtype": dtype,
                "packed": rng.random() < 0.5}
    l = _log(rng, 8, 3000)
    window = rng.choice([0, _log(rng, 1, 1000)])
    most = (2**33 if dtype == "bf16" else 2**31) // (l * l * hq * d)
    b = _log(rng, 1, max(1, min(256, most)))
    return {"op": op, "b": b, "l": l, "hq": hq, "hkv": hkv, "d": d, "window": window,
            "sinks": rng.choice([0, 4, rng.randint(0, 100)]) if window else 0, "dtype": dtype,
            "kv": rng.choice(["lens", "packed", "mask"])}


# ------------------------------------------------------------------ inputs
def _ramp(b, most, least=0):
    """Lengths of a batch from `least` to `most`, the same multiset for every seed."""
    return [most] if b == 1 else [least + ((most - least) * i) // (b - 1) for i in range(b)]


def _new_and_cached(case):
    """New events and events of the cache before them, entry by entry (their order is the seed's)."""
    if case["op"] == "paged" and not case["causal"]:  # candidates: not part of the history
        return [case["new"]] * case["b"], _ramp(case["b"], case["lk"])
    new = _ramp(case["b"], case["new"], 1 if case["new"] < 8 else 0) if case["packed"] else [case["new"]] * case["b"]
    return new, _ramp(case["b"], case["lk"] - case["new"])


def _frequencies(case):
    """Radians a position for each pair; with a factor, what turns less than once in 1000 positions turns that
    much slower, what turns more than four times as before, and a line in between."""
    rot = case["rot"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    if case["factor"] == 1.0:
        return f
    keep = ((1000 * f / (2 * math.pi) - 1) / 3).clamp(0, 1)
    return f * (keep + (1 - keep) / case["factor"])


def _offsets(counts):
    off = torch.zeros(counts.numel() + 1, dtype=torch.int32, device="cuda")
    off[1:] = counts.cumsum(0)
    return off


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", dtype=dt, generator=gen)

    def shuffled(lens):
        t = torch.tensor(lens, dtype=torch.int32, device="cuda")
        return t[torch.randperm(t.numel(), device="cuda", generator=gen)].contiguous()

    op, b, d = case["op"], case["b"], case["d"]
    s = {"op": op, "dtype": dt, "d": d, "neighbours": case.get("pairs") == "neighbours", "amplitude": 1.0}
    if "rot" in case:
        s["freqs"] = _frequencies(case)
        s["amplitude"] = 1.0 if case["factor"] == 1.0 else 1 + 0.1 * math.log(case["factor"])
    if op.startswith("rotary"):
        l, heads = case["l"], case["heads"]
        first = torch.randint(0, case["far"] + 1, (b, 1), device="cuda", generator=gen)
        s["x"] = normal(b, l, heads, d)
        s["positions"] = (first + torch.arange(l, device="cuda")).contiguous()
        if op == "rotary_train":
            s["grad"] = normal(b, l, heads, d)
        return s
    hq, hkv = case["hq"], case["hkv"]
    if op.startswith("window"):
        l = case["l"]
        lens = shuffled(_ramp(b, l))
        s.update(l=l, window=case["window"] or None, sinks=case["sinks"], lens=None, offsets=None, mask=None)
        if case["kv"] == "packed":
            n = sum(_ramp(b, l))
            s.update(q=normal(n, hq, d), k=normal(n, hkv, d), v=normal(n, hkv, d), offsets=_offsets(lens))
        else:
            s.update(q=normal(b, l, hq, d), k=normal(b, l, hkv, d), v=normal(b, l, hkv, d), lens=lens)
            if case["kv"] == "mask":  # events that do not count
                s["mask"] = torch.rand(b, l, device="cuda", generator=gen) < 0.9
        if op == "window_train":
            s["grad"] = torch.randn(s["q"].shape, device="cuda", dtype=dt, generator=gen)
        return s
    # a cache whose pages lie in any order, some of them nobody's
    page, width = case["page"], -(-case["lk"] // case["page"])
    pages = b * width + 3
    new, cached = _new_and_cached(case)
    n = sum(new)
    new, cached = shuffled(new), shuffled(cached)
    s["page_table"] = torch.randperm(pages, device="cuda", generator=gen)[: b * width].view(b, width).int()
    s["k_cache"], s["v_cache"] = normal(pages, page, hkv, d), normal(pages, page, hkv, d)
    s["kv_lens"] = (cached if op == "paged" and not case["causal"] else cached + new).int()
    s["offsets"] = _offsets(new) if case["packed"] else None
    s["new"] = case["new"]
    lead = (n,) if case["packed"] else (b, case["new"])
    s["q"] = normal(*lead, hq, d)
    if op == "append":
        s["k"], s["v"] = normal(*lead, hkv, d), normal(*lead, hkv, d)
    else:
        s.update(causal=case["causal"], window=case["window"] or None, sinks=case["sinks"])
    return s


def run(state):
    return (_run_own if own else _run_plain)(state)


# ------------------------------------------------------------------ the framework's calls
def _run_own(s):
    from dynamic_embedding_tables_amd import sequence
    op = s["op"]
    turn = {"interleaved": s["neighbours"], "amplitude": s["amplitude"]}
    if op.startswith("rotary"):
        y = sequence.rotary(s["x"], s["freqs"], s["positions"], **turn)
        if op == "rotary_fwd":
            return y
        return {"y": y, "dx": sequence.rotary_backward(s["grad"], s["freqs"], s["positions"], **turn)}
    if op == "append":
        q = sequence.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"], q=s["q"],
                                  q_offsets=s["offsets"], freqs=s["freqs"], **turn)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "paged":
        return sequence.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["kv_lens"],
                                        q_offsets=s["offsets"], max_q_len=s["new"] if s["offsets"] is not None else None,
                                        causal=s["causal"], window=s["window"], sinks=s["sinks"])
    how = {"lens": s["lens"], "offsets": s["offsets"], "kv_mask": s["mask"], "window": s["window"],
           "sinks": s["sinks"], "max_len": s["l"] if s["offsets"] is not None else None}
    if op == "window_fwd":
        return sequence.self_attention(s["q"], s["k"], s["v"], **how)
    o, lse = sequence.self_attention(s["q"], s["k"], s["v"], return_lse=True, **how)
    dq, dk, dv = sequence.self_attention_backward(s["grad"], s["q"], s["k"], s["v"], o, lse, **how)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


# ------------------------------------------------------------------ plain forms, in 32 bits
def _turned(x, positions, s, sign):
    """x [rows..., heads, d] turned by sign * position * frequency, the rest of each head as it is."""
    angle = positions.double()[..., None] * s["freqs"]
    c = (angle.cos() * s["amplitude"]).float()[..., None, :]
    n = (angle.sin() * (sign * s["amplitude"])).float()[..., None, :]
    rot = 2 * s["freqs"].numel()
    x = x.float()
    head, rest = x[..., :rot], x[..., rot:]
    if s["neighbours"]:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        head = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([head, rest], -1).to(s["dtype"])


def _entries(offsets, n):
    """Each packed row's entry and its place there."""
    row = torch.arange(n, device=offsets.device)
    entry = torch.searchsorted(offsets[1:].long().contiguous(), row, right=True)
    return entry, row - offsets.long()[entry]


def _run_plain(s):
    op = s["op"]
    if op.startswith("rotary"):
        y = _turned(s["x"], s["positions"], s, 1.0)
        return y if op == "rotary_fwd" else {"y": y, "dx": _turned(s["grad"], s["positions"], s, -1.0)}
    if op == "append":
        return _append_plain(s)
    return _paged_plain(s) if op == "paged" else _window_plain(s)


def _append_plain(s):
    lens, table, page = s["kv_lens"].long(), s["page_table"].long(), s["k_cache"].shape[1]
    if s["offsets"] is not None:
        entry, place = _entries(s["offsets"], s["k"].shape[0])
        new = (s["offsets"][1:] - s["offsets"][:-1]).long()
        pos = (lens - new)[entry] + place
    else:
        pos = (lens - s["new"])[:, None] + torch.arange(s["new"], device=lens.device)
        entry = torch.arange(lens.numel(), device=lens.device)[:, None].expand_as(pos)
    at = (table[entry, pos // page], pos % page)
    s["k_cache"][at] = _turned(s["k"], pos, s, 1.0)
    s["v_cache"][at] = s["v"]
    return {"q": _turned(s["q"], pos, s, 1.0), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _seen(query, key, window, sinks):
    """Whether each key counts for each query, by their positions."""
    near = key <= query
    return near if window is None else near & ((query - key < window) | (key < sinks))


def _softmax_product(q, k, v, gone, scale):
    """q [b, lq, hq, d], k and v [b, lk, hkv, d], gone [b, lq, lk]: (out, lse, weights), the last two by key head."""
    b, lq, hq, d = q.shape
    hkv, lk = k.shape[2], k.shape[1]
    q, k, v = _by_key_head(q, hkv), _by_key_head(k, hkv), _by_key_head(v, hkv)
    gone = gone[:, None, :, None].expand(b, hkv, lq, hq // hkv, lk).reshape(b * hkv, -1, lk)
    scores = (torch.bmm(q, k.transpose(1, 2)) * scale).masked_fill_(gone, -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1, total)
    return torch.bmm(p, v), top + total.log(), p


def _by_key_head(t, hkv):  # [b, l, heads, d] -> [b * hkv, l * (heads / hkv), d]
    b, l, heads, d = t.shape
    return t.reshape(b, l, hkv, heads // hkv, d).transpose(1, 2).reshape(b * hkv, -1, d)


def _by_row(t, b, l, heads):  # and back
    return t.reshape(b, -1, l, heads // (t.shape[0] // b), t.shape[-1]).transpose(1, 2).reshape(b, l, heads, -1)


def _paged_plain(s):
    lens, table = s["kv_lens"].long(), s["page_table"].long()
    b = lens.numel()
    keep = torch.arange(table.shape[1] * s["k_cache"].shape[1], device=lens.device) < lens[:, None]
    k, v = (torch.where(keep[:, :, None, None], c[table].flatten(1, 2), 0).float()
            for c in (s["k_cache"], s["v_cache"]))
    q, new = s["q"].float(), s["new"]
    count = torch.full_like(lens, new)
    if s["offsets"] is not None:
        entry, place = _entries(s["offsets"], q.shape[0])
        count = (s["offsets"][1:] - s["offsets"][:-1]).long()
        q = torch.zeros(b, new, *q.shape[1:], device=q.device).index_put((entry, place), q)
    key = torch.arange(k.shape[1], device=lens.device)
    query = (lens - count)[:, None] + torch.arange(new, device=lens.device)
    seen = keep[:, None, :].expand(b, new, -1)
    if s["causal"]:
        seen = seen & _seen(query[:, :, None], key, s["window"], s["sinks"])
    out = _by_row(_softmax_product(q, k, v, ~seen, 1 / math.sqrt(s["d"]))[0], b, new, q.shape[2])
    return (out if s["offsets"] is None else out[entry, place]).to(s["dtype"])


def _window_plain(s):
    dt, l, scale = s["dtype"], s["l"], 1 / math.sqrt(s["d"])
    train = s["op"] == "window_train"
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    g = s["grad"].float() if train else None
    hq, hkv = q.shape[-2], k.shape[-2]
    lens = s["lens"].long() if s["offsets"] is None else (s["offsets"][1:] - s["offsets"][:-1]).long()
    b = lens.numel()
    pos = torch.arange(l, device=q.device)
    keep = pos < lens[:, None]
    if s["offsets"] is not None:
        entry, place = _entries(s["offsets"], q.shape[0])
        at = torch.where(keep, s["offsets"][:-1].long()[:, None] + pos, 0)
        q, k, v = q[at], k[at], v[at]
        g = g[at] if train else None
    live = keep[:, :, None]  # rows past the length see nothing
    if s["mask"] is not None:
        keep = keep & s["mask"]
    k, v = (torch.where(keep[:, :, None, None], t, 0) for t in (k, v))
    seen = live & keep[:, None, :] & _seen(pos[:, None], pos, s["window"], s["sinks"])
    o, lse, p = _softmax_product(q, k, v, ~seen, scale)

    def rows(t, heads):
        t = _by_row(t, b, l, heads)
        return t if s["offsets"] is None else t[entry, place]

    if not train:
        return rows(o, hq).to(dt)
    q, g, k, v = _by_key_head(q, hkv), _by_key_head(g, hkv), _by_key_head(k, hkv), _by_key_head(v, hkv)
    dv = torch.bmm(p.transpose(1, 2), g)
    ds = p * (torch.bmm(g, v.transpose(1, 2)) - (g * o).sum(-1, keepdim=True)) * scale
    dq, dk = torch.bmm(ds, k), torch.bmm(ds.transpose(1, 2), q)
    return {"o": rows(o, hq).to(dt), "lse": rows(lse, hq)[..., 0].contiguous(), "dq": rows(dq, hq).to(dt),
            "dk": rows(dk, hkv).contiguous().to(dt), "dv": rows(dv, hkv).contiguous().to(dt)}


# ------------------------------------------------------------------ the definitions, in 64 bits
def _rotation(case, s, x, positions, back=False):
    """Every pair as a complex number, times amplitude e^(i position frequency); to turn back, its conjugate."""
    half = case["rot"] // 2
    out = x.double().clone()
    z = torch.polar(torch.full_like(s["freqs"], s["amplitude"]), s["freqs"] * 0)
    angle = positions.double().unsqueeze(-1) * s["freqs"]
    z = z * torch.complex(torch.cos(angle), torch.sin(-angle if back else angle))
    first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if case["pairs"] == "neighbours" else (
        slice(0, half), slice(half, 2 * half))
    w = torch.complex(out[..., first].contiguous(), out[..., second].contiguous()) * z.unsqueeze(-2)
    out[..., first], out[..., second] = w.real, w.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("rotary"):
        y = _rotation(case, s, s["x"], s["positions"])
        return y if op == "rotary_fwd" else {"y": y, "dx": _rotation(case, s, s["grad"], s["positions"], back=True)}
    if op == "append":
        return _append_exact(case, s)
    return _paged_exact(case, s) if op == "paged" else _window_exact(case, s)


def _append_exact(case, s):
    kc, vc, q = s["k_cache"].double(), s["v_cache"].double(), torch.empty_like(s["q"], dtype=torch.float64)
    table, lens = s["page_table"].long(), s["kv_lens"].tolist()
    ends = None if s["offsets"] is None else s["offsets"].tolist()
    for i, end in enumerate(lens):
        rows = i if ends is None else slice(ends[i], ends[i + 1])
        n = s["k"][rows].shape[0]
        pos = torch.arange(end - n, end, device="cuda")
        slots = table[i].repeat_interleave(case["page"])[pos] * case["page"] + pos.remainder(case["page"])
        kc.view(-1, *kc.shape[2:])[slots] = _rotation(case, s, s["k"][rows], pos)
        vc.view(-1, *vc.shape[2:])[slots] = s["v"][rows].double()
        q[rows] = _rotation(case, s, s["q"][rows], pos)
    return {"q": q, "k_cache": kc, "v_cache": vc}


def _heads_first(t, group=1):
    return t.double().repeat_interleave(group, 1).transpose(0, 1)


def _counts(queries, keys, window, sinks):
    """Which keys count for a query at each position: those up to it, less those that the window has left behind."""
    behind = torch.zeros(1, dtype=torch.bool, device=keys.device)
    if window is not None:
        behind = (keys[None] <= queries[:, None] - window) & (keys[None] >= sinks)
    return (keys[None] <= queries[:, None]) & ~behind


def _paged_exact(case, s):
    group, page = case["hq"] // case["hkv"], case["page"]
    out = torch.zeros_like(s["q"], dtype=torch.float64)
    ends = None if s["offsets"] is None else s["offsets"].tolist()
    for i, n in enumerate(s["kv_lens"].tolist()):
        rows = i if ends is None else slice(ends[i], ends[i + 1])
        q = _heads_first(s["q"][rows])
        if n == 0 or q.shape[1] == 0:
            continue
        mine = s["page_table"][i, : -(-n // page)].long()
        k, v = (_heads_first(c[mine].flatten(0, 1)[:n], group) for c in (s["k_cache"], s["v_cache"]))
        scores = q @ k.transpose(1, 2) / math.sqrt(case["d"])
        if case["causal"]:
            keys = torch.arange(n, device="cuda")
            counts = _counts(keys[n - q.shape[1]:], keys, s["window"], s["sinks"])
            scores = scores.masked_fill(~counts, -math.inf)
        out[rows] = (torch.softmax(scores, -1) @ v).transpose(0, 1)
    return out


def _window_exact(case, s):
    group, train, scale = case["hq"] // case["hkv"], case["op"] == "window_train", 1 / math.sqrt(case["d"])
    o, dq = (torch.zeros_like(s["q"], dtype=torch.float64) for _ in range(2))
    dk, dv = (torch.zeros_like(s["k"], dtype=torch.float64) for _ in range(2))
    lse = torch.full(s["q"].shape[:-1], -math.inf, dtype=torch.float64, device="cuda")
    ends = (s["offsets"] if s["offsets"] is not None else s["lens"]).tolist()
    for i in range(case["b"]):
        packed = s["offsets"] is not None
        rows = slice(ends[i], ends[i + 1]) if packed else slice(0, ends[i])
        mine = (lambda t: t[rows]) if packed else (lambda t: t[i, rows])
        q, k, v = _heads_first(mine(s["q"])), _heads_first(mine(s["k"]), group), _heads_first(mine(s["v"]), group)
        if q.shape[1] == 0:
            continue
        at = torch.arange(q.shape[1], device="cuda")
        counts = _counts(at, at, s["window"], s["sinks"])
        if s["mask"] is not None:
            counts = counts & mine(s["mask"])
        scores = (q @ k.transpose(1, 2) * scale).masked_fill(~counts, -math.inf)
        p = torch.softmax(scores, -1).nan_to_num(0.0)  # a row without a key
        mine(lse)[:] = torch.logsumexp(scores, -1).T
        mine(o)[:] = (p @ v).transpose(0, 1)
        if train:
            g = _heads_first(mine(s["grad"]))
            dp = g @ v.transpose(1, 2)
            ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * scale
            mine(dq)[:] = (ds @ k).transpose(0, 1)
            for into, per_head in ((dk, ds.transpose(1, 2) @ q), (dv, p.transpose(1, 2) @ g)):
                mine(into)[:] = per_head.reshape(case["hkv"], group, -1, case["d"]).sum(1).transpose(0, 1)
    return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv} if train else o


# ------------------------------------------------------------------ what a pass cannot do without
def _pairs(first, n, window, sinks):
    """(query, key) pairs that count for the queries at positions first .. first + n - 1, and the keys among them."""
    if n == 0:
        return 0, 0
    last = first + n - 1
    if not window:
        return n * (first + last + 2) // 2, last + 1
    p = range(first, last + 1)
    pairs = sum(min(x + 1, window) + min(sinks, max(0, x + 1 - window)) for x in p)
    lo = max(0, first - window + 1)
    return pairs, last + 1 - lo + min(sinks, lo)


def work(case):
    size, b, d = 4 if case["dtype"] == "f32" else 2, case["b"], case["d"]
    if case["op"].startswith("rotary"):
        n = b * case["l"]
        passes = 2 if case["op"] == "rotary_train" else 1
        return {"bytes": passes * 2 * n * case["heads"] * d * size + 8 * n,
                "flops": passes * 3 * n * case["heads"] * case["rot"]}
    hq, hkv = case["hq"], case["hkv"]
    if case["op"] == "append":
        n = sum(_new_and_cached(case)[0])
        return {"bytes": 2 * n * (hq + 2 * hkv) * d * size, "flops": 3 * n * (hq + hkv) * case["rot"]}
    if case["op"] == "paged":
        new, cached = _new_and_cached(case)
        if case["causal"]:
            # by the mean of the cached lengths, whose order is the seed's
            before = sum(cached) // b
            counts = [_pairs(before, n, case["window"], case["sinks"]) for n in new]
        else:
            counts = [(n * c, c) for n, c in zip(new, cached)]
        pairs, keys = sum(c[0] for c in counts), sum(c[1] for c in counts)
        return {"bytes": (2 * sum(new) * hq + 2 * keys * hkv) * d * size, "flops": 4 * pairs * hq * d}
    lens = _ramp(b, case["l"])
    rows = sum(lens) if case["kv"] == "packed" else b * case["l"]
    pairs = sum(_pairs(0, n, case["window"], case["sinks"])[0] for n in lens)
    qo, kv = 2 * rows * hq * d * size, 2 * sum(lens) * hkv * d * size
    if case["op"] == "window_fwd":
        return {"bytes": qo + kv, "flops": 4 * pairs * hq * d}
    return {"bytes": 2 * qo + kv + 2 * rows * hkv * d * size + 4 * rows * hq, "flops": 14 * pairs * hq * d}
