"""What the operators of a growing history make of inputs that are out of range or laid out unusually, on the GPU against
their definitions in 64 bits (bounds: history_plain)."""
import warnings

import pytest
import torch

import history_plain as plain
from sequence_plain import U, U32, within
from test_history_gpu import BF16, DTYPES, F32, I32, cache_case, generator, ints, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from dynamic_embedding_tables_amd import recis
    recis.load_library()


@pytest.fixture
def seq():
    from dynamic_embedding_tables_amd import sequence
    return sequence


def without_bad_pages(q, kc, vc, table, lens, offsets=None, causal=True, window=None, sinks=0):
    """{o, lse: (value, bound)}: paged attention to the keys whose page's number is one."""
    pages, page_size = kc.shape[:2]
    val = {"o": torch.zeros_like(q, dtype=torch.float64),
           "lse": torch.full(q.shape[:-1], -float("inf"), dtype=torch.float64)}
    err = {n: torch.full_like(x, 1e-30) for n, x in val.items()}
    for b, rows in enumerate(plain.new_rows(table.shape[0], q.shape[1], offsets)):
        at, n, total = (b, rows) if offsets is None else (rows,), len(rows), lens[b]
        if not n or not total:
            continue
        keys = torch.arange(total)
        there = (table[b] >= 0) & (table[b] < pages)
        ok = there[keys // page_size][None].expand(n, total)
        if causal:
            ok = ok & plain.seen(total - n + torch.arange(n), keys, window, sinks)
        known = torch.where(there, table[b], 0)
        got = plain.attention(q[at], plain.keys_of(kc, known, page_size, total),
                              plain.keys_of(vc, known, page_size, total), ok, q.shape[-1] ** -0.5)
        for name, (x, e) in got.items():
            val[name][at], err[name][at] = x, e
    return {n: (val[n], err[n]) for n in val}


@pytest.mark.parametrize("how", [{}, {"window": 70, "sinks": 9}, {"causal": False}])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new,page_size,heads", [
    (1, 16, (4, 4, 32)), (4, 5, (8, 2, 40)), (16, 64, (1, 1, 128)), (17, 64, (1, 1, 128)), (40, 5, (8, 2, 40)),
    (150, 16, (4, 2, 64)), (33, 24, (2, 2, 77)), (20, 1, (2, 1, 74)), (70, 128, (2, 1, 96)),
])
def test_keys_of_a_page_out_of_range_do_not_count(seq, new, page_size, heads, dtype, how):
    """The same for few rows and for many, told or not: such a key has no weight, and no other entry's key takes its
    place."""
    from dynamic_embedding_tables_amd import recis
    (hq, hkv, dim), lens = heads, [700, 150, 333, 260]
    gen = generator(new, page_size, dim, len(how))
    kc, vc, table = cache_case(gen, len(lens), lens, page_size, hkv, dim, dtype, garbage=0.0)
    kc[0], vc[0] = 3.0, 50.0   # page 0 would be noticed
    table[table == 0] = kc.shape[0] - 1
    pages = kc.shape[0]
    last = [-(-n // page_size) - 1 for n in lens]
    table[0, last[0] // 2], table[0, 0], table[0, last[0]] = -1, pages, 1 << 30
    table[1] = -1   # no key at all
    table[2, last[2] - 1:] = (1 << 31) - 1
    dev = [t.cuda() for t in (kc, vc, table, ints(*lens))]
    for packed in (False, True):
        if packed:
            counts = [max(0, new - i) for i in range(len(lens))]
            offsets = torch.tensor([sum(counts[:i]) for i in range(len(lens) + 1)], dtype=I32)
            q, more = normal(gen, sum(counts), hq, dim, dtype=dtype), {"q_offsets": offsets.cuda(), "max_q_len": new}
        else:
            q, offsets, more = normal(gen, len(lens), new, hq, dim, dtype=dtype), None, {}
        error = torch.zeros(1, dtype=I32).cuda()
        o, lse = seq.paged_attention(q.cuda(), *dev, return_lse=True, error=error, **how, **more)
        with pytest.raises(recis.RecisError) as e:
            seq.check(error)
        assert e.value.status == recis.RECIS_ERR_INVALID_ARG
        want = without_bad_pages(q, kc, vc, table, lens, offsets, **how)
        within(o, *want["o"], what=(packed, "o"))
        within(lse, *want["lse"], what=(packed, "lse"))
        assert torch.equal(seq.paged_attention(q.cuda(), *dev, **how, **more), o)


def leave_nan(*like):
    """Memory that the next tensors of these shapes are likely to get, full of NaN."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full_like(t, float("nan")) for t in like for _ in range(4)]
    del held


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,hq,hkv", [(16, 2, 2), (77, 4, 2), (128, 3, 1)])
@pytest.mark.parametrize("offsets,max_len", [
    ((0, 120, 361, 361), 360), ((0, 120, 400, 500), 360), ((-3, 120, 200, 360), 360), ((0, 120, (1 << 31) - 1), 360),
    ((-(1 << 31), 7, 300, 360), 360), ((-9, -5, 361, 400), 360), ((0, 300, 360), 299),
])
def test_rows_of_an_entry_out_of_range_are_zeros(seq, offsets, max_len, dim, hq, hkv, dtype):
    """An entry whose rows are not all there, or too many, is taken as one without rows: nothing that was in memory
    before comes back in its place."""
    from dynamic_embedding_tables_amd import recis
    gen = generator(dim, hq, max_len)
    q, grad = (normal(gen, 360, hq, dim, dtype=dtype) for _ in range(2))
    k, v = (normal(gen, 360, hkv, dim, dtype=dtype) for _ in range(2))
    good = [(lo, hi) for lo, hi in zip(offsets, offsets[1:]) if 0 <= lo <= hi <= 360 and hi - lo <= max_len]
    dev = [t.cuda() for t in (q, k, v)]
    kw = {"offsets": ints(*offsets).cuda(), "max_len": max_len, "window": 50, "sinks": 3}
    error = torch.zeros(1, dtype=I32).cuda()
    leave_nan(*dev)
    o, lse = seq.self_attention(*dev, return_lse=True, error=error, **kw)
    with pytest.raises(recis.RecisError):
        seq.check(error)
    leave_nan(*dev)
    grads = seq.self_attention_backward(grad.cuda(), *dev, o, lse, **kw)
    want = {n: [torch.zeros(t.shape, dtype=torch.float64) + (-float("inf") if n == "lse" else 0.0),
                torch.full(t.shape, 1e-30, dtype=torch.float64)]
            for n, t in (("o", q), ("lse", q[..., 0]), ("dq", q), ("dk", k), ("dv", v))}
    for lo, hi in good:
        pos = torch.arange(hi - lo)
        got = plain.attention(q[lo:hi], k[lo:hi], v[lo:hi], plain.seen(pos, pos, 50, 3), dim**-0.5, grad[lo:hi])
        for n, (x, e) in got.items():
            want[n][0][lo:hi], want[n][1][lo:hi] = x, e
    for name, t in zip(want, (o, lse, *grads)):
        within(t, *want[name], what=(offsets, name))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offsets", [(-3, 4, 8), (-(1 << 31), 4, 8), (0, 4, 9), (0, 5, (1 << 31) - 1), (-1, 4, 9)])
def test_append_of_an_entry_out_of_range_stores_nothing(seq, offsets, dtype):
    """As the attention that reads the cache: an entry whose rows are not all there is taken as one without rows."""
    from dynamic_embedding_tables_amd import recis
    gen, lens = generator(len(offsets), 91), [20, 17]
    kc, vc, table = cache_case(gen, 2, lens, 8, 2, 16, dtype, garbage=7.0)
    k, v = (normal(gen, 8, 2, 16, dtype=dtype) for _ in range(2))
    q, freqs = normal(gen, 8, 4, 16, dtype=dtype), seq.rotary_frequencies(16)
    dk, dv, error = kc.cuda(), vc.cuda(), torch.zeros(1, dtype=I32).cuda()
    got = seq.cache_append(k.cuda(), v.cuda(), dk, dv, table.cuda(), ints(*lens).cuda(), q=q.cuda(),
                           q_offsets=ints(*offsets).cuda(), freqs=freqs, error=error)
    with pytest.raises(recis.RecisError) as e:
        seq.check(error)
    assert e.value.status == recis.RECIS_ERR_INVALID_ARG
    want_k, bound_k, want_v = kc.double(), torch.zeros_like(kc, dtype=torch.float64), vc.clone()
    want_q = [torch.zeros_like(q, dtype=torch.float64), torch.full_like(q, 1e-30, dtype=torch.float64)]
    for b, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        if 0 <= lo and hi <= 8:
            pos = lens[b] - (hi - lo) + torch.arange(hi - lo)
            where = plain.slots(table[b], 8, pos)
            want_k[where], bound_k[where] = plain.rotary(k[lo:hi], freqs.cpu(), pos, False, 1.0)
            want_v[where] = v[lo:hi]
            want_q[0][lo:hi], want_q[1][lo:hi] = plain.rotary(q[lo:hi], freqs.cpu(), pos, False, 1.0)
    within(dk, want_k, bound_k)
    assert torch.equal(dv.cpu(), want_v)
    within(got, *want_q)


@pytest.mark.parametrize("new", [1, 30])
def test_page_tables_whose_rows_overlap(seq, new):
    """One history that several entries read (candidates of one user): its row of the table expanded, not repeated."""
    gen = generator(new, 92)
    kc, vc, table = cache_case(gen, 1, [90], 16, 2, 32, F32, garbage=0.0)
    q = normal(gen, 5, new, 4, 32).cuda()
    dev = (kc.cuda(), vc.cuda())
    lens = ints(90, 90, 17, 64, 33).cuda()
    want = seq.paged_attention(q, *dev, table.expand(5, -1).contiguous().cuda(), lens, causal=False)
    assert torch.equal(seq.paged_attention(q, *dev, table.cuda().expand(5, -1), lens, causal=False), want)
    row = torch.cat([table[0], table[0]]).cuda()   # entry b's pages begin one further on
    sliding = row.as_strided((5, table.shape[1]), (1, 1))
    want = seq.paged_attention(q, *dev, sliding.contiguous(), lens)
    assert torch.equal(seq.paged_attention(q, *dev, sliding, lens), want)
    k = normal(gen, 2, 1, 2, 32).cuda()   # and the append, to slots that the entries do not share
    two = table.cuda().expand(2, -1)
    seq.cache_append(k, k, *dev, two, ints(3, 20).cuda())
    for b, n in enumerate((3, 20)):
        page, slot = plain.slots(table[0], 16, torch.tensor([n - 1]))
        assert torch.equal(dev[0][page.cuda(), slot.cuda()], k[b]) and torch.equal(dev[1][page.cuda(), slot.cuda()], k[b])


@pytest.mark.parametrize("new", [1, 30])
def test_a_cache_that_is_copied_is_warned_about(seq, new):
    """Heads whose elements are strided: the whole cache is copied, on every call, and not silently."""
    gen = generator(new, 93)
    kc, vc, table = cache_case(gen, 2, [90, 40], 16, 2, 32, F32, garbage=0.0)
    q, kc, vc, table, lens = (t.cuda() for t in (normal(gen, 2, new, 4, 32), kc, vc, table, ints(90, 40)))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        want = seq.paged_attention(q, kc, vc, table, lens)
    apart = [t.transpose(2, 3).contiguous().transpose(2, 3) for t in (kc, vc)]
    for caches in ((apart[0], vc), (kc, apart[1]), apart):
        with pytest.warns(UserWarning, match="copied whole"):
            assert torch.equal(seq.paged_attention(q, *caches, table, lens), want)


@pytest.mark.parametrize("bad", [(1 << 31) - 1, -1, -(1 << 31), 49])
@pytest.mark.parametrize("dtype", DTYPES)
def test_an_entry_whose_length_is_out_of_range_has_no_keys(seq, dtype, bad):
    """The largest and the smallest number that a length can be, too: nothing is stored, zeros come back, and the other
    entries are as they would be."""
    gen, dim = generator(94), 32
    kc, vc, table = cache_case(gen, 2, [48, 48], 16, 2, dim, dtype, garbage=0.0)
    k, q = normal(gen, 2, 40, 2, dim, dtype=dtype).cuda(), normal(gen, 2, 40, 4, dim, dtype=dtype).cuda()
    freqs, good, lens = seq.rotary_frequencies(dim), ints(48, 45).cuda(), ints(bad, 45).cuda()
    stored = [(kc.cuda(), vc.cuda()) for _ in range(2)]
    turned = [seq.cache_append(k, k, *c, table.cuda(), n, q=q, freqs=freqs) for c, n in zip(stored, (good, lens))]
    assert not bool(turned[1][0].any()) and torch.equal(turned[1][1], turned[0][1])
    for t, was, now in zip((kc, vc), *stored):
        assert torch.equal(now[table[0].long().cuda()].cpu(), t[table[0].long()])
        assert torch.equal(now[table[1].long().cuda()], was[table[1].long().cuda()])
    for rows in (q, q[:, -1:]):
        for how in ({}, {"window": 9, "sinks": 2}, {"causal": False}):
            want = seq.paged_attention(rows, *stored[1], table.cuda(), good, return_lse=True, **how)
            got = seq.paged_attention(rows, *stored[1], table.cuda(), lens, return_lse=True, **how)
            assert not bool(got[0][0].any()) and bool((got[1][0] == -float("inf")).all())
            assert torch.equal(got[0][1], want[0][1]) and torch.equal(got[1][1], want[1][1])
    ends = [ints(40, 30).cuda(), ints(bad, 30).cuda()]
    (want, wl), (got, gl) = (seq.self_attention(q, k, k, lens=n, window=9, sinks=2, return_lse=True) for n in ends)
    assert not bool(got[0].any()) and bool((gl[0] == -float("inf")).all()) and torch.equal(got[1], want[1])
    grads = [seq.self_attention_backward(q, q, k, k, o, x, lens=n, window=9, sinks=2)
             for o, x, n in ((want, wl, ends[0]), (got, gl, ends[1]))]
    for a, b in zip(*grads):
        assert not bool(b[0].any()) and torch.equal(b[1], a[1])


@pytest.mark.parametrize("length,group,dim", [(64, 1, 64), (50, 2, 64), (64, 1, 128), (33, 4, 128)])
def test_short_histories_take_delta_from_the_weights(seq, length, group, dim):
    """bfloat16, one key with nearly all the weight: what is left of its dP after delta is small, and delta from out
    would bring out's rounding into it. Histories within one tile of keys have it from P and dP, all in 32 bits; the
    bound has no rounding to bfloat16 but that of dS where it meets K or Q, and of the results.

    P: its score's error, twice, and L's (history_plain). dP: d products, from -delta. delta: P's and dP's errors, and
    a sum of as many terms as there are keys."""
    gen = generator(length, dim, 95)
    q = (normal(gen, length, group, dim) * 0.3 + 1).to(BF16)
    k, v, grad = (normal(gen, length, h, dim) for h in (1, 1, group))
    k, scale = k * 0.3, dim**-0.5
    k[0] = 7 / (dim * scale)
    k, v, grad = (t.to(BF16) for t in (k, v, grad))
    dev = [t[None].cuda() for t in (q, k, v)]
    o, lse = seq.self_attention(*dev, return_lse=True)
    dq, dk, _ = seq.self_attention_backward(grad[None].cuda(), *dev, o, lse)
    ok, u, n = torch.ones(length, length).tril().bool(), U[BF16], length
    K, V = k[:, 0].double(), v[:, 0].double()
    tells_apart, want_k, err_k = False, 0.0, 1e-30
    for h in range(group):
        Q, G = q[:, h].double(), grad[:, h].double()
        S = scale * Q @ K.T
        eS = (dim + 6) * U32 * scale * (Q.abs() @ K.abs().T) + 4 * U32 * S.abs()
        L = torch.logsumexp(S.masked_fill(~ok, -float("inf")), -1, keepdim=True)
        P = torch.where(ok, torch.exp(S - L), 0.0)
        eP = 2 * eS.masked_fill(~ok, 0).amax(-1, keepdim=True) + eS + (n + 12) * U32
        eP = (eP + eP.amax(-1, keepdim=True) + 8 * U32 * (L.abs() + S.abs() + 1)) * 1.1
        dP, aP = G @ V.T, G.abs() @ V.abs().T
        delta = (P * dP).sum(-1, keepdim=True)
        edP = (dim + 2) * U32 * (aP + delta.abs())
        edelta = (P * (eP * dP.abs() + (1 + eP) * edP + n * U32 * dP.abs())).sum(-1, keepdim=True)
        dS = P * (dP - delta)
        edS = dS.abs() * (eP + 2 * U32) + P * (1 + eP) * (edP + edelta)
        edS = edS + u * (dS.abs() + edS)
        out = (P @ V).to(BF16).double()   # what delta from out would make of it
        wrong = P * (dP - (G * out).sum(-1, keepdim=True))
        want = scale * dS @ K
        bound = scale * (edS + (n + 2) * U32 * dS.abs()) @ K.abs()
        bound = bound + u * (want.abs() + bound) + 1e-30
        within(dq[0, :, h], want, bound, what=("dq", h))
        tells_apart |= bool(((scale * wrong @ K - want).abs() > bound).any())
        want_k = want_k + scale * dS.T @ Q
        err_k = err_k + scale * (edS + (n * group + 2) * U32 * dS.abs()).T @ Q.abs()
    err_k = err_k + u * (want_k.abs() + err_k)
    within(dk[0, :, 0], want_k, err_k, what="dk")
    assert tells_apart   # (dQ's bound: over dK's many rows the roundings of out may cancel)


@pytest.mark.parametrize("dtype", DTYPES)
def test_packed_calls_captured_into_a_graph(seq, dtype):
    """Packed histories and packed new events: the graph is replayed with other entries in the same rows."""
    gen, dim, rows = generator(96), 32, 120
    s = {"q": normal(gen, rows, 4, dim, dtype=dtype).cuda(), "k": normal(gen, rows, 2, dim, dtype=dtype).cuda(),
         "g": normal(gen, rows, 4, dim, dtype=dtype).cuda(), "off": ints(0, 50, 50, 120).cuda(), "at": ints(60, 9, 200).cuda(),
         "kc": torch.zeros(30, 16, 2, dim, dtype=dtype).cuda(), "vc": torch.zeros(30, 16, 2, dim, dtype=dtype).cuda(),
         "table": torch.randperm(30, generator=gen)[:30].view(3, 10).to(I32).cuda()}
    s["table"], s["kc"], s["vc"] = (t.repeat(*n).contiguous() for t, n in (
        (s["table"], (1, 2)), (s["kc"], (2, 1, 1, 1)), (s["vc"], (2, 1, 1, 1))))
    s["table"][:, 10:] += 30
    freqs = seq.rotary_frequencies(dim)

    def step():
        band = {"offsets": s["off"], "max_len": 120, "window": 20, "sinks": 3}
        o, lse = seq.self_attention(s["q"], s["k"], s["k"], return_lse=True, **band)
        grads = seq.self_attention_backward(s["g"], s["q"], s["k"], s["k"], o, lse, **band)
        turned = seq.cache_append(s["k"], s["k"], s["kc"], s["vc"], s["table"], s["at"], q=s["q"], q_offsets=s["off"],
                                  freqs=freqs)
        where = (s["kc"], s["vc"], s["table"], s["at"])
        many = seq.paged_attention(turned, *where, q_offsets=s["off"], max_q_len=120, return_lse=True)
        few = seq.paged_attention(turned, *where, q_offsets=s["few"], max_q_len=3, window=30, sinks=1, return_lse=True)
        return [o, lse, *grads, turned, *many, *few]

    s["few"] = ints(0, 3, 3, 5).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    ends = [(0, 50, 50, 120), (0, 1, 2, 3), (7, 60, 90, 100), (0, 0, 0, 0), (0, 120, 120, 120)]
    for i, off in enumerate(ends):
        for name in ("q", "k", "g"):
            s[name].copy_(normal(gen, *s[name].shape, dtype=dtype))
        s["off"].copy_(ints(*off)), s["few"].copy_(ints(*[(0, 3, 3, 5), (1, 2, 3, 4), (0, 0, 0, 2)][i % 3]))
        s["at"].copy_(ints(60 + 40 * i, 70, 250))
        kc, vc = s["kc"].clone(), s["vc"].clone()
        want = step()
        stored = s["kc"].clone(), s["vc"].clone()
        s["kc"].copy_(kc), s["vc"].copy_(vc)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(s["kc"], stored[0]) and torch.equal(s["vc"], stored[1])
        for j, (a, b) in enumerate(zip(want, held)):
            assert torch.equal(a, b), (off, j)
