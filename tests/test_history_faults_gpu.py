"""What the operators of a growing history make of inputs that are out of range or laid out unusually, on the GPU against
their definitions in 64 bits (bounds: history_plain)."""
import warnings

import pytest
import torch

import history_plain as plain
from sequence_plain import within
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
