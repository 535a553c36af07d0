"""The operators of a growing history on the GPU against their definitions in 64 bits, at the sizes, layouts and masks
where they can go wrong (bounds: history_plain)."""
import math
import warnings

import pytest
import torch

import history_plain as plain
from sequence_plain import TINY, U, U32, within

pytestmark = pytest.mark.gpu
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
DTYPES = [F32, BF16]


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


def generator(*key):
    return torch.Generator().manual_seed(sum((i + 1) * int(k) for i, k in enumerate(key)) + 29)


def normal(gen, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype)


def ints(*values):
    return torch.tensor(values, dtype=I32)


def on_gpu(kw):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in kw.items()}


def strided_copy(t, order):
    """The same values on the GPU with the axes stored in another order, and room between them."""
    big = torch.zeros([n + 1 for n in t.permute(order).shape[:-1]] + [t.shape[order[-1]] + 8], dtype=t.dtype,
                      device="cuda")
    view = big[tuple(slice(0, n) for n in t.permute(order).shape)].permute([order.index(i) for i in range(t.dim())])
    return view.copy_(t)


# ---------------------------------------------------------- rotary positions
ROTARY = [  # batch, seq, heads, dim, rotated
    (1, 1, 1, 2, 2), (2, 3, 1, 16, 16), (3, 7, 4, 32, 32), (1, 700, 2, 64, 64), (2, 33, 6, 40, 24), (5, 9, 3, 7, 4),
    (2, 50, 20, 128, 128), (1, 4, 2, 1024, 1024), (4, 5, 2, 34, 34), (2, 17, 5, 24, 0), (1, 3, 1, 9, 8),
    (2, 1030, 1, 12, 12), (3, 2, 2, 48, 44),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", ROTARY)
def test_rotary(seq, shape, dtype, interleaved):
    b, l, heads, dim, rot = shape
    gen = generator(*shape)
    x, g = normal(gen, b, l, heads, dim, dtype=dtype), normal(gen, b, l, heads, dim, dtype=dtype)
    freqs = seq.rotary_frequencies(rot, base=500.0)
    far = torch.randint(-(1 << 20), 1 << 31, (b, l), generator=gen)
    for positions in (None, torch.arange(l) * 3 + 5, far):
        at = (torch.arange(l) if positions is None else positions).expand(b, l)
        dev = None if positions is None else positions.cuda()
        y = seq.rotary(x.cuda(), freqs, dev, interleaved, amplitude=1.2)
        within(y, *plain.rotary(x, freqs.cpu(), at, interleaved, 1.2), what=shape)
        dx = seq.rotary_backward(g.cuda(), freqs, dev, interleaved, amplitude=1.2)
        within(dx, *plain.rotary(g, freqs.cpu(), at, interleaved, 1.2, back=True), what=shape)
        assert torch.equal(y[..., rot:].cpu(), x[..., rot:]) and torch.equal(dx[..., rot:].cpu(), g[..., rot:])
        again = x.cuda()
        assert seq.rotary(again, freqs, dev, interleaved, amplitude=1.2, out=again) is again and torch.equal(again, y)
        if b == 1:
            packed = seq.rotary(x[0].cuda(), freqs, None if dev is None else dev.reshape(-1), interleaved, 1.2)
            assert torch.equal(packed, y[0])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,rot", [(32, 32), (40, 24), (38, 30), (64, 16)])
def test_rotary_strides(seq, dim, rot, dtype, interleaved):
    gen = generator(dim, rot)
    x = normal(gen, 3, 11, 4, dim, dtype=dtype)
    freqs = seq.rotary_frequencies(rot)
    want = seq.rotary(x.cuda(), freqs, interleaved=interleaved)
    for order in ((0, 1, 2, 3), (0, 2, 1, 3), (2, 0, 1, 3), (1, 2, 0, 3)):
        assert torch.equal(seq.rotary(strided_copy(x, order), freqs, interleaved=interleaved), want), order
        out = strided_copy(torch.full_like(x, 7.0), order)
        seq.rotary(x.cuda(), freqs, interleaved=interleaved, out=out)
        assert torch.equal(out, want), order
    wide = torch.full((3, 11, 4, dim + 5), 7.0, dtype=dtype).cuda()   # unaligned, and its rest left alone
    wide[..., 3:3 + dim] = x.cuda()
    seq.rotary(wide[..., 3:3 + dim], freqs, interleaved=interleaved, out=wide[..., 3:3 + dim])
    assert torch.equal(wide[..., 3:3 + dim], want)
    assert bool((wide[..., :3] == 7).all()) and bool((wide[..., 3 + dim:] == 7).all())
    at = torch.arange(11).cuda() * 2
    assert torch.equal(seq.rotary(x.cuda(), freqs, at.expand(3, 11), interleaved),
                       seq.rotary(x.cuda(), freqs, at, interleaved))
    assert torch.equal(seq.rotary(x.cuda(), freqs, torch.arange(22).cuda()[::2], interleaved),
                       seq.rotary(x.cuda(), freqs, at, interleaved))


def test_rotary_gradient_is_the_difference_quotient(seq):
    """The map is linear, so the quotient of a step of any size is the gradient, up to the rounding of two results."""
    gen = generator(31)
    x, g, step = (normal(gen, 2, 9, 3, 24) for _ in range(3))
    freqs, at = seq.rotary_frequencies(20), torch.randint(0, 5000, (2, 9), generator=gen)
    up, down = (seq.rotary((x + s * step).cuda(), freqs, at.cuda(), amplitude=0.8) for s in (1, -1))
    slope = ((up.double() - down.double()) * g.cuda().double()).sum() / 2
    dx = seq.rotary_backward(g.cuda(), freqs, at.cuda(), amplitude=0.8).double()
    size = sum((t.cuda().double().abs() * g.cuda().double().abs()).sum() for t in (up, down)) + \
        (dx.abs() * step.cuda().double().abs()).sum()
    assert abs(slope - (dx * step.cuda().double()).sum()) <= 16 * U32 * 2 * size


def test_rotary_nothing_to_turn(seq):
    freqs = seq.rotary_frequencies(8)
    for shape in ((0, 2, 8), (0, 3, 2, 8), (2, 0, 2, 8)):
        assert seq.rotary(torch.empty(shape).cuda(), freqs).shape == shape


def test_rotary_not_finite_stays_in_its_pair(seq):
    x = torch.ones(1, 3, 2, 8)
    x[0, 1, 0, 2], x[0, 1, 1, 7] = math.nan, math.inf
    y = seq.rotary(x.cuda(), seq.rotary_frequencies(8)).cpu()
    bad = ~torch.isfinite(y)
    assert bad.sum() == 4 and bool(bad[0, 1, 0, [2, 6]].all()) and bool(bad[0, 1, 1, [3, 7]].all())


def test_rotary_beyond_32_bit_offsets(seq):
    l, heads, dim = 1 << 20, 20, 128   # 2.7e9 elements
    x = torch.empty(l, heads, dim, dtype=BF16, device="cuda")
    x[:] = torch.arange(dim, device="cuda", dtype=BF16)
    freqs = seq.rotary_frequencies(dim)
    y = seq.rotary(x, freqs, out=x)
    for at in (0, (1 << 31) // (heads * dim) + 3, l - 1):
        row = torch.arange(dim, dtype=BF16).expand(1, heads, dim)
        within(y[at:at + 1], *plain.rotary(row, freqs.cpu(), torch.tensor([at]), False, 1.0), what=at)


# ------------------------------------------------------------- paged cache
def cache_case(gen, batch, lens, page_size, heads, dim, dtype, spare=3, garbage=math.nan):
    """A cache whose pages lie in any order, what no entry owns being garbage; (k, v, table)."""
    width = max(1, max(-(-n // page_size) for n in lens))
    pages = batch * width + spare
    table = torch.randperm(pages, generator=gen)[: batch * width].view(batch, width).to(I32)
    k, v = (torch.full((pages, page_size, heads, dim), garbage, dtype=dtype) for _ in range(2))
    for b, n in enumerate(lens):
        page, slot = plain.slots(table[b], page_size, torch.arange(n))
        for t in (k, v):
            t[page, slot] = normal(gen, n, heads, dim, dtype=dtype)
    return k, v, table


APPEND = [  # new rows an entry, keys before them, page size, (q heads, kv heads, dim, rotated), packed
    ([1, 1, 1], [0, 5, 16], 4, (4, 2, 32, 32), False), ([3, 3], [0, 40], 16, (0, 1, 16, 16), False),
    ([5, 0, 1, 9], [3, 7, 0, 0], 5, (6, 3, 40, 24), True), ([1], [1000], 1, (2, 2, 64, 64), True),
    ([130, 0, 0, 77, 1], [3, 2, 0, 60, 64], 64, (4, 4, 32, 32), True), ([2] * 70, list(range(70)), 7, (1, 1, 128, 128), False),
    ([0] * 300 + [3] + [0] * 500 + [1, 2], [1] * 803, 8, (2, 1, 8, 8), True), ([4, 4], [10, 0], 3, (3, 1, 9, 6), False),
    ([600], [0], 24, (4, 4, 128, 128), False), ([2, 3], [1, 1], 16, (2, 2, 16, 0), True),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(APPEND)))
def test_cache_append(seq, case, dtype, interleaved):
    new, before, page_size, (hq, hkv, dim, rot), packed = APPEND[case]
    gen = generator(case, 3)
    lens = [n + c for n, c in zip(new, before)]
    kc, vc, table = cache_case(gen, len(new), lens, page_size, hkv, dim, dtype, garbage=7.0)
    front, back = (2, 3) if packed else (0, 0)
    offsets = torch.tensor([front] + [front + sum(new[:i + 1]) for i in range(len(new))], dtype=I32) if packed else None
    lead = (front + sum(new) + back,) if packed else (len(new), new[0])
    k, v = normal(gen, *lead, hkv, dim, dtype=dtype), normal(gen, *lead, hkv, dim, dtype=dtype)
    q = normal(gen, *lead, hq, dim, dtype=dtype) if hq else None
    freqs = seq.rotary_frequencies(rot)
    error = torch.zeros(1, dtype=I32).cuda()
    dk, dv = kc.cuda(), vc.cuda()
    got = seq.cache_append(k.cuda(), v.cuda(), dk, dv, table.cuda(), ints(*lens).cuda(), error=error,
                           q=None if q is None else q.cuda(), q_offsets=None if offsets is None else offsets.cuda(),
                           freqs=freqs, interleaved=interleaved, amplitude=0.9)
    seq.check(error)
    want_k, bound_k, want_v = kc.double(), torch.zeros_like(kc, dtype=torch.float64), vc.clone()
    want_q = None if q is None else (torch.zeros_like(q, dtype=torch.float64), torch.full_like(q, TINY, dtype=torch.float64))
    for b, rows in enumerate(plain.new_rows(len(new), new[0], offsets)):
        at = (rows,) if packed else (b, rows)
        pos = before[b] + torch.arange(new[b])
        where = plain.slots(table[b], page_size, pos)
        want_k[where], bound_k[where] = plain.rotary(k[at], freqs.cpu(), pos, interleaved, 0.9)
        want_v[where] = v[at]
        if q is not None:
            want_q[0][at], want_q[1][at] = plain.rotary(q[at], freqs.cpu(), pos, interleaved, 0.9)
    within(dk, want_k, bound_k)
    assert torch.equal(dv.cpu(), want_v)
    assert got is None if q is None else within(got, *want_q) is None


def test_cache_append_as_it_is_without_frequencies(seq):
    gen = generator(41)
    kc, vc, table = cache_case(gen, 2, [9, 12], 4, 2, 24, BF16, garbage=0.0)
    k, v = normal(gen, 2, 3, 2, 24, dtype=BF16), normal(gen, 2, 3, 2, 24, dtype=BF16)
    dk, dv = kc.cuda(), vc.cuda()
    seq.cache_append(k.cuda(), v.cuda(), dk, dv, table.cuda(), ints(9, 12).cuda())
    for b, n in enumerate((9, 12)):
        where = plain.slots(table[b], 4, torch.arange(n - 3, n))
        kc[where], vc[where] = k[b], v[b]
    assert torch.equal(dk.cpu(), kc) and torch.equal(dv.cpu(), vc)


@pytest.mark.parametrize("packed", [False, True])
def test_cache_append_padding_rows_and_idle_entries(seq, packed):
    """Rows at negative positions are not stored; an entry of length 0 is idle."""
    gen = generator(42)
    lens, new = [0, 2, 5, 4], 4
    kc, vc, table = cache_case(gen, 4, lens, 4, 1, 8, F32, garbage=7.0)
    kc[:], vc[:] = 7.0, 7.0
    k = normal(gen, 4, new, 1, 8)
    freqs = seq.rotary_frequencies(8)
    dk, dv, error = kc.cuda(), vc.cuda(), torch.zeros(1, dtype=I32).cuda()
    kd = (k.reshape(16, 1, 8) if packed else k).cuda()
    off = torch.arange(0, 17, 4, dtype=I32).cuda() if packed else None
    seq.cache_append(kd, kd, dk, dv, table.cuda(), ints(*lens).cuda(), q_offsets=off, error=error)
    q = seq.cache_append(kd, kd, dk.clone(), dv.clone(), table.cuda(), ints(*lens).cuda(), q=kd, q_offsets=off,
                         freqs=freqs, error=error)
    seq.check(error)
    assert bool(torch.isfinite(q).all())
    for b, n in enumerate(lens):
        take = min(n, new)
        where = plain.slots(table[b], 4, torch.arange(n - take, n))
        kc[where] = k[b, new - take:]
    assert torch.equal(dk.cpu(), kc) and torch.equal(dv.cpu(), kc)


@pytest.mark.parametrize("order", [(0, 1, 2, 3), (0, 2, 1, 3), (2, 0, 1, 3)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_cache_layouts(seq, dtype, order):
    """Append and attention over caches of other layouts (heads before slots, one head after the other, layers)."""
    gen = generator(43, order[0], order[1])
    lens, dim = [40, 3, 17], 32
    kc, vc, table = cache_case(gen, 3, lens, 8, 2, dim, dtype, garbage=0.0)
    k, v, q = (normal(gen, 3, 2, h, dim, dtype=dtype) for h in (2, 2, 4))
    freqs, tl = seq.rotary_frequencies(dim), (table.cuda(), ints(*lens).cuda())
    flat_k, flat_v = kc.cuda(), vc.cuda()
    other_k, other_v = strided_copy(kc, order), strided_copy(vc, order)
    wide = torch.full((3, 8), -1, dtype=I32).cuda()   # a table with room for more pages
    wide[:, :table.shape[1]] = table.cuda()
    narrow = wide[:, :table.shape[1]]
    for a, b in (((flat_k, flat_v), tl), ((other_k, other_v), (narrow, tl[1]))):
        seq.cache_append(k.cuda(), v.cuda(), *a, *b, freqs=freqs)
    assert torch.equal(flat_k, other_k) and torch.equal(flat_v, other_v)
    qt = q.cuda().transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(seq.paged_attention(q.cuda(), flat_k, flat_v, *tl),
                       seq.paged_attention(qt, other_k, other_v, narrow, tl[1]))


def test_cache_faults_are_recorded(seq):
    from dynamic_embedding_tables_amd import recis
    gen = generator(44)
    lens, dim = [12, 7, 30], 16

    def setup():
        kc, vc, table = cache_case(generator(44), 3, lens, 8, 2, dim, F32, garbage=7.0)
        return kc.cuda(), vc.cuda(), table.cuda(), ints(*lens).cuda()

    k = normal(gen, 3, 4, 2, dim).cuda()
    many = normal(gen, 3, 40, 2, dim).cuda()
    off = ints(0, 4, 8, 12)

    def with_table(at, to):
        def change(kc, vc, table, n, offsets):
            table[at] = to
        return change

    def with_len(at, to):
        def change(kc, vc, table, n, offsets):
            n[at] = to
        return change

    def with_offset(at, to):
        def change(kc, vc, table, n, offsets):
            offsets[at] = to
        return change

    cases = [with_table((0, 1), -1), with_table((0, 1), 1 << 30), with_table((2, 3), 15), with_len(1, -1),
             with_len(1, 33), with_len(2, 1 << 31 - 1)]
    packed = [with_offset(1, 20), with_offset(3, 13), with_offset(0, -1), with_offset(2, 1)]
    for i, (change, ragged) in enumerate([(c, False) for c in cases] + [(c, True) for c in packed]):
        print("fault", i, flush=True)
        kc, vc, table, n = setup()
        offsets = off.clone().cuda()
        change(kc, vc, table, n, offsets)
        kw = {"q_offsets": offsets} if ragged else {}
        rows = k.reshape(12, 2, dim) if ragged else k
        before = kc.clone()
        for error in (torch.zeros(1, dtype=I32).cuda(), None):
            out = seq.cache_append(rows, rows, kc, vc, table, n, q=rows, freqs=seq.rotary_frequencies(dim), error=error, **kw)
            assert out.shape == rows.shape
            if error is not None:
                with pytest.raises(recis.RecisError) as e:
                    seq.check(error)
                assert e.value.status == recis.RECIS_ERR_INVALID_ARG
        # the rest of the cache stays as it was
        own = torch.zeros(kc.shape[:2], dtype=torch.bool)
        for b in range(3):
            page, slot = plain.slots(setup()[2][b].cpu(), 8, torch.arange(32))
            own[page, slot] = True
        assert torch.equal(kc[~own.cuda()], before[~own.cuda()])
        for q in (rows, None if ragged else many):   # few rows, and many
            if q is None:
                continue
            for error in (torch.zeros(1, dtype=I32).cuda(), None):
                more = {"max_q_len": 12, **kw} if ragged else {}
                out = seq.paged_attention(q, kc, vc, table, n, error=error, **more)
                assert out.shape == q.shape
                if error is not None:
                    with pytest.raises(recis.RecisError):
                        seq.check(error)
    # more rows than max_q_len: an entry as if it had none
    kc, vc, table, n = setup()
    error = torch.zeros(1, dtype=I32).cuda()
    out = seq.paged_attention(k.reshape(12, 2, dim), kc, vc, table, n, q_offsets=off.cuda(), max_q_len=3, error=error)
    assert not bool(out.any())
    with pytest.raises(recis.RecisError):
        seq.check(error)


def test_cache_beyond_32_bit_offsets(seq):
    pages, page_size, heads, dim = 9000, 64, 32, 128   # 2.4e9 elements
    gen = generator(45)
    kc, vc = (torch.zeros(pages, page_size, heads, dim, dtype=BF16, device="cuda") for _ in range(2))
    table = torch.tensor([[8999, 2], [8200, 8998]], dtype=I32)
    lens, new = [100, 128], 70
    k, v, q = (normal(gen, 2, 128, heads, dim, dtype=BF16) for _ in range(3))
    for b, n in enumerate(lens):   # the whole history in two calls of one entry each
        at = slice(b, b + 1)
        for lo, hi in ((0, n - new), (n - new, n)):
            seq.cache_append(k[at, lo:hi].cuda(), v[at, lo:hi].cuda(), kc, vc, table[at].cuda(), ints(hi).cuda())
    few = seq.paged_attention(q[:, :1].cuda(), kc, vc, table.cuda(), ints(*lens).cuda())
    many = seq.paged_attention(q[:, :new].cuda(), kc, vc, table.cuda(), ints(*lens).cuda())
    for b, n in enumerate(lens):
        page, slot = plain.slots(table[b], page_size, torch.arange(n))
        assert torch.equal(kc[page.cuda(), slot.cuda()].cpu(), k[b, :n]) and torch.equal(vc[page.cuda(), slot.cuda()].cpu(), v[b, :n])
        for got, rows in ((few, 1), (many, new)):
            pos = torch.arange(n)
            ok = plain.seen(pos[n - rows:], pos)
            heads2 = slice(0, 2)
            want = plain.attention(q[b, :rows, heads2], k[b, :n, heads2], v[b, :n, heads2], ok, dim**-0.5)
            within(got[b, :, heads2], *want["o"], what=(b, rows))


PAGED = [  # new rows, keys of each entry, page size, (q heads, kv heads, dim)
    (1, [1, 0, 37, 200], 16, (4, 4, 32)), (1, [513, 64], 64, (16, 4, 128)), (2, [2, 100, 31, 1], 5, (6, 2, 40)),
    (1, [3000], 24, (2, 1, 64)), (3, [65, 2, 700], 32, (4, 2, 96)), (1, [300] * 70, 128, (4, 4, 32)), (4, [7, 90], 1, (4, 1, 128)),
    (40, [40, 130, 41], 16, (4, 4, 32)), (150, [150, 400], 64, (4, 2, 64)), (33, [90, 20, 33], 7, (6, 2, 40)),
    (17, [5, 1000, 0], 100, (1, 1, 128)), (70, [300, 71], 3, (3, 1, 77)), (9, [9, 64], 16, (8, 4, 9)), (5, [2500, 40], 16, (8, 2, 48)),
    (200, [1024], 128, (2, 2, 96)), (1, [9000, 5], 64, (3, 3, 16)),
]


@pytest.mark.parametrize("band", [None, (1, 0), (9, 4), (64, 3), (200, 0), "all"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", range(len(PAGED)))
def test_paged_attention(seq, case, dtype, band):
    new, lens, page_size, (hq, hkv, dim) = PAGED[case]
    gen = generator(case, 7, len(str(band)))
    kc, vc, table = cache_case(gen, len(lens), lens, page_size, hkv, dim, dtype)
    how = {"causal": False} if band == "all" else {} if band is None else {"window": band[0], "sinks": band[1]}
    where = [t.cuda() for t in (kc, vc, table, ints(*lens))]
    kw = {n: torch.nan_to_num(t.float()).to(dtype) for n, t in (("k", kc), ("v", vc))}
    for packed in (False, True):
        if packed:   # fewer rows in some entries than in others
            counts = [max(0, new - i) for i in range(len(lens))]
            offsets = torch.tensor([1] + [1 + sum(counts[:i + 1]) for i in range(len(lens))], dtype=I32)
            q, more = normal(gen, sum(counts) + 3, hq, dim, dtype=dtype), {"q_offsets": offsets.cuda(), "max_q_len": new}
        else:
            q, offsets, more = normal(gen, len(lens), new, hq, dim, dtype=dtype), None, {}
        error = torch.zeros(1, dtype=I32).cuda()
        o, lse = seq.paged_attention(q.cuda(), *where, return_lse=True, error=error, **how, **more)
        seq.check(error)
        want = plain.paged_attention(q, kw["k"], kw["v"], table, lens, dim**-0.5, offsets, **how)
        within(o, *want["o"], what=(packed, "o"))
        within(lse, *want["lse"], what=(packed, "lse"))
        into = torch.full_like(o, 7.0)
        assert seq.paged_attention(q.cuda(), *where, out=into, **how, **more) is into
        if packed:   # rows of no entry are left as they were
            inside = slice(1, 1 + sum(counts))
            assert torch.equal(into[inside], o[inside])
            assert bool((into[:1] == 7).all()) and bool((into[1 + sum(counts):] == 7).all())
            assert not bool(o[:1].any()) and not bool(o[1 + sum(counts):].any())
        else:
            assert torch.equal(into, o)


def test_paged_attention_pages_that_entries_share(seq):
    """Two users whose histories begin alike, and a page named twice by one of them."""
    gen = generator(46)
    kc, vc, _ = cache_case(gen, 1, [64], 8, 2, 32, F32, garbage=0.0)
    kc, vc = normal(gen, *kc.shape), normal(gen, *vc.shape)
    table, lens = torch.tensor([[3, 1, 4, 0], [3, 1, 5, 5]], dtype=I32), [27, 32]
    for new in (1, 20):
        q = normal(gen, 2, new, 4, 32)
        got = seq.paged_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), ints(*lens).cuda())
        within(got, *plain.paged_attention(q, kc, vc, table, lens, 32**-0.5)["o"])


@pytest.mark.parametrize("window,sinks", [(1, 0), (9, 4), (100, 33), (64, 64)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("new,page_size,heads", [(1, 16, (4, 4, 32)), (2, 5, (6, 2, 40)), (50, 16, (4, 2, 64)),
                                                 (140, 7, (2, 2, 77)), (300, 64, (2, 1, 128)), (33, 1, (3, 3, 16))])
def test_paged_attention_pages_behind_the_window_may_be_gone(seq, new, page_size, heads, dtype, window, sinks):
    """Pages that no new row sees a key of are not read: neither their numbers nor what lies there now."""
    (hq, hkv, dim), lens = heads, [700, 300, 411]
    gen = generator(new, page_size, window, 47)
    kc, vc, table = cache_case(gen, len(lens), lens, page_size, hkv, dim, dtype)
    q = normal(gen, len(lens), new, hq, dim, dtype=dtype).cuda()
    how = {"window": window, "sinks": sinks}
    before = seq.paged_attention(q, kc.cuda(), vc.cuda(), table.cuda(), ints(*lens).cuda(), return_lse=True, **how)
    spare = kc.shape[0] - 1 if not bool(kc[-1].isfinite().any()) else int((~kc.isfinite().flatten(1).any(1)).nonzero()[0])
    for gone in (-1, 1 << 30, spare):   # spare: a page of NaN
        now = table.clone()
        for b, n in enumerate(lens):
            page = torch.arange(table.shape[1])
            first, last = page * page_size, (page + 1) * page_size - 1
            now[b, (first >= sinks) & (last < n - new - window + 1)] = gone
        assert bool((now != table).any())
        error = torch.zeros(1, dtype=I32).cuda()
        after = seq.paged_attention(q, kc.cuda(), vc.cuda(), now.cuda(), ints(*lens).cuda(), return_lse=True, error=error, **how)
        seq.check(error)
        assert torch.equal(after[0], before[0]) and torch.equal(after[1], before[1])


@pytest.mark.parametrize("factor,scale", [(30.0, None), (1e-3, 1e3), (1.0, 1e-6)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_paged_attention_large_and_small_scores(seq, dtype, factor, scale):
    gen = generator(47, factor)
    lens = [700, 33]
    kc, vc, table = cache_case(gen, 2, lens, 16, 2, 64, dtype, garbage=0.0)
    kc = (kc.float() * factor).to(dtype)
    for new in (1, 30):
        q = normal(gen, 2, new, 4, 64, dtype=dtype)
        got = seq.paged_attention(q.cuda(), kc.cuda(), vc.cuda(), table.cuda(), ints(*lens).cuda(), scale=scale)
        within(got, *plain.paged_attention(q, kc, vc, table, lens, 64**-0.5 if scale is None else scale)["o"])


# ----------------------------------------------------------- self attention
SELF = [  # batch, len, q heads, kv heads, dim
    (1, 1, 1, 1, 1), (3, 2, 2, 1, 16), (2, 63, 4, 2, 32), (3, 64, 2, 2, 40), (2, 65, 3, 1, 64), (1, 130, 2, 2, 77),
    (4, 257, 2, 1, 32), (1, 400, 1, 1, 128), (2, 200, 6, 2, 96), (1, 700, 2, 2, 8), (5, 33, 8, 2, 128),
]
BANDS = [None, (1, 0), (5, 3), (64, 0), (70, 40), (100, 130)]


def self_case(gen, shape, dtype, kind, spoil=True):
    b, l, hq, hkv, d = shape
    lens = [l] if b == 1 else [l] + [int(torch.randint(0, l + 1, (1,), generator=gen)) for _ in range(b - 2)] + [0]
    kw = {}
    if kind.startswith("packed"):
        kw["offsets"] = torch.tensor([2] + [2 + sum(lens[:i + 1]) for i in range(b)], dtype=I32)
        kw["max_len"] = l
        lead = (2 + sum(lens) + 3,)
    else:
        lead = (b, l)
        if kind != "all":
            kw["lens"] = torch.tensor(lens, dtype=I32)
    q, grad = normal(gen, *lead, hq, d, dtype=dtype), normal(gen, *lead, hq, d, dtype=dtype)
    k, v = normal(gen, *lead, hkv, d, dtype=dtype), normal(gen, *lead, hkv, d, dtype=dtype)
    if "mask" in kind:
        kw["kv_mask"] = torch.rand(lead, generator=gen) < 0.7
        kw["kv_mask"][..., :3] = False   # first rows whose mask leaves nothing
    away = torch.ones(lead, dtype=torch.bool)
    if "offsets" in kw:
        away[2:2 + sum(lens)] = False
    else:
        for i in range(b):
            away[i, :lens[i] if "lens" in kw else l] = False
    if spoil:   # what lies outside the histories, and masked keys
        for t in (q, k, v, grad):
            t[away] = math.nan
        if "kv_mask" in kw:
            for t in (k, v):
                t[~kw["kv_mask"]] = math.nan
                t.view(-1, hkv, d)[(~kw["kv_mask"].reshape(-1)).nonzero()[:1, 0]] = torch.finfo(dtype).min
    return q, k, v, grad, kw


def check_self(seq, q, k, v, grad, kw, band, what="", move=lambda t: t.cuda(), scale=None):
    how = {} if band is None else {"window": band[0], "sinks": band[1]}
    clean = [torch.where(t.isfinite() & (t.float().abs() < 1e30), t, 0.0) for t in (q, k, v, grad)]
    s = q.shape[-1] ** -0.5 if scale is None else scale
    want = plain.self_attention(*clean[:3], s, kw.get("lens"), kw.get("offsets"), kw.get("kv_mask"), grad=clean[3], **how)
    gpu = {**on_gpu(kw), **how, "scale": scale}
    qd, kd, vd, gd = (move(t) for t in (q, k, v, grad))
    o, lse = seq.self_attention(qd, kd, vd, return_lse=True, **gpu)
    within(o, *want["o"], what=(what, "o"))
    within(lse, *want["lse"], what=(what, "lse"))
    assert torch.equal(seq.self_attention(qd, kd, vd, **gpu), o)
    got = seq.self_attention_backward(gd, qd, kd, vd, o, lse, **gpu)
    for name, t in zip(("dq", "dk", "dv"), got):
        within(t, *want[name], what=(what, name))
    again = seq.self_attention_backward(gd, qd, kd, vd, o, lse, **gpu)
    assert all(torch.equal(a, b) for a, b in zip(got, again)), "two calls on equal inputs differ"


@pytest.mark.parametrize("kind", ["all", "lens", "packed", "mask", "packed mask"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SELF)
def test_self_attention(seq, shape, dtype, kind):
    gen = generator(*shape, len(kind))
    case = self_case(gen, shape, dtype, kind)
    for band in BANDS:
        check_self(seq, *case, band, what=(shape, kind, band))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,band,kind", [
    ((1, 3000, 1, 1, 64), (200, 4), "all"), ((1, 2500, 4, 1, 32), (100, 33), "mask"), ((2, 1500, 2, 2, 128), None, "lens"),
    ((1, 2000, 2, 1, 40), (300, 129), "all"), ((70, 150, 2, 2, 32), (30, 2), "packed"), ((140, 300, 1, 1, 64), (90, 100), "lens"),
    ((1, 4000, 1, 1, 16), (17, 128), "packed mask"), ((300, 40, 4, 4, 64), None, "lens"),
])
def test_self_attention_of_long_and_many_histories(seq, shape, band, kind, dtype):
    """Split keys and rows, sinks far from most rows, few of them and many, pairs placed by dies."""
    case = self_case(generator(*shape, 5), shape, dtype, kind)
    check_self(seq, *case, band, what=(shape, kind, band))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [32, 40, 77])
def test_self_attention_strides(seq, dim, dtype):
    case = self_case(generator(dim, 8), (3, 70, 4, 2, dim), dtype, "mask")
    for order in ((0, 2, 1, 3), (2, 1, 0, 3), (1, 0, 2, 3)):
        check_self(seq, *case, (20, 3), what=order, move=lambda t: strided_copy(t, order))
    fused = torch.randn(2, 50, 8, dim).to(dtype).cuda()   # q, k and v of one projection
    q, k, v = fused[:, :, :4], fused[:, :, 4:6], fused[:, :, 6:]
    o, lse = seq.self_attention(q, k, v, return_lse=True)
    assert torch.equal(o, seq.self_attention(q.contiguous(), k.contiguous(), v.contiguous()))
    one = torch.ones((), dtype=dtype).cuda().expand(o.shape)   # a gradient that is one number everywhere
    for a, b in zip(seq.self_attention_backward(one, q, k, v, o, lse),
                    seq.self_attention_backward(one.contiguous(), q, k, v, o, lse)):
        assert torch.equal(a, b)


def shifted(t, by):
    """The same values on the GPU in rows two elements apart, beginning `by` elements into an allocation."""
    wide = torch.zeros(t.numel() // t.shape[-1] * (t.shape[-1] + 2) + by, dtype=t.dtype, device="cuda")
    return wide[by:].view(*t.shape[:-1], t.shape[-1] + 2)[..., :t.shape[-1]].copy_(t)


@pytest.mark.parametrize("by", [0, 1, 2])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [2, 10, 38, 74, 126])
def test_attention_of_even_heads_that_are_not_eights(seq, dim, dtype, by):
    """Rows of pairs, and the same from an address that is not one of a pair."""
    gen = generator(dim, by, 48)
    for kind, band in (("all", (40, 3)), ("packed mask", None)):
        check_self(seq, *self_case(gen, (3, 210, 4, 2, dim), dtype, kind), band, (kind, band), lambda t: shifted(t, by))
    lens, new = [300, 41], 40
    kc, vc, table = cache_case(gen, 2, lens, 24, 2, dim, dtype)
    q = normal(gen, 2, new, 4, dim, dtype=dtype)
    clean = [torch.nan_to_num(t.float()).to(dtype) for t in (kc, vc)]
    for rows in (new, 1):
        got = seq.paged_attention(shifted(q[:, :rows], by), shifted(kc, by), shifted(vc, by), table.cuda(), ints(*lens).cuda(),
                                  window=70, sinks=2)
        want = plain.paged_attention(q[:, :rows], *clean, table, lens, dim**-0.5, window=70, sinks=2)
        within(got, *want["o"], what=rows)


@pytest.mark.parametrize("factor,scale", [(30.0, None), (1e-3, 1e3), (1.0, 1e-6)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_self_attention_large_and_small_scores(seq, dtype, factor, scale):
    q, k, v, grad, kw = self_case(generator(61, factor), (2, 300, 2, 2, 32), dtype, "lens", spoil=False)
    check_self(seq, q, (k.float() * factor).to(dtype), v, grad, kw, (100, 2), scale=scale)


def test_self_attention_rows_that_see_themselves_alone_leave_no_score_gradient(seq):
    """A window of 1: the weight is 1 whatever the score, so q and k have no gradient; what remains is the rounding of
    the weight (scores of 64 products, |s| < 8: 2^-16) times dP, not the rounding of out (2^-9)."""
    gen = generator(62)
    q, k, v, grad = (normal(gen, 3, 200, 2, 64, dtype=BF16) for _ in range(4))
    dev = [t.cuda() for t in (q, k, v)]
    o, lse = seq.self_attention(*dev, window=1, return_lse=True)
    assert torch.equal(o.cpu(), v)
    dq, dk, dv = (t.cpu().double() for t in seq.self_attention_backward(grad.cuda(), *dev, o, lse, window=1))
    dp = (grad.double() * v.double()).sum(-1).abs().max()
    size = 64**-0.5 * dp * max(t.double().abs().max() for t in (q, k))
    assert dq.abs().max() <= 2.0**-15 * size and dk.abs().max() <= 2.0**-15 * size
    within(dv, grad.double(), 2.0**-7 * grad.double().abs())


def test_self_attention_without_a_band_to_speak_of(seq):
    """A window no row fills, and sinks without a window, change no bit."""
    gen = generator(63)
    q, k, grad = (normal(gen, 2, 150, h, 32, dtype=BF16).cuda() for h in (4, 2, 4))
    want, lse = seq.self_attention(q, k, k, return_lse=True)
    grads = seq.self_attention_backward(grad, q, k, k, want, lse)
    for kw in ({"window": 150}, {"window": (1 << 31) + 5}, {"sinks": 9}, {"window": 150, "sinks": 1 << 40}):
        assert torch.equal(seq.self_attention(q, k, k, **kw), want), kw
        for a, b in zip(grads, seq.self_attention_backward(grad, q, k, k, want, lse, **kw)):
            assert torch.equal(a, b), kw
    few = seq.self_attention(q, k, k, window=149, sinks=1 << 40)   # every key is a sink
    within(few, want.cpu().double(), 2 * 2.0**-7 * (want.cpu().double().abs() + 1))


def test_self_attention_nothing(seq):
    for b, l in ((0, 5), (3, 0), (0, 0)):
        q = torch.empty(b, l, 2, 16).cuda()
        o, lse = seq.self_attention(q, q, q, return_lse=True)
        assert o.shape == q.shape and lse.shape == (b, l, 2)
        assert all(t.shape == q.shape for t in seq.self_attention_backward(o, q, q, q, o, lse))
    q = torch.randn(4, 2, 16).cuda()   # packed rows that no entry has
    for off, most in ((ints(0), 5), (ints(0, 0, 0), 0), (ints(0, 0, 0), 9), (ints(2, 2), 3)):
        o, lse = seq.self_attention(q, q, q, offsets=off.cuda(), max_len=most, return_lse=True)
        assert not bool(o.any()) and bool((lse == -math.inf).all())
        for t in seq.self_attention_backward(q, q, q, q, o, lse, offsets=off.cuda(), max_len=most):
            assert not bool(t.any())


def test_self_attention_lengths_out_of_range_are_recorded(seq):
    from dynamic_embedding_tables_amd import recis
    q = torch.randn(3, 20, 2, 16).cuda()
    rows = q.reshape(60, 2, 16)
    for kw in ({"lens": ints(20, 21, 3)}, {"lens": ints(-1, 4, 3)}, {"offsets": ints(0, 20, 61, 61), "max_len": 60},
               {"offsets": ints(-3, 20, 30, 60), "max_len": 60}, {"offsets": ints(0, 30, 20, 60), "max_len": 60},
               {"offsets": ints(0, 30, 40, 60), "max_len": 25}):
        x = rows if "offsets" in kw else q
        for error in (torch.zeros(1, dtype=I32).cuda(), None):
            o, lse = seq.self_attention(x, x, x, window=7, sinks=2, return_lse=True, error=error, **on_gpu(kw))
            if error is not None:
                with pytest.raises(recis.RecisError) as e:
                    seq.check(error)
                assert e.value.status == recis.RECIS_ERR_INVALID_ARG
                error.zero_()
            grads = seq.self_attention_backward(x, x, x, x, o, lse, window=7, sinks=2, error=error, **on_gpu(kw))
            if error is not None:
                with pytest.raises(recis.RecisError):
                    seq.check(error)
        if kw.get("max_len") == 25:   # the entry of too many is taken as empty: zeros
            for t in (o, *grads):
                assert not bool(t[:30].any()) and bool(t[30:].any())


def test_self_attention_beyond_32_bit_offsets(seq):
    b, l, heads, dim = 9, 4096, 512, 128   # 2.4e9 elements; the last entry's rows alone are looked at
    q = torch.zeros(b, l, heads, dim, dtype=BF16, device="cuda")
    gen = generator(64)
    part = [normal(gen, 150, 4, dim, dtype=BF16) for _ in range(4)]
    lens = torch.zeros(b, dtype=I32)
    lens[-1] = 150
    k, v, grad = q[..., :4, :], q[..., 4:8, :], torch.zeros_like(q)
    q[-1, :150, 508:], q[-1, :150, 0:4], q[-1, :150, 4:8] = part[0].cuda(), part[1].cuda(), part[2].cuda()
    grad[-1, :150, 508:] = part[3].cuda()
    kw = {"window": 40, "sinks": 3}
    # the last four query heads read the last key head
    o, lse = seq.self_attention(q, k, v, lens=lens.cuda(), return_lse=True, **kw)
    ok = plain.seen(torch.arange(150), torch.arange(150), 40, 3)
    want = plain.attention(part[0], part[1][:, 3:], part[2][:, 3:], ok, dim**-0.5, part[3])
    within(o[-1, :150, 508:], *want["o"])
    assert not bool(o[:-1].any())
    dq, dk, dv = seq.self_attention_backward(grad, q, k, v, o, lse, lens=lens.cuda(), **kw)
    within(dq[-1, :150, 508:], *want["dq"])
    within(dv[-1, :150, 3:], *want["dv"])
    assert not bool(dk[:-1].any()) and not bool(dv[:-1].any())


def test_self_attention_gradient_is_the_difference_quotient(seq):
    gen = generator(65)
    shape = (2, 90, 4, 2, 24)
    q, k, v, grad, kw = self_case(gen, shape, F32, "mask", spoil=False)
    how = {**on_gpu(kw), "window": 30, "sinks": 2}
    o, lse = seq.self_attention(q.cuda(), k.cuda(), v.cuda(), return_lse=True, **how)
    grads = seq.self_attention_backward(grad.cuda(), q.cuda(), k.cuda(), v.cuda(), o, lse, **how)

    def loss(*x):   # in 64 bits, from the definition
        got = plain.self_attention(*x, shape[-1] ** -0.5, kw["lens"], None, kw["kv_mask"], 30, 2)["o"][0]
        return (got * grad.double()).sum()

    h = 1e-4
    for i, g in enumerate(grads):
        step = normal(gen, *(q, k, v)[i].shape).double()
        ends = []
        for s in (h, -h):
            x = [t.double() for t in (q, k, v)]
            x[i] = x[i] + s * step
            ends.append(loss(*x))
        slope = float(ends[0] - ends[1]) / (2 * h)
        size = float((g.cpu().double().abs() * step.abs()).sum())
        # the quotient's own error is of third order in h, the gradient's that of its 32-bit sums
        assert abs(slope - float((g.cpu().double() * step).sum())) <= size * (300 * U32 + 10 * h * h)


# ------------------------------------------------------------- all together
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("window,sinks", [(None, 0), (40, 3)])
def test_serving_in_chunks_is_training_at_once(seq, dtype, window, sinks):
    """A history taken whole, as in training, and event by event or chunk by chunk over a paged cache, as in serving:
    every position's result is the definition's, within its bounds, on the turned heads of the other path."""
    gen = generator(71)
    hq, hkv, dim, page_size, n = 4, 2, 32, 16, [150, 97, 3]
    b, l = len(n), max(n)
    q, k, v = (normal(gen, b, l, h, dim, dtype=dtype).cuda() for h in (hq, hkv, hkv))
    freqs, lens = seq.rotary_frequencies(dim, scaling="parts", factor=4.0, original_len=64), ints(*n).cuda()
    tq, tk = seq.rotary(q, freqs, amplitude=1.1), seq.rotary(k, freqs, amplitude=1.1)
    whole = seq.self_attention(tq, tk, v, lens=lens, window=window, sinks=sinks)
    want = plain.self_attention(tq.cpu(), tk.cpu(), v.cpu(), dim**-0.5, n, window=window, sinks=sinks)["o"]
    within(whole, *want)
    width = -(-l // page_size)
    table = torch.randperm(b * width, generator=gen).view(b, width).to(I32).cuda()
    kc, vc = (torch.full((b * width, page_size, hkv, dim), math.nan, dtype=dtype).cuda() for _ in range(2))
    done, error = [0] * b, torch.zeros(1, dtype=I32).cuda()
    for chunk in (1, 1, 90, 5, 33, 1, 200):
        counts = [min(chunk, n[i] - done[i]) for i in range(b)]
        rows = [(i, slice(done[i], done[i] + counts[i])) for i in range(b)]
        done = [d + c for d, c in zip(done, counts)]
        off = torch.tensor([0] + [sum(counts[:i + 1]) for i in range(b)], dtype=I32).cuda()
        qc, kk, vv = (torch.cat([t[r] for r in rows]) for t in (q, k, v))
        now = ints(*done).cuda()
        turned = seq.cache_append(kk, vv, kc, vc, table, now, q=qc, q_offsets=off, freqs=freqs, amplitude=1.1, error=error)
        got = seq.paged_attention(turned, kc, vc, table, now, q_offsets=off, max_q_len=chunk, window=window, sinks=sinks,
                                  error=error)
        assert torch.equal(turned, torch.cat([tq[r] for r in rows]))
        for (i, at), part in zip(rows, got.split(counts)):
            within(part, want[0][i, at], want[1][i, at], what=(chunk, i))
    seq.check(error)
    assert done == n


def test_training_step_on_a_table_s_rows(seq):
    """Layer norm, turned heads and windowed self attention over packed histories, and back: the gradient of the norm's
    input against the difference quotient of the same steps in 64 bits."""
    gen = generator(72)
    n, heads, dim = [40, 0, 65], 2, 16
    off = ints(0, 40, 40, 105)
    x, grad = normal(gen, 105, heads * dim), normal(gen, 105, heads, dim)
    w, bias = normal(gen, heads * dim), normal(gen, heads * dim)
    freqs = seq.rotary_frequencies(dim)
    at = torch.cat([torch.arange(c) for c in n])
    kw = {"offsets": off.cuda(), "max_len": 65, "window": 20, "sinks": 2}
    y, mean, rstd = seq.layer_norm(x.cuda(), w.cuda(), bias.cuda())
    h = y.view(105, heads, dim)
    t = seq.rotary(h, freqs, at.cuda())
    o, lse = seq.self_attention(t, t, h, return_lse=True, **kw)
    dq, dk, dv = seq.self_attention_backward(grad.cuda(), t, t, h, o, lse, **kw)
    dh = seq.rotary_backward(dq + dk, freqs, at.cuda()) + dv
    dx, _, _ = seq.layer_norm_backward(dh.view(105, -1), x.cuda(), mean, rstd, w.cuda())

    def loss(x):
        xc = x - x.mean(-1, keepdim=True)
        y = xc / ((xc * xc).mean(-1, keepdim=True) + 1e-5).sqrt() * w.double() + bias.double()
        h = y.view(105, heads, dim)
        t = turned(h)
        return (plain.self_attention(t, t, h, dim**-0.5, None, off, None, 20, 2)["o"][0] * grad.double()).sum()

    def turned(h):
        angle = at.double()[:, None] * freqs.cpu()
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        a, b = h[..., : dim // 2], h[..., dim // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    step, e = normal(gen, *x.shape).double(), 1e-4
    slope = float(loss(x.double() + e * step) - loss(x.double() - e * step)) / (2 * e)
    size = float((dx.cpu().double().abs() * step.abs()).sum())
    assert abs(slope - float((dx.cpu().double() * step).sum())) <= size * (1000 * U32 + 100 * e * e)


def _all_calls(seq, gen, dtype=BF16):
    """Inputs of every call, and a step that makes them all."""
    s = {"q": normal(gen, 2, 70, 4, 32, dtype=dtype).cuda(), "k": normal(gen, 2, 70, 2, 32, dtype=dtype).cuda(),
         "g": normal(gen, 2, 70, 4, 32, dtype=dtype).cuda(), "lens": ints(70, 33).cuda(),
         "at": torch.arange(70).cuda(), "kc": torch.zeros(40, 16, 2, 32, dtype=dtype).cuda(),
         "vc": torch.zeros(40, 16, 2, 32, dtype=dtype).cuda(),
         "table": torch.arange(40, dtype=I32).view(2, 20).flip(1).contiguous().cuda(), "kv_lens": ints(75, 300).cuda()}
    freqs = seq.rotary_frequencies(32)

    def step(**kw):
        band = {"window": 20, "sinks": 3, **kw}
        t = seq.rotary(s["q"], freqs, s["at"], **kw)
        o, lse = seq.self_attention(t, s["k"], s["k"], lens=s["lens"], return_lse=True, **band)
        dq, dk, dv = seq.self_attention_backward(s["g"], t, s["k"], s["k"], o, lse, lens=s["lens"], **band)
        dx = seq.rotary_backward(dq, freqs, s["at"], **kw)
        turned = seq.cache_append(s["k"], s["k"], s["kc"], s["vc"], s["table"], s["kv_lens"], q=s["q"], freqs=freqs, **kw)
        many = seq.paged_attention(turned, s["kc"], s["vc"], s["table"], s["kv_lens"], **kw)
        one = turned[:, -1:]
        few = seq.paged_attention(one, s["kc"], s["vc"], s["table"], s["kv_lens"], **kw)
        return [t, o, lse, dx, dk, dv, turned, many, few]

    return s, step


def test_on_another_stream(seq):
    s, step = _all_calls(seq, generator(81))
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = step(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_captured_into_a_graph(seq):
    gen = generator(82)
    s, step = _all_calls(seq, gen)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):   # new values, lengths and pages in the same tensors, eager work in between
        for name in ("q", "k", "g"):
            s[name].copy_(normal(gen, *s[name].shape, dtype=BF16))
        s["lens"].copy_(ints(70 - 20 * i, 30 * i % 71))
        s["kv_lens"].copy_(ints(320 - 80 * i, 3 * i))
        s["table"].copy_(torch.randperm(40, generator=gen).view(2, 20).to(I32))
        s["at"].copy_(torch.arange(70) + 1000 * i)
        kc, vc = s["kc"].clone(), s["vc"].clone()
        want = step()
        s["kc"].copy_(kc), s["vc"].copy_(vc)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, held):
            assert torch.equal(a, b), i


def test_inputs_that_require_a_gradient_are_warned_about(seq):
    gen = generator(83)
    q, freqs = normal(gen, 2, 5, 2, 16).cuda(), seq.rotary_frequencies(16)
    kc = torch.zeros(4, 8, 2, 16).cuda()
    where = (torch.arange(2, dtype=I32).view(2, 1).cuda(), ints(5, 5).cuda())
    calls = [lambda a: seq.rotary(a, freqs), lambda a: seq.self_attention(a, q, q), lambda a: seq.self_attention(q, a, q),
             lambda a: seq.self_attention(q, q, a), lambda a: seq.cache_append(a, q, kc, kc.clone(), *where),
             lambda a: seq.cache_append(q, a, kc, kc.clone(), *where), lambda a: seq.paged_attention(a, kc, kc, *where)]
    for call in calls:
        with pytest.warns(UserWarning, match="gradient|backward"):
            call(q.clone().requires_grad_())
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with torch.no_grad():
                call(q.clone().requires_grad_())


def test_refusals_on_tensors(seq):
    q, k = torch.randn(2, 5, 4, 16).cuda(), torch.randn(2, 5, 2, 16).cuda()
    freqs = seq.rotary_frequencies(16)
    off = ints(0, 5, 10).cuda()
    packed = k.reshape(10, 2, 16)
    kc, vc = torch.zeros(6, 8, 2, 16).cuda(), torch.zeros(6, 8, 2, 16).cuda()
    table, lens = torch.zeros(2, 3, dtype=I32).cuda(), ints(5, 5).cuda()
    o, lse = seq.self_attention(q, k, k, return_lse=True)
    refused = [
        lambda: seq.rotary(q.half(), freqs), lambda: seq.rotary(q, freqs.float()), lambda: seq.rotary(q[0, 0], freqs),
        lambda: seq.rotary(q, seq.rotary_frequencies(18)), lambda: seq.rotary(q, freqs, ints(0, 1, 2, 3, 4).cuda()),
        lambda: seq.rotary(q, freqs, torch.arange(4).cuda()), lambda: seq.rotary(q, freqs, out=q[:1]),
        lambda: seq.rotary(q, freqs, out=q[..., :1].expand(q.shape)), lambda: seq.rotary(q, freqs.cpu()),
        lambda: seq.cache_append(k, k[:, :4], kc, vc, table, lens), lambda: seq.cache_append(k, k, kc, vc[:5], table, lens),
        lambda: seq.cache_append(k.to(BF16), k.to(BF16), kc, vc, table, lens),
        lambda: seq.cache_append(k, k, kc, vc, table.long(), lens), lambda: seq.cache_append(k, k, kc, vc, table[:1], lens),
        lambda: seq.cache_append(k, k, kc, vc, table, lens.long()), lambda: seq.cache_append(k, k, kc, vc, table, lens[:1]),
        lambda: seq.cache_append(k, k, kc, vc, table, lens, q=q), lambda: seq.cache_append(packed, packed, kc, vc, table, lens),
        lambda: seq.cache_append(k, k, kc, vc, table, lens, q_offsets=off),
        lambda: seq.cache_append(k, k, kc[:1].expand(6, 8, 2, 16), vc, table, lens),
        lambda: seq.cache_append(k, k, kc.transpose(2, 3).contiguous().transpose(2, 3), vc, table, lens),
        lambda: seq.cache_append(k, k, kc, vc, table, lens, q=q[:, :4], freqs=freqs),
        lambda: seq.paged_attention(q, kc, vc, table, lens, window=0), lambda: seq.paged_attention(q, kc, vc, table, lens, sinks=-1),
        lambda: seq.paged_attention(q, kc, vc, table, lens, causal=False, window=4),
        lambda: seq.paged_attention(q, kc, vc, table, lens, q_offsets=off), lambda: seq.paged_attention(q, kc, vc, table, lens, max_q_len=5),
        lambda: seq.paged_attention(q[0], kc, vc, table, lens, q_offsets=off[:2]),
        lambda: seq.paged_attention(q.to(BF16), kc, vc, table, lens), lambda: seq.paged_attention(q[..., :8], kc, vc, table, lens),
        lambda: seq.paged_attention(q, kc, vc, table, lens, out=q[:1]), lambda: seq.paged_attention(q, kc[0], vc[0], table, lens),
        lambda: seq.paged_attention(q, kc, vc, table, lens, error=torch.zeros(2, dtype=I32).cuda()),
        lambda: seq.self_attention(q, k, k[:1]), lambda: seq.self_attention(q, k[:, :4], k[:, :4]),
        lambda: seq.self_attention(q, k, k, lens=lens.long()), lambda: seq.self_attention(q, k, k, max_len=5),
        lambda: seq.self_attention(q, k, k, offsets=off, max_len=5), lambda: seq.self_attention(q, k, k, window=0),
        lambda: seq.self_attention(packed, packed, packed, offsets=off),
        lambda: seq.self_attention(q, k, k, kv_mask=torch.ones(2, 4, dtype=torch.bool).cuda()),
        lambda: seq.self_attention(q, k.to(BF16), k.to(BF16)), lambda: seq.self_attention(q.cpu(), k, k),
        lambda: seq.self_attention_backward(q, q, k, k, o, lse[:1]), lambda: seq.self_attention_backward(q, q, k, k, o[:1], lse),
        lambda: seq.self_attention_backward(q, q, k, k, o, lse.double()),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(ValueError):
            call()
            print("not refused:", i)
    from dynamic_embedding_tables_amd import recis
    wide = torch.randn(1, 2, 1, 200).cuda()
    for call in (lambda: seq.self_attention(wide, wide, wide), lambda: seq.self_attention(q, k, k, scale=0.0),
                 lambda: seq.self_attention(torch.randn(1, 2, 3, 8).cuda(), *[torch.randn(1, 2, 2, 8).cuda()] * 2),
                 lambda: seq.paged_attention(q[:, :, :3], kc, vc, table, lens), lambda: seq.rotary(q, freqs, amplitude=math.nan),
                 lambda: seq.rotary(torch.randn(1, 1, 1, 2000).cuda(), freqs)):
        with pytest.raises(recis.RecisError):
            call()
