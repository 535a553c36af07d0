"""The sequence operators on the GPU against their definitions in 64 bits, at
the sizes, layouts and masks where they can go wrong (bounds: sequence_plain)."""
import math
import warnings

import pytest
import torch

import sequence_plain as plain
from sequence_plain import within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
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


def normal(gen, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype)


def generator(*key):
    return torch.Generator().manual_seed(abs(hash(key)) % (1 << 31) if not key else sum(
        (i + 1) * int(k) for i, k in enumerate(key)) + 17)


# ---------------------------------------------------------------- embedding
EMBED = [  # tokens, rows, dim
    (1, 1, 1), (1, 50, 8), (7, 3, 5), (64, 100, 16), (129, 1000, 33), (1024, 5000, 40), (1025, 5000, 40), (700, 3, 128), (1000, 4100, 8), (1000, 17, 64), (4097, 257, 100),
    (5000, 70000, 30), (300, 9, 1030), (2048, 65535, 128), (9000, 1, 24),
]


def tokens_of(gen, n, rows):
    """Many tokens on few rows, padding among them."""
    t = (torch.rand(n, generator=gen) ** 4 * rows).long().clamp(0, rows - 1)
    t[torch.rand(n, generator=gen) < 0.1] = -1
    return t


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,rows,dim", EMBED)
def test_embed(seq, n, rows, dim, dtype):
    gen = generator(n, rows, dim)
    t, w = tokens_of(gen, n, rows), normal(gen, rows, dim, dtype=dtype)
    out = seq.embed(t.cuda(), w.cuda(), scale=3.7)
    # one product in float32 and one rounding: the same bits as torch's
    want = torch.where((t >= 0)[:, None], w.float()[t.clamp_min(0)] * torch.tensor(3.7), 0).to(dtype)
    assert torch.equal(out.cpu(), want)
    within(out, plain.embed(t, w, 3.7), (2 * plain.U32 + plain.U[dtype]) * want.double().abs() + plain.TINY)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,rows,dim", EMBED)
def test_embed_backward(seq, n, rows, dim, dtype):
    gen = generator(n, rows, dim, 1)
    t, g = tokens_of(gen, n, rows), normal(gen, n, dim, dtype=dtype)
    for out_dtype in DTYPES:
        got = seq.embed_backward(t.cuda(), g.cuda(), rows, scale=0.3, dtype=out_dtype)
        assert got.dtype == out_dtype
        within(got, *plain.embed_backward(t, g, rows, 0.3, out_dtype), what=(n, rows, dim))
        again = seq.embed_backward(t.cuda(), g.cuda(), rows, scale=0.3, dtype=out_dtype)
        assert torch.equal(got, again), "two calls on equal inputs differ"


@pytest.mark.parametrize("law", ["one row", "all padding", "runs", "descending", "two ends"])
def test_embed_backward_token_orders(seq, law):
    gen = generator(3, len(law))
    n, rows, dim = 20000, 3000, 64
    t = {"one row": torch.full((n,), 1234), "all padding": torch.full((n,), -1),
         "runs": torch.arange(n) // 137, "descending": rows - 1 - torch.arange(n) * rows // n,
         "two ends": torch.where(torch.arange(n) % 2 == 0, 0, rows - 1)}[law]
    g = normal(gen, n, dim)
    got = seq.embed_backward(t.cuda(), g.cuda(), rows)
    within(got, *plain.embed_backward(t, g, rows, 1.0, F32), what=law)


def test_embed_no_tokens(seq):
    w = torch.randn(10, 4).cuda()
    none = torch.empty(0, dtype=torch.int64).cuda()
    assert seq.embed(none, w).shape == (0, 4)
    assert torch.equal(seq.embed_backward(none, torch.empty(0, 4).cuda(), 10), torch.zeros(10, 4).cuda())


def test_embed_strides_and_shapes(seq):
    gen = generator(4)
    big = normal(gen, 40, 50)
    for w in (big[:, 3:20], big[:, 4:20], big[::2, :16], big.t()):   # offset, aligned, strided rows, strided elements
        t = tokens_of(gen, 60, w.shape[0]).reshape(5, 12)
        wide = torch.full((60, 70), 7.0).cuda()
        wd = big.cuda().as_strided(w.shape, w.stride(), w.storage_offset())
        got = seq.embed(t.cuda(), wd, scale=2.0)
        assert got.shape == (5, 12, w.shape[1])
        assert torch.equal(got.cpu(), plain.embed(t, w, 2.0).float())
        into = wide[:, 2:2 + w.shape[1]]
        seq.embed(t.reshape(-1).cuda(), wd, scale=2.0, out=into)
        assert torch.equal(into.cpu(), plain.embed(t.reshape(-1), w, 2.0).float())
        assert bool((wide[:, :2] == 7).all()) and bool((wide[:, 2 + w.shape[1]:] == 7).all())
    t = tokens_of(gen, 50, 40)
    for g in (normal(gen, 50, 33)[:, 1:], normal(gen, 1, 32).expand(50, 32), normal(gen, 100, 32)[::2]):
        gd = g.cuda() if g.stride(0) else g[:1].cuda().expand(50, 32)
        wide = torch.full((40, 40), 7.0).cuda()
        seq.embed_backward(t.cuda(), gd, 40, out=wide[:, 5:37])
        within(wide[:, 5:37], *plain.embed_backward(t, g.contiguous(), 40, 1.0, F32))
        assert bool((wide[:, :5] == 7).all()) and bool((wide[:, 37:] == 7).all())


def test_embed_tokens_out_of_range_are_recorded(seq):
    from dynamic_embedding_tables_amd import recis
    w = torch.randn(10, 8).cuda()
    t = torch.tensor([3, 10, 1 << 40, -5, 9]).cuda()
    for call in (lambda e: seq.embed(t, w, error=e), lambda e: seq.embed_backward(t, torch.ones(5, 8).cuda(), 10, error=e)):
        error = torch.zeros(1, dtype=torch.int32).cuda()
        out = call(error)
        with pytest.raises(recis.RecisError) as e:
            seq.check(error)
        assert e.value.status == recis.RECIS_ERR_KEY_RANGE
        assert bool(torch.isfinite(out).all())
        call(None)   # nowhere to record it: still nothing out of bounds
    error = torch.zeros(1, dtype=torch.int32).cuda()
    seq.embed(t[:1], w, error=error)
    seq.check(error)
    assert torch.equal(seq.embed(t, w)[[1, 2, 3]], torch.zeros(3, 8).cuda())


def test_embed_values_that_are_not_finite(seq):
    w = torch.tensor([[1.0, math.inf], [math.nan, -math.inf], [2.0, 3.0]]).cuda()
    t = torch.tensor([0, 1, 2, -1]).cuda()
    within(seq.embed(t, w), plain.embed(t.cpu(), w.cpu(), 1.0), torch.tensor(0.0))
    g = torch.tensor([[math.inf, 1.0], [1.0, math.nan], [5.0, 6.0], [math.nan, math.nan]])
    got = seq.embed_backward(t, g.cuda(), 4).cpu()
    assert got[0].tolist() == [math.inf, 1.0] and got[1, 0] == 1 and math.isnan(got[1, 1])
    assert got[2].tolist() == [5.0, 6.0] and got[3].tolist() == [0.0, 0.0]


def test_embed_beyond_32_bit_offsets(seq):
    rows, dim = (1 << 24) + 64, 128   # 2^31 + 8192 elements
    t = torch.tensor([rows - 1, 5, -1, rows - 64, 1 << 23])
    w = torch.zeros(rows, dim, dtype=BF16, device="cuda")
    w[t[t >= 0].cuda()] = torch.randn(4, dim, device="cuda").to(BF16)
    out = seq.embed(t.cuda(), w)
    for i, row in enumerate(t.tolist()):
        assert torch.equal(out[i], w[row] if row >= 0 else torch.zeros_like(out[i]))
    del w
    g = torch.randn(5, dim, device="cuda").to(BF16)
    dw = seq.embed_backward(t.cuda(), g, rows)
    for i, row in enumerate(t.tolist()):
        if row >= 0:
            assert torch.equal(dw[row], g[i])
            dw[row] = 0
    assert not bool(dw.any())


def test_embed_gradient_is_the_difference_quotient(seq):
    gen = generator(6)
    t, w, g = tokens_of(gen, 500, 40), normal(gen, 40, 16), normal(gen, 500, 16)
    way = normal(gen, 40, 16)
    h = 0.25   # the operator is linear: any step will do
    hi, lo = (seq.embed(t.cuda(), (w + s * h * way).cuda(), scale=1.5).cpu().double() for s in (1, -1))
    slope = ((hi - lo) * g.double()).sum() / (2 * h)
    dw = seq.embed_backward(t.cuda(), g.cuda(), 40, scale=1.5).cpu().double()
    noise = 4 * plain.U32 * (hi.abs() * g.double().abs()).sum() / h
    bound = plain.embed_backward(t, g, 40, 1.5, F32)[1]
    assert abs(slope - (dw * way.double()).sum()) <= noise + (bound * way.double().abs()).sum()


# --------------------------------------------------------------- layer norm
NORM = [(1, 1), (3, 2), (5, 7), (64, 16), (33, 128), (7, 100), (129, 64), (17, 777), (4, 1000), (9, 1024), (3, 2500),
        (2, 4100), (5, 8192), (2, 16384), (1, 16383), (2100, 128), (4099, 40)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,dim", NORM)
def test_layer_norm(seq, m, dim, dtype):
    gen = generator(m, dim, 2)
    x = normal(gen, m, dim, dtype=dtype, scale=2.0) + 0.5
    for w_dtype in DTYPES:
        w, b = normal(gen, dim, dtype=w_dtype), normal(gen, dim, dtype=w_dtype)
        y, mean, rstd = seq.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=1e-5)
        want = plain.layer_norm(x, w, b, 1e-5, dtype)
        for name, got in (("y", y), ("mean", mean), ("rstd", rstd)):
            within(got, *want[name], what=(name, m, dim))
        assert torch.equal(seq.layer_norm(x.cuda(), w.cuda(), b.cuda(), eps=1e-5, stats=False), y)
    y, _, _ = seq.layer_norm(x.cuda())
    within(y, *plain.layer_norm(x, None, None, 1e-5, dtype)["y"])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,dim", NORM)
def test_layer_norm_backward(seq, m, dim, dtype):
    gen = generator(m, dim, 3)
    x, g = normal(gen, m, dim, dtype=dtype, scale=2.0) + 0.5, normal(gen, m, dim, dtype=dtype)
    for w_dtype in DTYPES:
        w = normal(gen, dim, dtype=w_dtype)
        _, mean, rstd = seq.layer_norm(x.cuda(), w.cuda())
        got = seq.layer_norm_backward(g.cuda(), x.cuda(), mean, rstd, w.cuda())
        want = plain.layer_norm_backward(g, x, w, 1e-5, dtype, w_dtype)
        for name, t in zip(("dx", "dw", "db"), got):
            within(t, *want[name], what=(name, m, dim))
        again = seq.layer_norm_backward(g.cuda(), x.cuda(), mean, rstd, w.cuda())
        assert all(torch.equal(a, b) for a, b in zip(got, again)), "two calls on equal inputs differ"
    dx, dw, db = seq.layer_norm_backward(g.cuda(), x.cuda(), mean, rstd, need_weight=False)
    assert dw is None and db is None
    within(dx, *plain.layer_norm_backward(g, x, None, 1e-5, dtype, F32)["dx"])


def test_layer_norm_no_rows(seq):
    x = torch.empty(0, 16).cuda()
    y, mean, rstd = seq.layer_norm(x)
    assert y.shape == (0, 16) and mean.shape == (0,)
    dx, dw, db = seq.layer_norm_backward(x, x, mean, rstd)
    assert dx.shape == (0, 16) and not bool(dw.any()) and not bool(db.any())


def test_layer_norm_constant_rows_and_large_means(seq):
    x = torch.cat([torch.full((2, 96), 3.25), torch.zeros(1, 96), 4096 + torch.randn(3, 96, generator=generator(7))])
    y, mean, rstd = seq.layer_norm(x.cuda())
    want = plain.layer_norm(x, None, None, 1e-5, F32)
    assert bool((y[:3] == 0).all()) and mean[:3].tolist() == [3.25, 3.25, 0.0]
    for name, got in (("y", y), ("mean", mean), ("rstd", rstd)):
        within(got, *want[name], what=name)


def test_layer_norm_rows_that_are_not_finite_stay_alone(seq):
    gen = generator(8)
    for dim in (128, 777):
        x = normal(gen, 6, dim)
        x[1, 3], x[4, 0] = math.nan, math.inf
        y, mean, rstd = seq.layer_norm(x.cuda())
        want = plain.layer_norm(x[[0, 2, 3, 5]], None, None, 1e-5, F32)["y"]
        within(y[[0, 2, 3, 5]], *want)
        assert bool(torch.isnan(y[[1, 4]]).all())
        dx, _, _ = seq.layer_norm_backward(torch.ones_like(y), x.cuda(), mean, rstd)
        assert bool(torch.isfinite(dx[[0, 2, 3, 5]]).all())


def test_layer_norm_strides_and_in_place(seq):
    gen = generator(9)
    big = normal(gen, 30, 200)
    for x in (big[:, 4:132], big[:, 3:131], big[::3, :128]):
        xd = big.cuda().as_strided(x.shape, x.stride(), x.storage_offset())
        want = plain.layer_norm(x, None, None, 1e-5, F32)
        y, mean, rstd = seq.layer_norm(xd)
        within(y, *want["y"])
        g = normal(gen, *x.shape)
        dx, dw, _ = seq.layer_norm_backward(g.cuda().expand_as(y), xd, mean, rstd)
        back = plain.layer_norm_backward(g, x, None, 1e-5, F32, F32)
        within(dx, *back["dx"])
        within(dw, *back["dw"])
        one = seq.layer_norm_backward(g[:1].cuda().expand_as(y), xd, mean, rstd)  # a broadcast gradient
        within(one[1], *plain.layer_norm_backward(g[:1].expand_as(x), x, None, 1e-5, F32, F32)["dw"])
        seq.layer_norm(xd, out=xd)
        within(xd, *want["y"])
    x = normal(gen, 4, 5, 6, 64)
    y, mean, rstd = seq.layer_norm(x.cuda())
    assert y.shape == x.shape and mean.shape == rstd.shape == (4, 5, 6)


def test_layer_norm_beyond_32_bit_offsets(seq):
    store = torch.zeros((1 << 31) + 256, dtype=BF16, device="cuda")
    x = store.as_strided((2, 128), (1 << 31, 1))
    gen = generator(10)
    host = normal(gen, 2, 128, dtype=BF16)
    x.copy_(host)
    y, mean, rstd = seq.layer_norm(x)
    within(y, *plain.layer_norm(host, None, None, 1e-5, BF16)["y"])
    dx, _, _ = seq.layer_norm_backward(x, x, mean, rstd)
    within(dx, *plain.layer_norm_backward(host, host, None, 1e-5, BF16, F32)["dx"])


def test_layer_norm_gradient_is_the_difference_quotient(seq):
    gen = generator(11)
    x, w, b, g = normal(gen, 20, 48), normal(gen, 48), normal(gen, 48), normal(gen, 20, 48)
    way, h = normal(gen, 20, 48), 2.0**-6

    def loss(f, s):
        return (f(x + s * h * way) * g.double()).sum() / (2 * h)

    def kernel(z):
        return seq.layer_norm(z.cuda(), w.cuda(), b.cuda(), stats=False).cpu().double()

    def exact(z):
        return plain.layer_norm(z, w, b, 1e-5, F32)["y"][0]

    slope = loss(kernel, 1) - loss(kernel, -1)
    _, mean, rstd = seq.layer_norm(x.cuda(), w.cuda(), b.cuda())
    dx, dw, db = seq.layer_norm_backward(g.cuda(), x.cuda(), mean, rstd, w.cuda())
    along = (dx.cpu().double() * way.double()).sum()
    back = plain.layer_norm_backward(g, x, w, 1e-5, F32, F32)
    step = abs(loss(exact, 1) - loss(exact, -1) - (back["dx"][0] * way.double()).sum())  # the step's own error
    noise = sum((plain.layer_norm(x + s * h * way, w, b, 1e-5, F32)["y"][1] * g.double().abs()).sum() / (2 * h)
                for s in (1, -1))
    assert abs(slope - along) <= step + noise + (back["dx"][1] * way.double().abs()).sum()
    # in w and b the operator is linear
    wayw = normal(gen, 48)
    hi, lo = (seq.layer_norm(x.cuda(), (w + s * wayw).cuda(), b.cuda(), stats=False).cpu().double() for s in (1, -1))
    slope = ((hi - lo) * g.double()).sum() / 2
    noise = (plain.layer_norm(x, w + wayw.abs(), b, 1e-5, F32)["y"][1] * g.double().abs()).sum() * 4
    assert abs(slope - (dw.cpu().double() * wayw.double()).sum()) <= noise + (back["dw"][1] * wayw.abs().double()).sum()


# ---------------------------------------------------------- cross attention
ATTN = [  # batch, q_len, kv_len, q_heads, kv_heads, head_dim
    (1, 1, 1, 1, 1, 1), (2, 1, 200, 4, 4, 32), (3, 3, 65, 4, 2, 40), (2, 17, 64, 2, 1, 128), (2, 70, 130, 6, 2, 64),
    (1, 129, 257, 2, 2, 20), (2, 1, 1500, 8, 2, 128), (5, 33, 31, 1, 1, 7), (1, 200, 100, 3, 3, 64), (3, 2, 700, 4, 1, 96),
    (2, 40, 16, 4, 2, 33), (9, 5, 300, 2, 2, 16), (2, 37, 150, 2, 1, 48), (2, 66, 140, 2, 2, 96), (1, 20, 90, 2, 1, 88),
    (2, 1, 400, 4, 1, 80), (2, 3, 333, 2, 2, 48),
]
KINDS = ["all", "lens", "packed", "mask", "packed mask"]


def attn_case(gen, shape, dtype, kind, spoil=True):
    """Host tensors and the call's keyword arguments; keys that do not count hold NaN and the type's lowest value."""
    b, lq, lk, hq, hkv, d = shape
    q = normal(gen, b, lq, hq, d, dtype=dtype)
    kw, lens = {}, [lk]
    if b > 1:
        lens = [lk] + [int(torch.randint(0, lk + 1, (1,), generator=gen)) for _ in range(b - 2)] + [0]
    if kind.startswith("packed"):
        front, back = 2, 3
        kw["kv_offsets"] = torch.tensor([front] + [front + sum(lens[:i + 1]) for i in range(b)], dtype=torch.int32)
        kw["max_kv_len"] = lk
        shape_k = (front + sum(lens) + back, hkv, d)
    else:
        shape_k = (b, lk, hkv, d)
        if kind != "all":
            kw["kv_lens"] = torch.tensor(lens, dtype=torch.int32)
    k, v = normal(gen, *shape_k, dtype=dtype), normal(gen, *shape_k, dtype=dtype)
    if "mask" in kind:
        m = torch.rand(shape_k[:-2], generator=gen) < 0.7
        if kind == "mask" and b > 2:
            m[1] = False   # an entry whose mask leaves nothing
        kw["kv_mask"] = m
    kept = plain.kept_keys(k, kw.get("kv_lens"), kw.get("kv_offsets"), kw.get("kv_mask"))
    if spoil:
        away = torch.ones(shape_k[:-2], dtype=torch.bool)
        for i, rows in enumerate(kept):
            (away if kind.startswith("packed") else away[i])[rows] = False
        for t in (k, v):
            t[away] = math.nan
            first = away.nonzero()[:1]
            if len(first):
                t[tuple(first[0])] = torch.finfo(dtype).min
    return q, k, v, kw, kept


def on_gpu(kw):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in kw.items()}


def check_attention(seq, q, k, v, kw, kept, scale=None, grad=None, move=lambda t: t.cuda(), what=""):
    packed = "kv_offsets" in kw
    s = q.shape[-1] ** -0.5 if scale is None else scale
    want = plain.attention(q, torch.nan_to_num(k.float()).to(k.dtype), torch.nan_to_num(v.float()).to(v.dtype), s, kept,
                           packed, grad)
    gpu = on_gpu(kw)
    qd, kd, vd = move(q), move(k), move(v)
    o, lse = seq.cross_attention(qd, kd, vd, return_lse=True, scale=scale, **gpu)
    within(o, *want["o"], what=(what, "o"))
    within(lse, *want["lse"], what=(what, "lse"))
    assert torch.equal(seq.cross_attention(qd, kd, vd, scale=scale, **gpu), o)
    if grad is not None:
        got = seq.cross_attention_backward(move(grad), qd, kd, vd, o, lse, scale=scale, **gpu)
        for name, t in zip(("dq", "dk", "dv"), got):
            within(t, *want[name], what=(what, name))
        again = seq.cross_attention_backward(move(grad), qd, kd, vd, o, lse, scale=scale, **gpu)
        assert all(torch.equal(a, b) for a, b in zip(got, again)), "two calls on equal inputs differ"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", ATTN)
def test_cross_attention(seq, shape, dtype, kind):
    gen = generator(*shape, len(kind))
    q, k, v, kw, kept = attn_case(gen, shape, dtype, kind)
    check_attention(seq, q, k, v, kw, kept, grad=normal(gen, *q.shape, dtype=dtype), what=(shape, kind))


def test_cross_attention_single_keys_leave_no_score_gradient(seq):
    """One key: the weight is 1 whatever the score, so q and k have no gradient; what remains is the rounding of the
    weight (scores of 64 products, |s| < 8: 2^-16) times dP, not the rounding of out (2^-9)."""
    gen = generator(18)
    q, k, v, grad = (normal(gen, 4, n, 2, 64, dtype=BF16) for n in (7, 1, 1, 7))
    dev = [t.cuda() for t in (q, k, v)]
    o, lse = seq.cross_attention(*dev, return_lse=True)
    dq, dk, dv = (t.cpu().double() for t in seq.cross_attention_backward(grad.cuda(), *dev, o, lse))
    dp = torch.einsum("bqhd,bkhd->bqhk", grad.double(), v.double()).abs().max()
    size = 64**-0.5 * dp * max(t.double().abs().max() for t in (q, k))
    assert dq.abs().max() <= 2.0**-15 * size and dk.abs().max() <= 7 * 2.0**-15 * size
    within(dv[:, 0], grad.double().sum(1), 9 * 2.0**-8 * grad.double().abs().sum(1))


def test_cross_attention_no_keys_no_queries(seq):
    for q_len, kv_len in ((3, 0), (0, 5), (0, 0)):
        q, k = torch.randn(2, q_len, 2, 16).cuda(), torch.randn(2, kv_len, 2, 16).cuda()
        o, lse = seq.cross_attention(q, k, k, return_lse=True)
        assert not bool(o.any()) and bool((lse == -math.inf).all())
        dq, dk, dv = seq.cross_attention_backward(torch.ones_like(q), q, k, k, o, lse)
        assert not bool(dq.any()) and not bool(dk.any()) and not bool(dv.any())
    q, k = torch.randn(0, 3, 2, 16).cuda(), torch.randn(0, 5, 2, 16).cuda()
    assert seq.cross_attention(q, k, k).shape == q.shape
    off = torch.zeros(3, dtype=torch.int32).cuda()
    q, k = torch.randn(2, 3, 2, 16).cuda(), torch.randn(4, 2, 16).cuda()   # packed rows that no entry has
    for most in (0, 7):
        o, lse = seq.cross_attention(q, k, k, kv_offsets=off, max_kv_len=most, return_lse=True)
        assert not bool(o.any())
        _, dk, dv = seq.cross_attention_backward(q, q, k, k, o, lse, kv_offsets=off, max_kv_len=most)
        assert not bool(dk.any()) and not bool(dv.any())


@pytest.mark.parametrize("dtype", DTYPES)
def test_cross_attention_strides(seq, dtype):
    gen = generator(12)
    shape = (2, 9, 70, 4, 2, 32)
    q, k, v, kw, kept = attn_case(gen, shape, dtype, "lens")
    grad = normal(gen, *q.shape, dtype=dtype)

    def heads_first(t):
        return t.transpose(1, 2).contiguous().cuda().transpose(1, 2)

    def unaligned(t):   # every row starts two bytes or four off
        wide = torch.zeros(*t.shape[:-1], t.shape[-1] + 3, dtype=t.dtype).cuda()
        wide[..., 1:-2] = t.cuda()
        return wide[..., 1:-2]

    def elements_apart(t):
        wide = torch.zeros(*t.shape, 2, dtype=t.dtype).cuda()
        wide[..., 0] = t.cuda()
        return wide[..., 0]

    for move in (heads_first, unaligned, elements_apart):
        check_attention(seq, q, k, v, kw, kept, grad=grad, move=move, what=move.__name__)
    one = normal(gen, 1, 1, 1, 32, dtype=dtype)   # a broadcast gradient
    qd, kd, vd = q.cuda(), k.cuda(), v.cuda()
    o, lse = seq.cross_attention(qd, kd, vd, return_lse=True, **on_gpu(kw))
    got = seq.cross_attention_backward(one.cuda().expand(q.shape), qd, kd, vd, o, lse, **on_gpu(kw))
    clean = [torch.nan_to_num(t.float()).to(dtype) for t in (k, v)]
    want = plain.attention(q, *clean, 32**-0.5, kept, False, one.expand(q.shape))
    for name, t in zip(("dq", "dk", "dv"), got):
        within(t, *want[name], what=name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("factor,scale", [(1.0, 8.0), (30.0, None), (1e-4, 1e-3)])
def test_cross_attention_large_and_small_scores(seq, factor, scale, dtype):
    gen = generator(13, int(factor * 10))
    q, k, v, kw, kept = attn_case(gen, (2, 20, 150, 2, 2, 24), dtype, "mask")
    check_attention(seq, (q.float() * factor).to(dtype), k, v, kw, kept, scale=scale,
                    grad=normal(gen, *q.shape, dtype=dtype))


def test_cross_attention_infinite_scores_and_values(seq):
    q = torch.ones(1, 1, 1, 8)
    k = torch.zeros(1, 80, 1, 8)
    k[0, 70] = -math.inf              # weight 0, from a tile of its own
    v = torch.arange(80.0).reshape(1, 80, 1, 1).expand(1, 80, 1, 8).clone()
    o = seq.cross_attention(q.cuda(), k.cuda(), v.cuda())
    want = (v.sum(1) - 70.0) / 79
    within(o, want[:, None].double(), torch.tensor(100 * 80 * plain.U32))
    k[:] = -math.inf                  # every score -inf: no weight anywhere, as without a key
    o, lse = seq.cross_attention(q.cuda(), k.cuda(), v.cuda(), return_lse=True)
    assert bool((lse == -math.inf).all())
    v[0, 3] = math.nan
    assert bool(torch.isnan(seq.cross_attention(q.cuda(), torch.zeros_like(k).cuda(), v.cuda())).all())


def test_cross_attention_lengths_out_of_range_are_recorded(seq):
    from dynamic_embedding_tables_amd import recis
    q, k = torch.randn(2, 3, 2, 16).cuda(), torch.randn(2, 70, 2, 16).cuda()
    bad = [dict(kv_lens=[71, 5]), dict(kv_lens=[3, -1]), dict(kv_offsets=[0, 5, 150], max_kv_len=70),
           dict(kv_offsets=[0, 5, 4], max_kv_len=70), dict(kv_offsets=[-2, 5, 6], max_kv_len=70),
           dict(kv_offsets=[0, 9, 12], max_kv_len=8)]
    for kw in bad:
        kw = {n: torch.tensor(x, dtype=torch.int32).cuda() if isinstance(x, list) else x for n, x in kw.items()}
        kv = k if "kv_lens" in kw else k.reshape(140, 2, 16)
        error = torch.zeros(1, dtype=torch.int32).cuda()
        o, lse = seq.cross_attention(q, kv, kv, return_lse=True, error=error, **kw)
        with pytest.raises(recis.RecisError) as e:
            seq.check(error)
        assert e.value.status == recis.RECIS_ERR_INVALID_ARG
        assert int((lse == -math.inf).all(-1).all(-1).sum()) >= 1   # taken as empty
        error.zero_()
        seq.cross_attention_backward(q, q, kv, kv, o, lse, error=error, **kw)
        with pytest.raises(recis.RecisError):
            seq.check(error)
        seq.cross_attention(q, kv, kv, **kw)


def test_cross_attention_beyond_32_bit_offsets(seq):
    gen = generator(14)
    q, k, v, kw, kept = attn_case(gen, (2, 3, 90, 2, 2, 32), BF16, "lens", spoil=False)
    kw["kv_lens"][1] = 77
    kept = plain.kept_keys(k, kw["kv_lens"])
    store = torch.zeros((1 << 31) + 90 * 64, dtype=BF16, device="cuda")

    def far(t):
        if t.shape[1] != 90:
            return t.cuda()
        at = store.as_strided(t.shape, ((1 << 31), 64, 32, 1)) if t is k else t.cuda()
        at.copy_(t)
        return at

    check_attention(seq, q, k, v, kw, kept, grad=normal(gen, *q.shape, dtype=BF16), move=far)


def test_cross_attention_gradient_is_the_difference_quotient(seq):
    gen = generator(15)
    q, k, v, kw, kept = attn_case(gen, (2, 6, 50, 4, 2, 24), F32, "mask", spoil=False)
    kept = plain.kept_keys(k, kw["kv_lens"], None, kw["kv_mask"])
    grad, h, s = normal(gen, *q.shape), 2.0**-5, 24**-0.5
    o, lse = seq.cross_attention(q.cuda(), k.cuda(), v.cuda(), return_lse=True, **on_gpu(kw))
    got = seq.cross_attention_backward(grad.cuda(), q.cuda(), k.cuda(), v.cuda(), o, lse, **on_gpu(kw))
    want = plain.attention(q, k, v, s, kept, False, grad)
    for i, name in enumerate(("dq", "dk", "dv")):
        way = normal(gen, *(q, k, v)[i].shape)
        slope = along = exact = noise = 0.0
        for sign in (1, -1):
            moved = [t + sign * h * way if j == i else t for j, t in enumerate((q, k, v))]
            out = seq.cross_attention(*(t.cuda() for t in moved), **on_gpu(kw)).cpu().double()
            val, bound = plain.attention(*moved, s, kept, False)["o"]
            slope += sign * (out * grad.double()).sum() / (2 * h)
            exact += sign * (val * grad.double()).sum() / (2 * h)
            noise += (bound * grad.double().abs()).sum() / (2 * h)
        along = (got[i].cpu().double() * way.double()).sum()
        step = abs(exact - (want[name][0] * way.double()).sum())   # the step's own error
        assert abs(slope - along) <= step + noise + (want[name][1] * way.double().abs()).sum(), name


# ------------------------------------------------------------ together
def test_on_another_stream(seq):
    gen = generator(16)
    side = torch.cuda.Stream()
    t, w, g = tokens_of(gen, 5000, 300).cuda(), normal(gen, 300, 64).cuda(), normal(gen, 5000, 64).cuda()
    q, k = normal(gen, 4, 30, 2, 32).cuda(), normal(gen, 4, 500, 2, 32).cuda()

    def every(stream=None):
        y, mean, rstd = seq.layer_norm(g, stream=stream)
        o, lse = seq.cross_attention(q, k, k, return_lse=True, stream=stream)
        return [seq.embed(t, w, stream=stream), seq.embed_backward(t, g, 300, stream=stream), y, mean, rstd, o, lse,
                *seq.layer_norm_backward(g, g, mean, rstd, stream=stream),
                *seq.cross_attention_backward(q, q, k, k, o, lse, stream=stream)]

    want = every()
    side.wait_stream(torch.cuda.current_stream())
    got = every(side)
    with torch.cuda.stream(side):
        inner = every()
    torch.cuda.current_stream().wait_stream(side)
    for a, b, c in zip(want, got, inner):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_captured_into_a_graph(seq):
    gen = generator(17)
    t, w, g = tokens_of(gen, 3000, 200).cuda(), normal(gen, 200, 64).cuda(), normal(gen, 3000, 64).cuda()
    q, k = normal(gen, 2, 1, 4, 64).cuda(), normal(gen, 2, 2000, 2, 64).cuda()
    lens = torch.tensor([2000, 700], dtype=torch.int32).cuda()

    def step():
        y, mean, rstd = seq.layer_norm(seq.embed(t, w, scale=8.0))
        dx, dw, db = seq.layer_norm_backward(g, y, mean, rstd)
        o, lse = seq.cross_attention(q, k, k, kv_lens=lens, return_lse=True)
        return [y, dx, dw, db, seq.embed_backward(t, dx, 200), o, lse,
                *seq.cross_attention_backward(q, q, k, k, o, lse, kv_lens=lens)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):   # new values in the same tensors, eager work in between
        w.copy_(normal(gen, 200, 64))
        g.copy_(normal(gen, 3000, 64))
        k.copy_(normal(gen, 2, 2000, 2, 64))
        t.copy_(tokens_of(gen, 3000, 200))
        lens.copy_(torch.tensor([2000 - 300 * i, 64 * i], dtype=torch.int32))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, held):
            assert torch.equal(a, b)


def test_refusals_on_tensors(seq):
    x = torch.randn(4, 8).cuda()
    with pytest.raises(ValueError):
        seq.embed(torch.zeros(3, dtype=torch.int32).cuda(), x)
    with pytest.raises(ValueError):
        seq.embed(torch.zeros(3, dtype=torch.int64), x)             # on the host
    with pytest.raises(ValueError):
        seq.embed(torch.zeros(3, dtype=torch.int64).cuda(), x.half())
    with pytest.raises(ValueError):
        seq.embed(torch.zeros(3, dtype=torch.int64).cuda(), x, out=torch.empty(3, 9).cuda())
    with pytest.raises(ValueError):
        seq.embed_backward(torch.zeros(3, dtype=torch.int64).cuda(), x, 5)
    with pytest.raises(ValueError):
        seq.layer_norm(x, torch.ones(7).cuda())
    with pytest.raises(ValueError):
        seq.layer_norm(x, torch.ones(8).cuda(), torch.ones(8).cuda().to(BF16))
    y, mean, rstd = seq.layer_norm(x)
    with pytest.raises(ValueError):
        seq.layer_norm_backward(x, x, mean[:2], rstd)
    q, k = torch.randn(2, 3, 4, 8).cuda(), torch.randn(2, 5, 2, 8).cuda()
    o, lse = seq.cross_attention(q, k, k, return_lse=True)
    for kw in (dict(kv_lens=torch.zeros(3, dtype=torch.int32).cuda()), dict(kv_lens=torch.zeros(2, dtype=torch.int64).cuda()),
               dict(kv_mask=torch.ones(2, 4, dtype=torch.bool).cuda()), dict(kv_offsets=torch.zeros(3, dtype=torch.int32).cuda()),
               dict(max_kv_len=4)):
        with pytest.raises(ValueError):
            seq.cross_attention(q, k, k, **kw)
        with pytest.raises(ValueError):
            seq.cross_attention_backward(q, q, k, k, o, lse, **kw)
    with pytest.raises(ValueError):
        seq.cross_attention(q, k, k.to(BF16))
    from dynamic_embedding_tables_amd import recis
    for bad, status in (((q, k[:, :, :1].expand(2, 5, 3, 8)), recis.RECIS_ERR_INVALID_ARG),   # 4 heads over 3
                        ((torch.randn(1, 1, 1, 130).cuda(), torch.randn(1, 1, 1, 130).cuda()), recis.RECIS_ERR_UNSUPPORTED)):
        with pytest.raises(recis.RecisError) as e:
            seq.cross_attention(bad[0], bad[1], bad[1])
        assert e.value.status == status
    with pytest.raises(recis.RecisError) as e:
        seq.cross_attention(q, k, k, scale=0.0)
    assert e.value.status == recis.RECIS_ERR_INVALID_ARG
    with pytest.raises(recis.RecisError) as e:
        seq.layer_norm(torch.randn(1, 16385).cuda())
    assert e.value.status == recis.RECIS_ERR_UNSUPPORTED


@pytest.mark.parametrize("most", [(1 << 31) + 64, (1 << 32) + 9, 1 << 40])
def test_key_counts_past_32_bits_are_refused(seq, most):
    from dynamic_embedding_tables_amd import recis
    q, k = torch.randn(2, 3, 2, 16).cuda(), torch.randn(9, 2, 16).cuda()
    off = torch.tensor([0, 4, 9], dtype=torch.int32).cuda()
    o, lse = seq.cross_attention(q, k, k, kv_offsets=off, max_kv_len=9, return_lse=True)
    for call in (lambda: seq.cross_attention(q, k, k, kv_offsets=off, max_kv_len=most),
                 lambda: seq.cross_attention_backward(q, q, k, k, o, lse, kv_offsets=off, max_kv_len=most)):
        with pytest.raises(recis.RecisError) as e:
            call()
        assert e.value.status == recis.RECIS_ERR_UNSUPPORTED


def test_embed_of_more_blocks_than_a_launch_dimension(seq):
    """2^24 + 64 blocks of 1024 elements."""
    dim = 65535
    n = ((1 << 34) + (1 << 16)) // dim + 1
    gen = generator(19)
    w = normal(gen, 3, dim, dtype=BF16).cuda()
    t = (torch.arange(n) % 4 - 1).cuda()
    out = seq.embed(t, w, scale=2.0)
    want = torch.cat([torch.zeros(1, dim, dtype=BF16, device="cuda"), w * 2])
    for first in range(4):   # every row, a quarter of them at a time
        assert bool((out[first::4] == want[first]).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_cross_attention_of_more_blocks_than_a_launch_dimension(seq, dtype):
    """65536 entries of 0 to 2 packed keys, 8 heads, max_kv_len 4096 (f32) or 8192: 2^25 key tiles.  Every tile past
    an entry's keys has nothing to do, so the results are those of max_kv_len 2."""
    gen = generator(20)
    lens = torch.arange(1 << 16, dtype=torch.int32) % 3
    off = torch.zeros((1 << 16) + 1, dtype=torch.int32)
    off[1:] = lens.cumsum(0)
    q, grad = (normal(gen, 1 << 16, 1, 8, 8, dtype=dtype).cuda() for _ in range(2))
    k, v = (normal(gen, int(off[-1]), 8, 8, dtype=dtype).cuda() for _ in range(2))

    def both(most):
        kw = {"kv_offsets": off.cuda(), "max_kv_len": most}
        o, lse = seq.cross_attention(q, k, v, return_lse=True, **kw)
        return o, lse, *seq.cross_attention_backward(grad, q, k, v, o, lse, **kw)

    wide, narrow = both(4096 if dtype == F32 else 8192), both(2)
    assert all(torch.equal(a, b) for a, b in zip(wide, narrow))
    some = slice((1 << 16) - 30, 1 << 16)   # the last entries against the definition
    first = int(off[some.start])
    kept = [torch.arange(int(off[i]) - first, int(off[i + 1]) - first) for i in range(some.start, some.stop)]
    want = plain.attention(q[some].cpu(), k[first:].cpu(), v[first:].cpu(), 8**-0.5, kept, True, grad[some].cpu())
    for name, t in zip(("o", "lse", "dq", "dk", "dv"), wide):
        within(t[some] if t.shape[0] == 1 << 16 else t[first:], *want[name], what=name)


def test_check_waits_for_the_stream_that_records(seq):
    from dynamic_embedding_tables_amd import recis
    side = torch.cuda.Stream()
    w, t = torch.randn(10, 8).cuda(), torch.tensor([3, 10]).cuda()
    for stream in (None, side):
        error = torch.zeros(1, dtype=torch.int32).cuda()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(1 << 27)   # some 50 ms of the stream's time
        seq.embed(t, w, error=error, stream=side)
        with pytest.raises(recis.RecisError) as e:
            seq.check(error, **({"stream": stream} if stream else {}))
        assert e.value.status == recis.RECIS_ERR_KEY_RANGE
        torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [32, 33])
@pytest.mark.parametrize("front,back", [(0, 5000), (4001, 0), (70000, 90001)])
def test_packed_rows_outside_the_entries_get_zeros(seq, front, back, dim, dtype):
    """Buffers of a fixed capacity, of which the entries take a part."""
    gen = generator(24, front, back, dim)
    lens = [130, 0, 7]
    off = torch.tensor([front + sum(lens[:i]) for i in range(4)], dtype=torch.int32)
    rows = front + sum(lens) + back
    q, grad = normal(gen, 3, 5, 4, dim, dtype=dtype), normal(gen, 3, 5, 4, dim, dtype=dtype)
    k, v = torch.full((rows, 2, dim), math.nan, dtype=dtype), torch.full((rows, 2, dim), math.nan, dtype=dtype)
    used = slice(front, front + sum(lens))
    k[used], v[used] = normal(gen, sum(lens), 2, dim, dtype=dtype), normal(gen, sum(lens), 2, dim, dtype=dtype)
    kw = on_gpu({"kv_offsets": off, "max_kv_len": 150})
    dev = [t.cuda() for t in (q, k, v)]
    o, lse = seq.cross_attention(*dev, return_lse=True, **kw)
    for fill in (math.nan, 3.0):   # what the allocator's memory holds before
        junk = [torch.full((rows, 2, dim), fill, dtype=dtype, device="cuda") for _ in range(3)]
        del junk
        _, dk, dv = seq.cross_attention_backward(grad.cuda(), *dev, o, lse, **kw)
        for t in (dk, dv):
            assert not bool(t[:front].any()) and not bool(t[used.stop:].any())
    kept = [torch.arange(int(off[i]), int(off[i + 1])) - front for i in range(3)]
    want = plain.attention(q, k[used], v[used], dim**-0.5, kept, True, grad)
    within(dk[used], *want["dk"])
    within(dv[used], *want["dv"])


@pytest.mark.parametrize("layout", ["lens", "mask", "packed mask"])
def test_cross_attention_score_gradients_of_few_keys(seq, layout):
    """Three keys that count, by a length or by a mask over 700: delta is taken in float32, so a score gradient is off
    by its own roundings only.  (delta from the rounded out is off by 2^-9 of sum |dO| |O|, far above a score gradient
    whose weight is near 1.)"""
    gen = generator(22)
    n, d, scale = 3, 64, 0.5   # scores of deviation 4: one key often has nearly all the weight
    q, grad = normal(gen, 3, 50, 4, d, dtype=BF16), normal(gen, 3, 50, 4, d, dtype=BF16)
    k, v = normal(gen, 3, 700, 2, d, dtype=BF16), normal(gen, 3, 700, 2, d, dtype=BF16)
    places = torch.tensor([[0, 350, 699], [63, 64, 65], [5, 300, 301]])
    if layout == "lens":
        places = torch.arange(n).expand(3, n)
        kw = {"kv_lens": torch.full((3,), n, dtype=torch.int32)}
    else:
        kw = {"kv_mask": torch.zeros(3, 700, dtype=torch.bool).scatter_(1, places, True)}
    kept = list(places)
    want = plain.attention(q, k, v, scale, kept, False, grad)
    packed = layout.startswith("packed")
    if packed:
        kw = {"kv_mask": kw["kv_mask"].reshape(-1), "kv_offsets": torch.arange(4, dtype=torch.int32) * 700,
              "max_kv_len": 700}
    dev = [(t.reshape(2100, 2, d) if packed and t.shape[1] == 700 else t).cuda() for t in (q, k, v)]
    o, lse = seq.cross_attention(*dev, return_lse=True, scale=scale, **on_gpu(kw))
    dq, dk, dv = (t.cpu().double().reshape(s.shape) for t, s in zip(
        seq.cross_attention_backward(grad.cuda(), *dev, o, lse, scale=scale, **on_gpu(kw)), (q, k, v)))
    for name, t in (("o", o), ("lse", lse), ("dv", dv)):
        within(t, *want[name], what=name)
    u, ub = plain.U32, plain.U[BF16]
    for b in range(3):
        for h in range(4):
            Q, G, K, V = (t.double() for t in (q[b, :, h], grad[b, :, h], k[b, kept[b], h // 2], v[b, kept[b], h // 2]))
            P = torch.softmax(scale * Q @ K.T, -1)
            # a weight's relative error: its score's (a float32 sum of d products, and the lse of the forward), the exponential's
            size = scale * Q.abs() @ K.abs().T
            eP = (d + 16) * u * size + 2 * want["lse"][1][b, :, h][:, None] + 16 * u * (size.amax(-1, keepdim=True) + 1)
            dP, mag = G @ V.T, G.abs() @ V.abs().T
            edP = (d + 2) * u * mag
            delta, edelta = (P * dP).sum(-1, keepdim=True), (P * (eP * dP.abs() + edP + (n + 2) * u * dP.abs())).sum(
                -1, keepdim=True)
            dS = P * (dP - delta)
            edS = dS.abs() * (eP + ub) + P * (1 + eP) * (1 + ub) * (edP + edelta + 4 * u * (dP.abs() + delta.abs()))
            value, bound = scale * dS @ K, scale * (edS + 8 * u * dS.abs()) @ K.abs()
            within(dq[b, :, h], value, bound + ub * (value.abs() + bound) + plain.TINY, what=(layout, "dq"))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("d", [32, 40, 77, 128])
def test_cross_attention_masks_that_leave_64_keys_or_65(seq, d, packed):
    gen = generator(25, d)
    lk, counts = 5000, (64, 65, 0, 1, 3, 4000)
    q, k, v = (normal(gen, len(counts), n, 2, d, dtype=BF16) for n in (20, lk, lk))
    mask = torch.zeros(len(counts), lk, dtype=torch.bool)
    for b, n in enumerate(counts):
        mask[b, torch.randperm(lk, generator=gen)[:n]] = True
    mask[3:5] = False
    mask[3, lk - 1] = True
    mask[4, [0, 2047, 2048]] = True   # the ends of the first 2048 keys
    kw = {"kv_mask": mask}
    if packed:
        off = torch.arange(len(counts) + 1, dtype=torch.int32) * lk
        kw, k, v = {"kv_mask": mask.reshape(-1), "kv_offsets": off, "max_kv_len": lk}, k.reshape(-1, 2, d), v.reshape(-1, 2, d)
    kept = plain.kept_keys(k, None, kw.get("kv_offsets"), kw["kv_mask"])
    check_attention(seq, q, k, v, kw, kept, grad=normal(gen, *q.shape, dtype=BF16), what=(d, packed))


@pytest.mark.parametrize("scale", [math.inf, math.nan])
@pytest.mark.parametrize("n", [600, 5000])   # gradient by one launch and by sorted tokens
def test_embed_rows_without_a_token_are_zero_whatever_the_scale(seq, n, scale):
    gen = generator(21, n)
    t, w, g = tokens_of(gen, n, 40) * 3, normal(gen, 120, 33), normal(gen, n, 33)   # rows 0, 3, 6 ... and -3
    t[5] = 120                                                                       # beyond the table
    for dtype in DTYPES:
        out = seq.embed(t.cuda(), w.to(dtype).cuda(), scale=scale).cpu()
        gone = (t < 0) | (t >= 120)
        assert bool((out[gone] == 0).all()) and not bool(torch.isfinite(out[~gone]).any())
        dw = seq.embed_backward(t.cuda(), g.to(dtype).cuda(), 120, scale=scale).cpu()
        named = torch.zeros(120, dtype=torch.bool)
        named[t[~gone]] = True
        assert bool((dw[~named] == 0).all()) and not bool(torch.isfinite(dw[named]).any())


def test_empty_head_vectors_are_refused(seq):
    from dynamic_embedding_tables_amd import recis
    q, k = torch.randn(2, 3, 4, 0).cuda(), torch.randn(2, 5, 2, 0).cuda()
    lse = torch.zeros(2, 3, 4).cuda()
    for call in (lambda: seq.cross_attention(q, k, k), lambda: seq.cross_attention_backward(q, q, k, k, q, lse)):
        with pytest.raises(recis.RecisError) as e:
            call()
        assert e.value.status == recis.RECIS_ERR_INVALID_ARG


def test_inputs_that_require_a_gradient_are_warned_about(seq):
    """The calls record no graph: who asks for gradients through them is told so, and gets the same result."""
    gen = generator(23)
    t = tokens_of(gen, 20, 6).cuda()
    w, x, q = normal(gen, 6, 16).cuda(), normal(gen, 20, 16).cuda(), normal(gen, 2, 5, 2, 16).cuda()
    one = torch.ones(16).cuda()
    calls = [(lambda a: seq.embed(t, a), w), (lambda a: seq.layer_norm(a, one)[0], x),
             (lambda a: seq.layer_norm(x, a)[0], one), (lambda a: seq.layer_norm(x, one, a)[0], one),
             (lambda a: seq.cross_attention(a, q, q), q), (lambda a: seq.cross_attention(q, a, q), q),
             (lambda a: seq.cross_attention(q, q, a), q)]
    for call, a in calls:
        want = call(a)
        with pytest.warns(UserWarning, match="gradient"):
            got = call(a.clone().requires_grad_())
        assert torch.equal(got, want) and not got.requires_grad
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with torch.no_grad():
                call(a.clone().requires_grad_())
            call(a.clone().requires_grad_().detach())


# ------------------------------------------- what only large sizes reach
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,rows,dim", [
    (70001, 50021, 16),      # 69 tiles of 1024 keys: the counts are scanned by a kernel of their own
    (300007, 50021, 8),      # tiles of 4096 keys
    (262144, 300, 3), (262145, 300, 3),   # the last call of the small tiles, the first of the large
    (5000, 4200000, 4),      # three sort passes, over a result that is stored past the caches
    (70001, 4194303, 1), (70001, 4194304, 1), (300007, 5000000, 2),
])
def test_embed_backward_of_many_tokens(seq, n, rows, dim, dtype):
    gen = generator(26, n, rows, dim)
    t, g = tokens_of(gen, n, rows), normal(gen, n, dim, dtype=dtype)
    t[::7] = rows // 3       # a token that fills a seventh of the call
    t[n // 2] = rows - 1
    got = seq.embed_backward(t.cuda(), g.cuda(), rows, scale=0.3)
    within(got, *plain.embed_backward(t, g, rows, 0.3, dtype), what=(n, rows, dim))
    assert torch.equal(seq.embed_backward(t.cuda(), g.cuda(), rows, scale=0.3), got), "two calls on equal inputs differ"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [128, 127])
def test_embed_past_the_caches(seq, dim, dtype):
    gen = generator(27, dim)
    n = (40 << 20) // (dim * dtype.itemsize)   # 40 MiB
    t, w = tokens_of(gen, n, 3000), normal(gen, 3000, dim, dtype=dtype)
    want = torch.where((t >= 0)[:, None], w.float()[t.clamp_min(0)] * torch.tensor(3.7), 0).to(dtype)
    assert torch.equal(seq.embed(t.cuda(), w.cuda(), scale=3.7).cpu(), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,dim", [
    (1050001, 5), (33001, 1025),                       # forward: more rows than 2^14 blocks hold
    (50001, 64), (30011, 128), (7001, 1000), (2003, 4096), (1001, 16384), (901, 8193),  # the same of the backward's
])
def test_layer_norm_blocks_take_turns(seq, m, dim, dtype):
    gen = generator(28, m, dim)
    x, g, w, b = normal(gen, m, dim, dtype=dtype), normal(gen, m, dim, dtype=dtype), normal(gen, dim), normal(gen, dim)
    y, mean, rstd = seq.layer_norm(x.cuda(), w.cuda(), b.cuda())
    dx, dw, db = seq.layer_norm_backward(g.cuda(), x.cuda(), mean, rstd, w.cuda())
    want = {**plain.layer_norm(x, w, b, 1e-5, dtype), **plain.layer_norm_backward(g, x, w, 1e-5, dtype, F32)}
    for name, got in (("y", y), ("mean", mean), ("rstd", rstd), ("dx", dx), ("dw", dw), ("db", db)):
        within(got, *want[name], what=(name, m, dim))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [16, 15, 64, 63, 127, 128, 255, 256, 511, 512, 1023, 1024, 2047, 2048, 4095, 4096, 8191,
                                 8192, 16383, 16384])   # every form of a row over the lanes, at its longest
def test_layer_norm_row_forms(seq, dim, dtype):
    gen = generator(29, dim)
    x, g = normal(gen, 37, dim, dtype=dtype), normal(gen, 37, dim, dtype=dtype)
    y, mean, rstd = seq.layer_norm(x.cuda())
    within(y, *plain.layer_norm(x, None, None, 1e-5, dtype)["y"])
    want = plain.layer_norm_backward(g, x, None, 1e-5, dtype, F32)
    for name, got in zip(("dx", "dw", "db"), seq.layer_norm_backward(g.cuda(), x.cuda(), mean, rstd)):
        within(got, *want[name], what=(name, dim))


@pytest.mark.parametrize("kind", ["lens", "packed mask"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [   # batch, q_len, kv_len, q_heads, kv_heads, head_dim
    (2, 700, 600, 2, 2, 32), (1, 1100, 300, 4, 2, 33),   # more than 2048 rows with their keys split
    (67, 1, 300, 6, 3, 16), (67, 40, 100, 3, 3, 32),     # heads of an entry together, the last turn of the dies not full
    (131, 150, 90, 1, 1, 24),                            # several row tiles, pairs that do not fill a turn
    (131, 40, 330, 8, 8, 16), (131, 20, 290, 4, 4, 128), (131, 70, 200, 4, 4, 96), (131, 70, 200, 4, 4, 48),
    (131, 1, 1000, 8, 8, 16),                            # a block walks all the keys: both tile buffers more than once
])
def test_cross_attention_of_many_blocks(seq, shape, dtype, kind):
    gen = generator(*shape, len(kind), 30)
    q, k, v, kw, kept = attn_case(gen, shape, dtype, kind)
    check_attention(seq, q, k, v, kw, kept, grad=normal(gen, *q.shape, dtype=dtype), what=(shape, kind))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d", [16, 21])
def test_packed_entries_of_too_many_keys_get_zeros(seq, d, dtype):
    """An entry of more than max_kv_len keys is taken as empty, in the gradients as well."""
    gen = generator(31, d)
    lens = [70, 300, 0, 5, 71]
    off = torch.tensor([sum(lens[:i]) for i in range(6)], dtype=torch.int32)
    rows = sum(lens)
    q, grad = normal(gen, 5, 3, 4, d, dtype=dtype), normal(gen, 5, 3, 4, d, dtype=dtype)
    k, v = normal(gen, rows, 2, d, dtype=dtype), normal(gen, rows, 2, d, dtype=dtype)
    kw = on_gpu({"kv_offsets": off, "max_kv_len": 70, "error": torch.zeros(1, dtype=torch.int32)})
    dev = [t.cuda() for t in (q, k, v)]
    o, lse = seq.cross_attention(*dev, return_lse=True, **kw)
    junk = [torch.full((rows, 2, d), math.nan, dtype=dtype, device="cuda") for _ in range(3)]
    del junk   # what the results' memory holds before
    got = (o, lse, *seq.cross_attention_backward(grad.cuda(), *dev, o, lse, **kw))
    kept = [torch.arange(int(off[i]), int(off[i + 1])) if n <= 70 else torch.arange(0) for i, n in enumerate(lens)]
    want = plain.attention(q, k, v, d**-0.5, kept, True, grad)
    for name, t in zip(("o", "lse", "dq", "dk", "dv"), got):
        within(t, *want[name], what=name)
    from dynamic_embedding_tables_amd import recis
    with pytest.raises(recis.RecisError):
        seq.check(kw["error"])


def test_a_masked_backward_captured_into_a_graph(seq):
    """Masks that leave few keys in one replay and many in the next, in a packed buffer partly in use."""
    gen = generator(32)
    q, grad = normal(gen, 4, 20, 4, 64, dtype=BF16).cuda(), normal(gen, 4, 20, 4, 64, dtype=BF16).cuda()
    k, v = normal(gen, 3000, 2, 64, dtype=BF16).cuda(), normal(gen, 3000, 2, 64, dtype=BF16).cuda()
    off, mask = torch.tensor([0, 600, 600, 1200, 1500], dtype=torch.int32).cuda(), torch.ones(3000, dtype=torch.bool).cuda()

    def step():
        kw = {"kv_offsets": off, "kv_mask": mask, "max_kv_len": 700}
        o, lse = seq.cross_attention(q, k, v, return_lse=True, **kw)
        return [o, lse, *seq.cross_attention_backward(grad, q, k, v, o, lse, **kw)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i, share in enumerate((0.02, 0.9, 0.1, 0.0, 1.0)):
        mask.copy_(torch.rand(3000, generator=gen) < share)
        off.copy_(torch.tensor([5 * i, 600, 650 + i, 1200, 1900 - 100 * i], dtype=torch.int32))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, held):
            assert torch.equal(a, b), share
