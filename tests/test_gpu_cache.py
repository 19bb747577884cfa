"""The paged 8-bit cache on the GPU: codes and scales byte for byte, what is read back bit for bit,
attention against float64 (the tolerance is derived in cache_reference.attention)."""
import math

import pytest
import torch

from tests import cache_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
P_EPS = {"bf16": 2.0 ** -16, "f32": 2.0 ** -23}  # the probabilities' terms, and their sum's


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_hadamard32_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.lib()
    return m


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def offsets_of(new):
    o = [0]
    for n in new:
        o.append(o[-1] + n)
    return o


def rows(T, heads, dim, dtype, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, heads, dim), generator=g) * torch.exp(spread * torch.randn((T, heads, 1), generator=g))
    return x.to(DT[dtype])


SETS = [  # lengths, newest tokens
    ([1, 32, 33], [1, 1, 1]),
    ([31, 64, 65, 100, 7], [31, 33, 1, 100, 0]),
    ([257, 40, 0, 96], [200, 8, 0, 96]),
    ([5, 300], [9, 270]),   # more rows than tokens
]


@pytest.mark.parametrize("dtype,fmt,ceil", [("bf16", 0, False), ("bf16", 1, True), ("f32", 0, True),
                                            ("f32", 1, False)])
@pytest.mark.parametrize("heads,dim,page", [(2, 128, 64), (1, 64, 32), (3, 192, 96), (2, 256, 160)])
@pytest.mark.parametrize("lengths,new", SETS)
def test_write_and_read(mx, lengths, new, heads, dim, page, dtype, fmt, ceil):
    table, n_pages = ref.table_of(lengths, page)
    cache = ref.Cache(n_pages, heads, page, dim, fmt, seed=1)
    for b, (length, n) in enumerate(zip(lengths, new)):  # what is there already
        cache.random_sequence(table[b], max(length - n, 0), 10 + b)
    dev = [t.to(DEV) for t in cache.tensors()]
    off = offsets_of(new)
    T = off[-1] + 3  # rows behind the last sequence
    k, v = rows(T, heads, dim, dtype, 3), rows(T, heads, dim, dtype, 4)
    both = torch.stack([k, v], 1).to(DEV)  # token distances of a joint projection
    for b, (length, n) in enumerate(zip(lengths, new)):
        cache.write(k[off[b]:off[b + 1]], v[off[b]:off[b + 1]], table[b], length, ceil)
    args = (*dev, table.to(DEV), i32(lengths))
    mx.mx_cache_write(both[:, 0], both[:, 1], *args, offsets=i32(off), fmt=fmt, scale_rule=int(ceil))
    for name, got, want in zip(("kq", "ks", "vq", "vs"), dev, cache.tensors()):
        assert torch.equal(got.cpu(), want), name
    before = torch.full((2, T, heads, dim), 7.0, dtype=DT[dtype], device=DEV)
    out = mx.mx_cache_read(*args, offsets=i32(off), fmt=fmt, k=before[0], v=before[1])
    for x, got in zip("kv", out):
        want = torch.full((T, heads, dim), 7.0, dtype=torch.float64)
        for b, (length, n) in enumerate(zip(lengths, new)):
            want[off[b]:off[b + 1]] = cache.tokens(x, table[b], length - n, n)[0]
        assert torch.equal(got.cpu(), want.to(DT[dtype])), x


@pytest.mark.parametrize("dtype,fmt", [("bf16", 0), ("f32", 1)])
def test_token_by_token(mx, dtype, fmt):
    """A block that grows: the scale takes the largest token so far, and codes that fall below the
    least normal are rounded once for each growth, as the reference does it."""
    heads, dim, page, count = 2, 64, 32, 70
    table, n_pages = ref.table_of([count, count], page)
    cache = ref.Cache(n_pages, heads, page, dim, fmt, seed=2)
    dev = [t.to(DEV) for t in cache.tensors()]
    k, v = rows(2 * count, heads, dim, dtype, 5, 4.0), rows(2 * count, heads, dim, dtype, 6, 4.0)
    kd, vd = k.to(DEV), v.to(DEV)
    for i in range(count):
        mx.mx_cache_write(kd[2 * i:2 * i + 2], vd[2 * i:2 * i + 2], *dev, table.to(DEV),
                          i32([i + 1, i + 1]), fmt=fmt)
        for b in range(2):
            r = 2 * i + b
            cache.write(k[r:r + 1], v[r:r + 1], table[b], i + 1)
    for name, got, want in zip(("kq", "ks", "vq", "vs"), dev, cache.tensors()):
        assert torch.equal(got.cpu(), want), name


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_not_finite(mx, bad):
    """The block's scale is 0xFF and its tokens' codes zero, older and later ones too; the other
    head and the other sequence keep theirs."""
    heads, dim, page = 2, 64, 32
    lengths = [40, 40]
    table, n_pages = ref.table_of(lengths, page)
    cache = ref.Cache(n_pages, heads, page, dim, 0, seed=3)
    k, v = rows(80, heads, dim, "bf16", 7, 0.5), rows(80, heads, dim, "bf16", 8, 0.5)
    k[10, 1, 3] = bad
    v[45, 0, 63] = bad
    dev = [t.to(DEV) for t in cache.tensors()]
    for step in ((0, 9), (9, 20), (20, 40)):  # older tokens, the bad one, later ones
        off, n = [0, step[1] - step[0], 2 * (step[1] - step[0])], step[1] - step[0]
        rk = torch.cat([k[step[0]:step[1]], k[40 + step[0]:40 + step[1]]])
        rv = torch.cat([v[step[0]:step[1]], v[40 + step[0]:40 + step[1]]])
        mx.mx_cache_write(rk.to(DEV), rv.to(DEV), *dev, table.to(DEV), i32([step[1]] * 2), offsets=i32(off))
        for b in range(2):
            cache.write(rk[b * n:b * n + n], rv[b * n:b * n + n], table[b], step[1])
    for name, got, want in zip(("kq", "ks", "vq", "vs"), dev, cache.tensors()):
        assert torch.equal(got.cpu(), want), name
    assert (cache.ks == 255).sum() >= 1 and (cache.vs == 255).sum() >= 1
    got = mx.mx_cache_read(*dev, table.to(DEV), i32(lengths), offsets=i32([0, 40, 80]), rows=80,
                           out_dtype=torch.float32)
    for x, t in zip("kv", got):
        for b in range(2):
            want = cache.tokens(x, table[b], 0, 40)[0].float()
            assert torch.equal(torch.nan_to_num(t[40 * b:40 * b + 40].cpu(), 99.0), torch.nan_to_num(want, 99.0))


def test_missing_pages(mx):
    """Table entries that are no page, tokens beyond the table, rows that are nobody's."""
    heads, dim, page = 1, 64, 32
    lengths, new = [100, 150, 20], [100, 60, 20]
    table, n_pages = ref.table_of([100, 128, 20], page, seed=4)
    table[0, 1], table[1, 2] = -1, n_pages  # 150 tokens are more than the table holds as well
    cache = ref.Cache(n_pages, heads, page, dim, 0, seed=5)
    dev = [t.to(DEV) for t in cache.tensors()]
    off = [4] + [4 + o for o in offsets_of(new)[1:]]
    k, v = rows(off[-1] + 5, heads, dim, "bf16", 9), rows(off[-1] + 5, heads, dim, "bf16", 10)
    for b in range(3):
        cache.write(k[off[b]:off[b + 1]], v[off[b]:off[b + 1]], table[b], lengths[b])
    args = (*dev, table.to(DEV), i32(lengths))
    mx.mx_cache_write(k.to(DEV), v.to(DEV), *args, offsets=i32(off))
    for name, got, want in zip(("kq", "ks", "vq", "vs"), dev, cache.tensors()):
        assert torch.equal(got.cpu(), want), name
    out = torch.full((2, off[-1] + 5, heads, dim), 7.0, device=DEV)
    mx.mx_cache_read(*args, offsets=i32(off), k=out[0], v=out[1])
    for x, got in zip("kv", out.cpu()):
        want = torch.full_like(got, 7.0)
        for b in range(3):
            want[off[b]:off[b + 1]] = cache.tokens(x, table[b], lengths[b] - new[b], new[b])[0].float()
        assert torch.equal(got, want)


def check_attention(mx, cache, table, lengths, new, group, dtype, scale=None, seed=20, size=1.0,
                    **kw):
    off = offsets_of(new)
    T, heads = off[-1], cache.heads * group
    g = torch.Generator().manual_seed(seed)
    q = (size * torch.randn((T, heads, cache.dim), generator=g)).to(DT[dtype])
    dev = [t.to(DEV) for t in cache.tensors()]
    o = None if all(n == 1 for n in new) else i32(off)
    got, lse = mx.mx_cache_attention(q.to(DEV), *dev, table.to(DEV), i32(lengths), offsets=o,
                                     scale=scale, fmt=cache.fmt, with_lse=True, **kw)
    got, lse = got.cpu(), lse.cpu()
    f = cache.dim ** -0.5 if scale is None else scale
    half = torch.finfo(DT[dtype]).eps / 2
    for b, (length, n) in enumerate(zip(lengths, new)):
        want, want_lse, tol = ref.attention(cache, q[off[b]:off[b + 1]], table[b], length, f, P_EPS[dtype])
        x, l = got[off[b]:off[b + 1]].double(), lse[off[b]:off[b + 1]].double()
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(x), nan), (b, "NaN")
        err = (x - want).abs()[~nan]
        allowed = (tol + half * (want.abs() + tol))[~nan]
        assert (err <= allowed).all(), (b, length, (err / allowed.clamp_min(1e-300)).max())
        none = torch.isinf(want_lse)
        assert torch.equal(torch.isnan(l), torch.isnan(want_lse)), (b, "lse NaN")
        assert torch.equal(l[none], want_lse[none])
        ok = ~none & ~torch.isnan(want_lse)
        # log of a sum whose relative error is the probabilities', 2^-22 of the larger parts
        lim = 1e-4 + 2.0 ** -20 * want_lse[ok].abs()
        assert ((l - want_lse)[ok].abs() <= lim).all(), (b, "lse")
    return got, lse


def filled(lengths, heads, page, dim, fmt, seed=30, spread=0.4, **kw):
    table, n_pages = ref.table_of(lengths, page, seed=seed, **kw)
    cache = ref.Cache(n_pages, heads, page, dim, fmt, seed=seed)
    for b, n in enumerate(lengths):
        cache.random_sequence(table[b], n, seed + b, spread)
    return cache, table


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("dim,page,wide", [(64, 32, 25), (64, 32, None), (128, 64, 40), (128, 64, None),
                                           (192, 96, None), (192, 96, 9), (256, 2048, None),
                                           (256, 160, None)])
@pytest.mark.parametrize("lengths,new,heads,group", [
    ([1, 31, 32, 33, 63, 64, 65, 200], [1] * 8, 2, 4),           # one token each
    ([0, 5, 300], [1, 1, 1], 1, 17),                             # no token; more than one row tile
    ([40, 130, 7, 96, 65], [3, 2, 7, 5, 0], 2, 3),               # a few
    ([70, 300], [9, 40], 1, 8),                                  # more rows than a workgroup has
    ([2, 90], [5, 33], 1, 1),                                    # rows before the first token
])
def test_attention(mx, lengths, new, heads, group, dim, page, wide, fmt, dtype):
    """Slots behind the tokens, blocks behind them and pages of nobody hold random bytes, NaN codes
    and scales among them. A table wider than the tokens: they may be divided among workgroups."""
    cache, table = filled(lengths, heads, page, dim, fmt, width=wide)
    check_attention(mx, cache, table, lengths, new, group, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_long(mx, dtype):
    """Chunks of several steps and their join, with a short sequence beside a long one."""
    lengths = [5000, 3, 1333]
    cache, table = filled(lengths, 1, 64, 128, 0, seed=40)
    check_attention(mx, cache, table, lengths, [1, 1, 1], 8, dtype, size=2.0)
    check_attention(mx, cache, table, lengths, [4, 2, 1], 8, dtype, seed=21)


@pytest.mark.parametrize("dtype,fmt", [("bf16", 0), ("f32", 1)])
@pytest.mark.parametrize("dim,page,wide", [(64, 32, 80), (128, 64, 30), (192, 96, 20), (256, 160, 12)])
@pytest.mark.parametrize("lengths,new,heads,group", [
    ([1, 700, 33, 0, 65, 1800], [1] * 6, 2, 4),
    ([700, 90, 1500], [9, 1, 20], 2, 3),
    ([400, 0, 1100], [40, 0, 3], 1, 8),
])
def test_attention_divided(mx, lengths, new, heads, group, dim, page, wide, fmt, dtype):
    """Tables that are too wide for a workgroup each."""
    cache, table = filled(lengths, heads, page, dim, fmt, width=wide, seed=41)
    check_attention(mx, cache, table, lengths, new, group, dtype)


@pytest.mark.parametrize("lengths,pages", [
    ([700, 30, 1500, 900], 40),      # 64 heads leave 8 workgroups each: a part is 2 steps a wave,
    ([2500, 1500, 900, 30], 40),     # 4 steps,
    ([6000, 30, 2500, 1500], 100),   # and cut evenly, with parts of several items
    ([1500, 700], 24),               # many heads, 1536 tokens: a workgroup each
])
@pytest.mark.parametrize("new", [1, 2])
def test_attention_many_heads(mx, lengths, pages, new):
    heads, page = 64, 64
    table, n_pages = ref.table_of([min(n, 1024) for n in lengths], page, seed=42, width=pages)
    cache = ref.Cache(n_pages, heads, page, 64, 0, seed=42)
    for b, n in enumerate(lengths):
        cache.random_sequence(table[b], min(n, 1024), 42 + b, 0.4)
        for i in range(16, -(-n // page)):  # the same pages again
            table[b, i] = table[b, i % 16]
    check_attention(mx, cache, table, lengths, [new] * len(lengths), 1, "bf16")


@pytest.mark.parametrize("lengths", [[13000], [13000, 9001], [0, 12800, 13000, 12500]])
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "f32")])
def test_attention_long_many_heads(mx, lengths, dim, dtype):
    """Long sequences, which half of the workgroups have: 128 heads leave 4 each."""
    heads, page = 128, 64
    table, n_pages = ref.table_of([min(n, 512) for n in lengths], page, seed=43, width=210)
    cache = ref.Cache(n_pages, heads, page, dim, 0, seed=43)
    for b, n in enumerate(lengths):
        cache.random_sequence(table[b], min(n, 512), 43 + b, 0.4)
        for i in range(8, -(-n // page)):
            table[b, i] = table[b, i % 8]
    check_attention(mx, cache, table, lengths, [1] * len(lengths), 1, dtype)


def test_attention_many_wide_sequences(mx):
    """More sequences than a wave has lanes or a workgroup has threads, divided."""
    for count, heads in ((70, 2), (600, 1), (65, 40)):
        lengths = [(37 * b) % 331 for b in range(count)]
        new = [min(n, b % 3) for b, n in enumerate(lengths)]
        cache, table = filled(lengths, heads, 32, 64, 0, seed=61, width=60)
        check_attention(mx, cache, table, lengths, new, 2, "bf16")
        one = [1] * count
        check_attention(mx, cache, table, lengths, one, 2, "bf16", seed=22)


@pytest.mark.parametrize("size,scale", [(60.0, None), (1.0, 5.0), (1.0, 0.0), (1.0, -0.3)])
def test_attention_scores(mx, size, scale):
    """One token that takes all, the mean, and a negative scale."""
    lengths = [130, 777]
    cache, table = filled(lengths, 2, 32, 64, 0, seed=50)
    check_attention(mx, cache, table, lengths, [2, 3], 2, "bf16", scale=scale, size=size)
    check_attention(mx, cache, table, lengths, [2, 3], 2, "f32", scale=scale, size=size)


def test_attention_many_sequences(mx):
    """More sequences than a workgroup has threads, some of them empty."""
    lengths = [(7 * b) % 90 for b in range(600)]
    new = [min(n, b % 3) for b, n in enumerate(lengths)]
    cache, table = filled(lengths, 1, 32, 64, 0, seed=60)
    check_attention(mx, cache, table, lengths, new, 2, "bf16")
    cache, table = filled(lengths, 1, 32, 64, 0, seed=60, width=30)
    check_attention(mx, cache, table, lengths, new, 2, "bf16")
    few = 70  # more than a wave has lanes, few enough for a workgroup each
    check_attention(mx, cache, table[:few, :4].contiguous(), lengths[:few], new[:few], 2, "bf16")


def test_attention_not_finite_block(mx):
    """A block with scale 0xFF makes the rows NaN that see one of its tokens, and no others."""
    lengths, new = [100, 80], [10, 2]
    for x, wide in (("k", None), ("v", None), ("k", 40), ("v", 40)):
        cache, table = filled(lengths, 2, 32, 64, 0, seed=70, width=wide)
        at = cache.block(table[0], 96)  # tokens 96 .. 99: seen by the last 4 of 10 rows
        (cache.ks if x == "k" else cache.vs)[at[0], 1, at[1]] = 255
        if x == "k":
            cache.kq[at[0], 1, 32 * at[1]:32 * at[1] + 32] = 0
        else:
            cache.vq[at[0], 1, at[1]] = 0
        got, _ = check_attention(mx, cache, table, lengths, new, 2, "bf16")
        assert torch.isnan(got[6:10, 2:]).all() and not torch.isnan(got[:6]).any()
        assert not torch.isnan(got[:, :2]).any()


@pytest.mark.parametrize("width", [None, 30])
def test_attention_missing_pages(mx, width):
    """Tokens without a page are not attended to; a sequence of nothing else gives zeros."""
    lengths, new = [200, 64, 150], [3, 1, 2]
    cache, table = filled(lengths, 2, 32, 64, 0, seed=80, width=width)
    table[0, 0], table[0, 3], table[0, 6] = -1, -7, cache.kq.shape[0]
    table[1, :] = -1
    check_attention(mx, cache, table, lengths, new, 2, "bf16")
    short = table[:, :3].contiguous()  # tokens beyond the table
    check_attention(mx, cache, short, lengths, new, 2, "bf16")
    none = ref.Cache(0, 2, 32, 64, 0)
    check_attention(mx, none, table, lengths, new, 2, "bf16")
    check_attention(mx, cache, table[:, :0].contiguous(), lengths, new, 2, "f32")


def test_attention_shared_pages(mx):
    """Sequences that begin with the same pages."""
    lengths = [100, 120, 96]
    table, n_pages = ref.table_of(lengths, 32, seed=90)
    table[1, :3], table[2, :3] = table[0, :3], table[0, :3]
    cache = ref.Cache(n_pages, 2, 32, 128, 1, seed=90)
    cache.random_sequence(table[1], 120, 1)
    k = rows(4, 2, 128, "f32", 2)
    cache.write(k, k, table[0], 100)
    check_attention(mx, cache, table, lengths, [1, 1, 1], 4, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_layouts(mx, dtype):
    """Queries and outputs inside larger buffers, heads before tokens, single rows; rows of nobody
    are left as they are."""
    lengths, new = [150, 40, 33], [1, 4, 2]
    cache, table = filled(lengths, 2, 32, 64, 0, seed=100)
    dev = [t.to(DEV) for t in cache.tensors()]
    off = [2, 3, 7, 9]
    T, heads = 12, 4
    q = rows(T, heads, 64, dtype, 11, 0.3)
    args = (*dev, table.to(DEV), i32(lengths))
    plain = torch.full((T, heads, 64), 7.0, dtype=DT[dtype], device=DEV)
    mx.mx_cache_attention(q.to(DEV), *args, offsets=i32(off), out=plain)
    assert (plain[:2] == 7.0).all() and (plain[9:] == 7.0).all() and not (plain[2:9] == 7.0).any()
    wide = torch.full((T, 3 * heads + 1, 64 + 16), 9.0, dtype=DT[dtype], device=DEV)
    wide[:, 1:1 + heads, :64] = q.to(DEV)
    out = torch.full((heads, T, 64), 7.0, dtype=DT[dtype], device=DEV)
    lse = torch.full((T, heads), 5.0, device=DEV)
    got, _ = mx.mx_cache_attention(wide[:, 1:1 + heads, :64], *args, offsets=i32(off),
                                   out=out.transpose(0, 1), lse=lse)
    assert torch.equal(got, plain) and got.data_ptr() == out.data_ptr()
    assert (lse[:2] == 5.0).all() and (lse[9:] == 5.0).all() and not (lse[2:9] == 5.0).any()
    # out beside q in one buffer of joint projections
    joint = torch.zeros((T, 2 * heads, 64), dtype=DT[dtype], device=DEV)
    joint[:, :heads] = q.to(DEV)
    got = mx.mx_cache_attention(joint[:, :heads], *args, offsets=i32(off), out=joint[:, heads:])
    assert torch.equal(got[2:9], plain[2:9])
    one = mx.mx_cache_attention(q[2:3].to(DEV), *dev, table[:1].to(DEV), i32(lengths[:1]))
    off1 = mx.mx_cache_attention(q[2:3].to(DEV), *dev, table[:1].to(DEV), i32(lengths[:1]), offsets=i32([0, 1]))
    assert torch.equal(one, off1)


def test_empty_calls(mx):
    """No rows, no sequences, no pages."""
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    cache = (z(2, 1, 32, 64), z(2, 1, 1), z(2, 1, 1, 64, 32), z(2, 1, 1))
    pages, lengths = i32([[0], [1]]), i32([4, 5])
    none = torch.zeros((0, 1, 64), device=DEV)
    assert mx.mx_cache_attention(none, *cache, pages, lengths, offsets=i32([0, 0, 0])).shape == (0, 1, 64)
    mx.mx_cache_write(none, none, *cache, pages, lengths, offsets=i32([0, 0, 0]))
    assert mx.mx_cache_read(*cache, pages, lengths, offsets=i32([0, 0, 0]), rows=0)[0].shape == (0, 1, 64)
    assert mx.mx_cache_attention(none, *cache, pages[:0], lengths[:0]).shape == (0, 1, 64)
    empty = (z(0, 1, 32, 64), z(0, 1, 1), z(0, 1, 1, 64, 32), z(0, 1, 1))
    q = torch.ones((2, 1, 64), device=DEV)
    mx.mx_cache_write(q, q, *empty, pages, lengths)
    assert (mx.mx_cache_read(*empty, pages, lengths)[0] == 0).all()
    out, lse = mx.mx_cache_attention(q, *empty, pages, lengths, with_lse=True)
    assert (out == 0).all() and torch.isinf(lse).all()


def test_same_bits_and_streams(mx):
    """Twice the same outputs; on another stream too."""
    lengths = [900, 33, 2000]
    cache, table = filled(lengths, 2, 64, 128, 0, seed=110)
    dev = [t.to(DEV) for t in cache.tensors()]
    q = rows(3, 8, 128, "bf16", 12, 0.3).to(DEV)
    args = (*dev, table.to(DEV), i32(lengths))
    a = mx.mx_cache_attention(q, *args)
    b = mx.mx_cache_attention(q, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c = mx.mx_cache_attention(q, *args, stream=side)
    k = rows(3, 2, 128, "bf16", 13).to(DEV)
    mx.mx_cache_write(k, k, *args, stream=side)
    r = mx.mx_cache_read(*args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b) and torch.equal(a, c)
    r2 = mx.mx_cache_read(*args)
    assert torch.equal(r[0], r2[0]) and torch.equal(r[1], r2[1])


@pytest.mark.parametrize("width", [None, 40])
def test_graph_with_growing_lengths(mx, width):
    """One captured step (write, then attend) replayed as the sequences grow, beside eager work."""
    heads, group, dim, page, B = 2, 4, 64, 32, 3
    start, steps = [30, 1, 200], 5
    table, n_pages = ref.table_of([n + steps for n in start], page, seed=120, width=width)
    cache = ref.Cache(n_pages, heads, page, dim, 0, seed=120)
    for b in range(B):
        cache.random_sequence(table[b], start[b], 120 + b)
    dev = [t.to(DEV) for t in cache.tensors()]
    eager = [t.clone() for t in dev]
    pages, lengths = table.to(DEV), i32(start)
    q, k, v = (torch.zeros((B, h, dim), dtype=torch.bfloat16, device=DEV)
               for h in (heads * group, heads, heads))
    out = torch.empty_like(q)
    side = torch.cuda.Stream()

    def step(c, o):
        lengths.add_(1)
        mx.mx_cache_write(k, v, *c, pages, lengths)
        return mx.mx_cache_attention(q, *c, pages, lengths, out=o)

    scratch = [t.clone() for t in dev]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(scratch, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(dev, out)
    lengths.copy_(i32(start))
    for s in range(steps):
        q.copy_(rows(B, heads * group, dim, "bf16", 200 + s, 0.3))
        k.copy_(rows(B, heads, dim, "bf16", 300 + s))
        v.copy_(rows(B, heads, dim, "bf16", 400 + s))
        graph.replay()
        now = lengths.clone()
        torch.cuda.synchronize()
        mx.mx_cache_write(k, v, *eager, pages, now)
        want = mx.mx_cache_attention(q, *eager, pages, now)
        assert now.tolist() == [n + s + 1 for n in start]
        for x, y in zip(dev, eager):
            assert torch.equal(x, y)
        assert torch.equal(out, want)


def test_far_pages(mx):
    """Code offsets beyond 2^32 bytes."""
    heads, page, dim = 8, 64, 128
    n_pages = (1 << 32) // (heads * page * dim) + 40
    kq = torch.empty((n_pages, heads, page, dim), dtype=torch.uint8, device=DEV)
    vq = torch.empty((n_pages, heads, page // 32, dim, 32), dtype=torch.uint8, device=DEV)
    ks = torch.empty((n_pages, heads, page // 32), dtype=torch.uint8, device=DEV)
    vs = torch.empty_like(ks)
    lengths = [150, 70]
    far = torch.tensor([[n_pages - 1, n_pages - 3, n_pages - 2], [n_pages - 30, 0, -1]], dtype=torch.int32)
    near, n_near = ref.table_of(lengths, page, seed=130, width=3)
    cache = ref.Cache(n_near, heads, page, dim, 0, seed=130)
    k, v = rows(220, heads, dim, "bf16", 14, 0.4), rows(220, heads, dim, "bf16", 15, 0.4)
    for b, (f, t) in enumerate(((0, 150), (150, 220))):
        cache.write(k[f:t], v[f:t], near[b], lengths[b])
    args = (kq, ks, vq, vs, far.to(DEV), i32(lengths))
    mx.mx_cache_write(k.to(DEV), v.to(DEV), *args, offsets=i32([0, 150, 220]))
    got = mx.mx_cache_read(*args, offsets=i32([0, 150, 220]), rows=220, out_dtype=torch.float32)
    for x, t in zip("kv", got):
        want = torch.cat([cache.tokens(x, near[b], 0, lengths[b])[0] for b in range(2)])
        assert torch.equal(t.cpu(), want.float())
    q = rows(2, 16, dim, "bf16", 16, 0.3).to(DEV)
    dev = [t.to(DEV) for t in cache.tensors()]
    assert torch.equal(mx.mx_cache_attention(q, *args),
                       mx.mx_cache_attention(q, *dev, near.to(DEV), i32(lengths)))


def test_attention_most_joined_rows(mx):
    """More rows than one dimension of the join's grid has threads for: 2^26 and a few, of one sequence
    whose table holds few tokens. Each of a head's 64 workgroups has many items and parts of two."""
    heads, group, dim, page, T = 8, 8, 64, 32, (1 << 20) + 3
    lengths = [1 << 20, 190]
    cache, table = filled([1920, 190], heads, page, dim, 0, seed=140)
    dev = [t.to(DEV) for t in cache.tensors()]
    few = T - (1 << 20)
    g = torch.Generator().manual_seed(141)
    one = torch.randn((1, heads * group, dim), generator=g).bfloat16()
    q = one.to(DEV).expand(T, -1, -1).contiguous()
    # the table has the first 1920 tokens of the first sequence: the rows from there on see the same
    got, lse = mx.mx_cache_attention(q, *dev, table.to(DEV), i32(lengths), offsets=i32([0, 1 << 20, T]),
                                     with_lse=True)
    seen = page * 60
    want, want_lse, tol = ref.attention(cache, one, table[0], seen, dim ** -0.5, P_EPS["bf16"])
    half = torch.finfo(torch.bfloat16).eps / 2
    limit = (tol + half * (want.abs() + tol))[0].to(DEV)
    lo, hi = want[0].to(DEV) - limit, want[0].to(DEV) + limit
    for first in range(seen - 1, 1 << 20, 1 << 16):
        part = got[first:min(first + (1 << 16), 1 << 20)].double()
        assert ((part >= lo) & (part <= hi)).all(), first
    assert ((lse[seen - 1:1 << 20].double() - want_lse[0].to(DEV)).abs() <= 1e-4 + 2.0 ** -20 * 8).all()
    want, _, tol = ref.attention(cache, one.expand(few, -1, -1), table[1], 190, dim ** -0.5, P_EPS["bf16"])
    err = (got[1 << 20:].cpu().double() - want).abs()
    assert (err <= tol + half * (want.abs() + tol)).all()


@pytest.mark.parametrize("bad", [1e4, math.inf])
def test_refused_drafts(mx, bad):
    """A draft that is written over: the block keeps the scale that it made where older tokens stay, and
    they what that scale left of them; written from the first slot on, it starts anew."""
    heads, dim, page = 1, 64, 32
    table, n_pages = ref.table_of([70], page)
    cache = ref.Cache(n_pages, heads, page, dim, 0, seed=150)
    dev = [t.to(DEV) for t in cache.tensors()]
    k, v = rows(70, heads, dim, "bf16", 151, 0.5), rows(70, heads, dim, "bf16", 152, 0.5)

    def write(first, count, kk=k, vv=v):
        kk, vv = kk[first:first + count], vv[first:first + count]
        off, n = i32([0, count]), first + count
        mx.mx_cache_write(kk.to(DEV), vv.to(DEV), *dev, table.to(DEV), i32([n]), offsets=off)
        cache.write(kk, vv, table[0], n)
        for name, got, want in zip(("kq", "ks", "vq", "vs"), dev, cache.tensors()):
            assert torch.equal(got.cpu(), want), (name, first, count)

    first, second = cache.block(table[0], 32), cache.block(table[0], 64)
    write(0, 40)
    before = int(cache.ks[first[0], 0, first[1]])
    draft = k.clone()
    draft[41], draft[66] = bad, bad
    write(40, 28, draft, v)     # in the block of tokens 32 .. and at the start of the next one
    large = int(cache.ks[first[0], 0, first[1]])
    assert large > before and (large == 255) == math.isinf(bad)
    write(40, 24)               # refused: the same positions again
    assert int(cache.ks[first[0], 0, first[1]]) == large
    write(64, 3)                # tokens 64 .. from the block's first slot on
    assert int(cache.ks[second[0], 0, second[1]]) < large
