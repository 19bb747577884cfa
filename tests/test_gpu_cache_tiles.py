"""Attention of sequences with several row tiles (16, 32 or 64 rows each) whose steps are cut evenly:
many cache heads leave few workgroups each, so that parts end inside tiles and sequences and most rows
are joined. Against float64, with the tolerance that cache_reference.attention derives."""
import math

import pytest
import torch

from tests import cache_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
P_EPS = {"bf16": 2.0 ** -16, "f32": 2.0 ** -23}


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_hadamard32_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.lib()
    return m


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


def attention(k, v, q, length, scale, p_eps):
    """cache_reference.attention for one head, all rows at once: k, v [tokens][dim] float64 (all of them
    exist), q [n][group][dim] -> out, tolerance [n][group][dim], lse [n][group]."""
    n, group, dim = q.shape
    u = 2.0 ** -24
    x = q.double().reshape(n * group, dim)
    seen = (length - n + 1 + torch.arange(n)).repeat_interleave(group)
    out = torch.zeros((n * group, dim), dtype=torch.float64)
    tol, lse = torch.zeros_like(out), torch.full((n * group,), -math.inf, dtype=torch.float64)
    rows = (seen > 0).nonzero()[:, 0]
    if len(rows):
        hidden = torch.arange(length) >= seen[rows, None]
        s = x[rows] @ k.T * scale
        size = (x[rows].abs() @ k.abs().T * abs(scale)).masked_fill(hidden, 0.0).amax(1)
        most = s.masked_fill(hidden, 0.0).abs().amax(1)
        s = s.masked_fill(hidden, -math.inf)
        w = torch.softmax(s, 1)
        rel = (dim + 8) * u * size + 8 * u * most + 8 * u
        out[rows] = w @ v
        lse[rows] = torch.logsumexp(s, 1)
        tol[rows] = (2 * rel + p_eps + (3 * seen[rows] / 8 + 64) * u)[:, None] * (w @ v.abs())
    return out.view(n, group, dim), tol.view(n, group, dim), lse.view(n, group)


def check(mx, lengths, new, heads, group, dim, page, width, dtype, fmt, seed):
    """Sequences of more than 512 tokens have the same 512 again and again."""
    table, n_pages = ref.table_of([min(n, 512) for n in lengths], page, seed=seed, width=width)
    cache = ref.Cache(n_pages, heads, page, dim, fmt, seed=seed)
    own = 512 // page
    kv = []
    for b, n in enumerate(lengths):
        held = min(n, 512)
        cache.random_sequence(table[b], held, seed + b, 0.4)
        one = [cache.tokens(x, table[b], 0, held)[0] for x in "kv"]
        for i in range(own, -(-n // page)):
            table[b, i] = table[b, i % own]
        kv.append([t[torch.arange(n) % 512] for t in one])
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    g = torch.Generator().manual_seed(seed + 1000)
    q = torch.randn((off[-1], heads * group, dim), generator=g).to(DT[dtype])
    dev = [t.to(DEV) for t in cache.tensors()]
    args = (q.to(DEV), *dev, table.to(DEV), i32(lengths))
    got, lse = mx.mx_cache_attention(*args, offsets=i32(off), fmt=fmt, with_lse=True)
    again = mx.mx_cache_attention(*args, offsets=i32(off), fmt=fmt)
    assert torch.equal(got, again)
    got, lse = got.cpu().double(), lse.cpu().double()
    half = torch.finfo(DT[dtype]).eps / 2
    for b, (length, n) in enumerate(zip(lengths, new)):
        for h in range(heads if n else 0):
            rows, cols = slice(off[b], off[b + 1]), slice(h * group, (h + 1) * group)
            want, tol, want_lse = attention(kv[b][0][:, h], kv[b][1][:, h], q[rows, cols], length, dim ** -0.5,
                                            P_EPS[dtype])
            err = (got[rows, cols] - want).abs()
            assert (err <= tol + half * (want.abs() + tol)).all(), (b, h, float(err.max()))
            none = torch.isinf(want_lse)
            l = lse[rows, cols]
            assert torch.equal(l[none], want_lse[none]), (b, h)
            assert ((l - want_lse)[~none].abs() <= 1e-4 + 2.0 ** -20 * want_lse[~none].abs()).all(), (b, h)


CASES = {  # lengths, newest tokens, group; 64 heads: 8 workgroups for each
    "tiles of 16": ([1500, 700, 30, 900], [40, 3, 1, 2], 1),
    "tiles of 16, half of the workgroups": ([6400, 6300, 6350, 6400], [13, 1, 1, 0], 4),
    "tiles of 32": ([1500, 700, 900, 30], [70, 10, 20, 5], 1),
    "tiles of 32, rows before the first token": ([40, 1900, 0, 700], [50, 9, 0, 3], 2),
    "tiles of 64": ([1500, 900, 10, 1300], [200, 41, 0, 100], 1),
    "tiles of 64, three query heads": ([800, 1200], [65, 30], 3),
}


def test_the_reference():
    """All rows at once give what cache_reference gives one by one."""
    table, n_pages = ref.table_of([90], 32)
    cache = ref.Cache(n_pages, 2, 32, 64, 0, seed=1)
    cache.random_sequence(table[0], 90, 2)
    for length, n in ((90, 7), (5, 9)):
        q = torch.randn((n, 4, 64), generator=torch.Generator().manual_seed(3))
        out, lse, tol = ref.attention(cache, q, table[0], length, 0.125, 2.0 ** -16)
        for h in range(2):
            k, v = (cache.tokens(x, table[0], 0, length)[0][:, h] for x in "kv")
            o, t, l = attention(k, v, q[:, 2 * h:2 * h + 2], length, 0.125, 2.0 ** -16)
            assert torch.allclose(o, out[:, 2 * h:2 * h + 2], rtol=1e-12, atol=1e-14)
            assert torch.allclose(t, tol[:, 2 * h:2 * h + 2], rtol=1e-12, atol=0)
            assert torch.allclose(l, lse[:, 2 * h:2 * h + 2], rtol=1e-12)


@pytest.mark.parametrize("dtype,fmt", [("bf16", 0), ("f32", 1)])
@pytest.mark.parametrize("dim,page", [(64, 32), (128, 64), (192, 64), (256, 128)])
@pytest.mark.parametrize("case", list(CASES))
def test_few_sequences(mx, case, dim, page, dtype, fmt):
    lengths, new, group = CASES[case]
    check(mx, lengths, new, 64, group, dim, page, 6656 // page, dtype, fmt, seed=200)


@pytest.mark.parametrize("dim,page,dtype,fmt", [(64, 32, "bf16", 0), (128, 64, "f32", 1), (192, 64, "bf16", 0),
                                                (256, 128, "f32", 0)])
@pytest.mark.parametrize("every,many", [(7, 60), (5, 80), (4, 170)])
def test_more_sequences_than_lanes(mx, every, many, dim, page, dtype, fmt):
    """70 sequences, one of `every` with `many` new tokens (16, 32 and 64 rows a tile), others with up to
    two."""
    lengths = [(97 * b) % 331 for b in range(70)]
    new = [min(n, many if b % every == 0 else b % 3) for b, n in enumerate(lengths)]
    new[3 * every] = lengths[3 * every] + 2  # more rows than tokens
    check(mx, lengths, new, 32, 2, dim, page, 2048 // page, dtype, fmt, seed=300)


def test_two_turns_of_threads(mx):
    """300 sequences: a workgroup's threads go over them twice."""
    lengths = [(53 * b) % 211 for b in range(300)]
    new = [min(n, 40 if b % 20 == 0 else b % 2) for b, n in enumerate(lengths)]
    check(mx, lengths, new, 16, 3, 64, 32, 64, "bf16", 0, seed=400)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("low,high,size", [(0, 13, 2.0 ** 108), (1, 30, 2.0 ** 90), (225, 238, 2.0 ** -100)])
@pytest.mark.parametrize("dim,width", [(64, None), (128, 60), (256, 30)])
def test_ends_of_the_scales(mx, low, high, size, fmt, dim, width, dtype):
    """Scale bytes down to 0, which stands for a subnormal, and up to where sums of the values stay in
    fp32's range. A code times its scale is exact down to bf16's least subnormal, 2^-133: below, half
    of that comes to every key and value."""
    lengths, new, heads, group, page = [90, 33], [3, 1], 2, 2, 32
    table, n_pages = ref.table_of(lengths, page, width=width, seed=500)
    cache = ref.Cache(n_pages, heads, page, dim, fmt, seed=500)
    for b, n in enumerate(lengths):
        cache.random_sequence(table[b], n, 500 + b, 0.4)
    g = torch.Generator().manual_seed(501)
    for s in (cache.ks, cache.vs):
        s.copy_(torch.randint(low, high, s.shape, generator=g, dtype=torch.uint8))
    q = (size * torch.randn((4, heads * group, dim), generator=g)).to(DT[dtype])
    dev = [t.to(DEV) for t in cache.tensors()]
    f = dim ** -0.5
    got = mx.mx_cache_attention(q.to(DEV), *dev, table.to(DEV), i32(lengths), offsets=i32([0, 3, 4]),
                                fmt=fmt).cpu().double()
    half, least = torch.finfo(DT[dtype]).eps / 2, 2.0 ** -134
    row = 0
    for b, (length, n) in enumerate(zip(lengths, new)):
        x = q[row:row + n]
        want, _, tol = ref.attention(cache, x, table[b], length, f, P_EPS[dtype])
        v = cache.tokens("v", table[b], 0, length)[0].abs().amax((0, 2)).repeat_interleave(group)
        score = 2 * least * x.double().abs().sum(2, keepdim=True) * f
        tol = tol + 2 * score * v[None, :, None] + 2 * least
        err = (got[row:row + n] - want).abs()
        assert torch.isfinite(got[row:row + n]).all()
        assert (err <= tol + half * (want.abs() + tol) + least).all(), float((err / want.abs().amax()).max())
        row += n
