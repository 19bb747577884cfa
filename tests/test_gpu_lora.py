"""Low-rank adapters against float64. With u = 2^-24: A x is an fp32 sum of K products (exact for
bf16), formed by the matrix core and joined in parts: at most K + 64 roundings or dropped parts of
u sum |a x|; fp32 products add one each. The sum over the rank, the scaling and the addition of base
are another rank + 8 units of their magnitudes, the output one rounding."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_hadamard32_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.lib()
    return m


def operands(T, N, K, r, E, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, K), generator=g) * torch.exp(torch.randn((T, 1), generator=g))
    a = torch.randn((E, r, K), generator=g) * K ** -0.5
    b = torch.randn((E, N, r), generator=g) * torch.exp(torch.randn((E, 1, 1), generator=g))
    index = torch.randint(-1, E + 1, (T,), generator=g, dtype=torch.int32)
    scaling = 2 * torch.rand((E,), generator=g) - 0.5
    base = torch.randn((T, N), generator=g)
    return x.to(DT[dtype]), a.to(DT[dtype]), b.to(DT[dtype]), index, scaling, base


def expected(x, a, b, index, scaling, base):
    T, K = x.shape
    E, r = a.shape[0], a.shape[1]
    y = torch.zeros((T, b.shape[1]), dtype=torch.float64)
    size = y.clone()
    for t in range(T):
        e = int(index[t])
        if 0 <= e < E:
            s = 1.0 if scaling is None else float(scaling[e])
            xd, ad, bd = x[t].double(), a[e].double(), b[e].double()
            h = ad @ xd
            y[t] = s * (bd @ h)
            size[t] = abs(s) * (bd.abs() @ ((K + 64) * U * (ad.abs() @ xd.abs()) + (r + 8) * U * h.abs()))
    if base is not None:
        y, size = y + base.double(), size + 8 * U * base.double().abs()
    return y, size


def check(got, want, size):
    half = torch.finfo(got.dtype).eps / 2
    err = (got.cpu().double() - want).abs()
    allowed = size + half * (want.abs() + size) + 1e-40
    assert (err <= allowed).all(), float((err / allowed).max())


SIZES = [  # T, N, K, rank, adapters
    (1, 17, 32, 8, 1), (1, 4096, 4096, 16, 8), (1, 300, 8, 128, 3), (3, 1003, 4128, 24, 2),
    (16, 256, 264, 16, 40), (37, 1003, 4128, 40, 5), (64, 512, 2720, 64, 64), (65, 130, 320, 8, 70),
    (130, 64, 1024, 128, 200), (200, 700, 96, 72, 3), (5, 1, 8192, 16, 2), (260, 33, 72, 32, 1),
    (2, 14336, 128, 48, 1),
    # one kernel for bf16: the largest K, more tokens than adapters, N and K odd multiples
    (16, 3000, 4096, 16, 16), (7, 1003, 1000, 8, 3), (16, 40, 8, 8, 1), (1, 14336, 4096, 16, 8),
    (12, 2049, 3528, 16, 30),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K,r,E", SIZES)
def test_against_float64(mx, T, N, K, r, E, dtype):
    x, a, b, index, scaling, base = operands(T, N, K, r, E, dtype)
    d = [t.to(DEV) for t in (x, a, b, index)]
    for bs, s, out in ((base, scaling, "bf16"), (base.bfloat16(), None, "f32"), (None, scaling, "f32"),
                       (base, None, "f32")):
        want, size = expected(x, a, b, index, s, bs)
        got = mx.mx_lora(*d, base=None if bs is None else bs.to(DEV),
                         scaling=None if s is None else s.to(DEV), out_dtype=DT[out])
        assert got.dtype == DT[out]
        check(got, want, size)


@pytest.mark.parametrize("T", [150, 15])
@pytest.mark.parametrize("which", ["none", "one", "runs", "all"])
def test_orders(mx, which, T):
    """Tokens of one adapter, in runs, each its own, and none: the same bits in any order."""
    N, K, r, E = 320, 512, 16, 150
    x, a, b, index, scaling, base = operands(T, N, K, r, E, "bf16", seed=2)
    t = torch.arange(T, dtype=torch.int32)
    index = {"none": torch.full_like(t, -5), "one": torch.full_like(t, 149), "runs": t // 37, "all": t.flip(0)}[which]
    d = [y.to(DEV) for y in (x, a, b, index, scaling, base)]
    got = mx.mx_lora(d[0], d[1], d[2], d[3], base=d[5], scaling=d[4])
    want, size = expected(x, a, b, index, scaling, base)
    check(got, want, size)
    if which == "none":
        assert torch.equal(got.cpu(), base)
    perm = torch.randperm(T, generator=torch.Generator().manual_seed(3)).to(DEV)
    again = mx.mx_lora(d[0][perm], d[1], d[2], d[3][perm], base=d[5][perm], scaling=d[4])
    assert torch.equal(again, got[perm])  # whichever tokens share a product


def test_types_and_defaults(mx):
    x, a, b, index, scaling, base = operands(5, 40, 64, 8, 3, "bf16", seed=4)
    d = [y.to(DEV) for y in (x, a, b, index)]
    assert mx.mx_lora(*d).dtype == torch.bfloat16
    assert mx.mx_lora(*d, base=base.to(DEV)).dtype == torch.float32
    assert mx.mx_lora(*d, base=base.to(DEV), out_dtype=torch.bfloat16).dtype == torch.bfloat16


@pytest.mark.parametrize("out_dtype", ["bf16", "f32"])
def test_in_place_and_layouts(mx, out_dtype):
    """out that is base; rows of larger buffers at addresses that are not 16-byte aligned."""
    x, a, b, index, scaling, base = operands(70, 1003, 96, 16, 4, "bf16", seed=5)
    base = base.to(DT[out_dtype])
    d = [y.to(DEV) for y in (x, a, b, index)]
    s = scaling.to(DEV)
    want = mx.mx_lora(*d, base=base.to(DEV), scaling=s)
    own = base.to(DEV)
    got = mx.mx_lora(*d, base=own, scaling=s, out=own)
    assert got is own and torch.equal(own, want)
    wide = torch.full((70, 1100), 3.0, dtype=DT[out_dtype], device=DEV)
    wide[:, 5:1008] = base.to(DEV)
    xw = torch.zeros((70, 200), dtype=torch.bfloat16, device=DEV)
    xw[:, 8:104] = d[0]
    out = wide[:, 5:1008]
    mx.mx_lora(xw[:, 8:104], *d[1:], base=out, scaling=s, out=out)
    assert torch.equal(out, want) and (wide[:, :5] == 3.0).all() and (wide[:, 1008:] == 3.0).all()


def test_others_infinities_stay_theirs(mx):
    """An adapter, or a token, that is not finite spoils its own rows alone."""
    x, a, b, index, scaling, base = operands(20, 100, 64, 16, 4, "bf16", seed=6)
    index = torch.arange(20, dtype=torch.int32) % 4
    want, size = expected(x, a, b, index, scaling, base)
    a[1, 3, 5], b[2, 7] = math.inf, math.nan
    x[4, 0] = math.nan
    d = [y.to(DEV) for y in (x, a, b, index)]
    got = mx.mx_lora(*d, base=base.to(DEV), scaling=scaling.to(DEV)).cpu()
    assert torch.isnan(got[4]).all() and torch.isnan(got[2::4, 7]).all()
    good = [t for t in range(20) if t % 4 in (0, 3) and t != 4]
    check(got[good], want[good], size[good])
    rest = [n for n in range(100) if n != 7]
    check(got[2::4][:, rest], want[2::4][:, rest], size[2::4][:, rest])


def test_nothing_to_add(mx):
    """No adapters, no tokens, no outputs, no rank."""
    dev = dict(device=DEV)
    x = torch.ones((3, 16), **dev)
    i = torch.zeros(3, dtype=torch.int32, **dev)
    base = torch.arange(15.0, **dev).view(3, 5)
    e = lambda *s: torch.zeros(s, **dev)  # noqa: E731
    assert torch.equal(mx.mx_lora(x, e(0, 8, 16), e(0, 5, 8), i, base=base), base)
    assert torch.equal(mx.mx_lora(x, e(2, 0, 16), e(2, 5, 0), i, base=base), base)
    assert torch.equal(mx.mx_lora(e(3, 0), e(2, 8, 0), e(2, 5, 8), i, base=base), base)
    assert (mx.mx_lora(x, e(0, 8, 16), e(0, 5, 8), i) == 0).all()
    assert mx.mx_lora(e(0, 16), e(2, 8, 16), e(2, 5, 8), i[:0]).shape == (0, 5)
    assert mx.mx_lora(x, e(2, 8, 16), e(2, 0, 8), i).shape == (3, 0)


def test_stream_and_graph(mx):
    """On another stream; captured and replayed with other tokens and other adapters, with eager work
    between."""
    T, N, K, r, E = 9, 600, 512, 16, 4
    x, a, b, index, scaling, base = operands(T, N, K, r, E, "bf16", seed=7)
    d = [y.to(DEV) for y in (x, a, b, index, scaling, base)]
    want = mx.mx_lora(*d[:4], base=d[5], scaling=d[4])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mx.mx_lora(*d[:4], base=d[5], scaling=d[4], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mx.mx_lora(*d[:4], base=d[5], scaling=d[4], out=out)
    for seed in range(4):
        x, _, _, index, _, base = operands(T, N, K, r, E, "bf16", seed=20 + seed)
        for t, y in ((d[0], x), (d[3], index), (d[5], base)):
            t.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mx.mx_lora(*d[:4], base=d[5], scaling=d[4]))


def test_many_tokens(mx):
    """Beyond 2^31 bytes of base and output."""
    T, N, K, r, E = 40000, 14336, 64, 8, 3
    g = torch.Generator(device=DEV).manual_seed(8)
    x = torch.randn((T, K), generator=g, device=DEV).bfloat16()
    a = torch.randn((E, r, K), generator=g, device=DEV).bfloat16()
    b = torch.randn((E, N, r), generator=g, device=DEV).bfloat16()
    index = torch.randint(-1, E, (T,), generator=g, device=DEV, dtype=torch.int32)
    base = torch.randn((T, N), generator=g, device=DEV)
    got = mx.mx_lora(x, a, b, index, base=base)
    rows = torch.tensor([0, 1, 63, 64, 20000, T - 2, T - 1], device=DEV)
    want, size = expected(x[rows].cpu(), a.cpu(), b.cpu(), index[rows].cpu(), None, base[rows].cpu())
    check(got[rows], want, size)
