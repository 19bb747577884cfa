"""The decoding modules together: norm, MXFP4 projections with low-rank adapters, cache and attention,
step after step. Every stage is checked against float64 on the inputs that it had."""
import numpy as np
import pytest
import torch

import workloads as wl
from tests import cache_reference as ref
from tests.test_gpu_cache import P_EPS, i32
from tests.test_gpu_lora import U, expected

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def lin():
    from mxfp4_block_scaled_hadamard32_amd import linear
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return linear


class Layer(torch.nn.Module):
    """x -> norm -> one projection to queries, keys and values (adapters beside it) -> attention ->
    output projection -> x + that."""

    def __init__(self, lin, hidden, heads, group, dim, pages, page, adapters, rank, hadamard, seed=1):
        super().__init__()
        g = torch.Generator().manual_seed(seed)
        width = (heads * group + 2 * heads) * dim
        spec = lin.QuantSpec(hadamard=int(hadamard), sign_mask=wl.sign_mask() if hadamard else 0)
        rnd = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.norm = lin.MXRMSNorm(hidden, device=DEV)
        self.w_in = rnd(width, hidden).bfloat16() * hidden ** -0.5
        self.w_out = rnd(hidden, heads * group * dim).bfloat16() * 0.05
        self.qkv = lin.MXDecodeLinear(self.w_in.to(DEV), spec)
        self.out = lin.MXDecodeLinear(self.w_out.to(DEV), lin.QuantSpec(), w_block=32)
        a = (rnd(adapters, rank, hidden) * hidden ** -0.5).bfloat16()
        b = (rnd(adapters, width, rank) * 0.3).bfloat16()
        s = 0.5 + torch.rand((adapters,), generator=g)
        self.adapters = lin.MXAdapters(a.to(DEV), b.to(DEV), s.to(DEV))
        self.cache = lin.MXCache(pages, heads, dim, page, device=DEV)
        self.sizes = heads, group, dim

    def forward(self, x, index, pages, lengths, offsets=None, seen=None):
        heads, group, dim = self.sizes
        y = self.norm(x)
        z = self.qkv(y, self.adapters, index)
        h = z.view(x.shape[0], (group + 2) * heads, dim)
        q, k, v = h[:, :group * heads], h[:, group * heads:(group + 1) * heads], h[:, (group + 1) * heads:]
        o = self.cache(q, k, v, pages, lengths, offsets)
        r = self.out(o.view(x.shape[0], -1))
        if seen is not None:
            seen.update(y=y, z=z, q=q, k=k, v=v, o=o, r=r)
        return x + r


def weights(orc, layer):
    w = orc.dequantize_f64(layer.codes.cpu().numpy(), layer.scales.cpu().numpy(), layer.codes.shape[0],
                           2 * layer.codes.shape[1], layer.w_block)
    return torch.from_numpy(np.asarray(w))


def close(got, want, size):
    got = got.cpu()
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double() - want).abs()
    allowed = size + half * (want.abs() + size) + 1e-40
    assert (err <= allowed).all(), float((err / allowed).max())


def check_stages(orc, layer, cache, table, lengths, new, index, seen):
    heads, group, dim = layer.sizes
    y = seen["y"].detach().cpu()
    W, K = weights(orc, layer.qkv), y.shape[1]
    X, turned = y.double(), 0.0
    if layer.qkv.spec.hadamard:
        from tests.norm_reference import hadamard_f64
        X = torch.from_numpy(hadamard_f64(X.numpy(), layer.qkv.spec.sign_mask)) / 32
        # five stages, each rounds values of at most the block's sum of magnitudes
        blocks = y.double().abs().view(-1, K // 32, 32).sum(2).repeat_interleave(32, 1) / 32
        turned = 5 * U * (blocks @ W.abs().T)
    # the projection in fp32, the documented bound; then the adapters' and the single rounding
    base, size = X @ W.T, ((160 + K / 128) * U) * (X.abs() @ W.abs().T) + turned
    ad = layer.adapters
    want, more = expected(y, ad.a.cpu(), ad.b.cpu(), index, ad.scaling.cpu(), None)
    close(seen["z"], base + want, size + more + 8 * U * base.abs())
    row = 0
    k, v, q = (seen[n].cpu() for n in "kvq")
    for b, (length, n) in enumerate(zip(lengths, new)):
        cache.write(k[row:row + n], v[row:row + n], table[b], length)
        o, _, tol = ref.attention(cache, q[row:row + n], table[b], length, dim ** -0.5, P_EPS["bf16"])
        close(seen["o"][row:row + n], o, tol)
        row += n
    for name, t in zip(("kq", "ks", "vq", "vs"), cache.tensors()):
        assert torch.equal(getattr(layer.cache, name).cpu(), t), name
    O, Wo = seen["o"].cpu().double().reshape(row, -1), weights(orc, layer.out)
    close(seen["r"], O @ Wo.T, (160 + O.shape[1] / 128) * U * (O.abs() @ Wo.abs().T))


def mirror(layer, pages, page):
    """The module's cache, zeros at first, as the reference keeps it."""
    heads, _, dim = layer.sizes
    c = ref.Cache(pages, heads, page, dim)
    for t in c.tensors():
        t.zero_()
    return c


@pytest.mark.parametrize("hadamard", [False, True])
def test_prompts_then_tokens(lin, orc, hadamard):
    """Ragged prompts, then a few steps of one token each, then drafts of several tokens."""
    page, prompts, B = 32, [40, 1, 95], 3
    total = [n + 8 for n in prompts]
    table, pages = ref.table_of(total, page, seed=1)
    layer = Layer(lin, 256, 2, 4, 64, pages, page, adapters=3, rank=16, hadamard=hadamard)
    cache = mirror(layer, pages, page)
    tables, lengths = table.to(DEV), list(prompts)
    g = torch.Generator().manual_seed(5)
    for step, new in enumerate([prompts, [1, 1, 1], [1, 1, 1], [3, 1, 4], [1, 1, 1]]):
        if step:
            lengths = [l + n for l, n in zip(lengths, new)]
        off = [0]
        for n in new:
            off.append(off[-1] + n)
        index = torch.cat([torch.full((n,), (2, -1, 0)[b], dtype=torch.int32) for b, n in enumerate(new)])
        x = torch.randn((off[-1], 256), generator=g).bfloat16()
        seen = {}
        offsets = None if max(new) == 1 and len(new) == B else i32(off)
        layer(x.to(DEV), index.to(DEV), tables, i32(lengths), offsets, seen=seen)
        check_stages(orc, layer, cache, table, lengths, new, index, seen)


def test_captured_steps(lin):
    """A captured step, replayed while the sequences grow, gives what eager steps give."""
    page, start, steps = 32, [31, 5, 64, 0], 4
    B = len(start)
    table, pages = ref.table_of([n + steps + 1 for n in start], page, seed=2)
    make = lambda: Layer(lin, 512, 2, 4, 128, pages, page, adapters=5, rank=8, hadamard=False)  # noqa: E731
    eager, captured = make(), make()
    tables, lengths = table.to(DEV), i32(start)
    index = torch.tensor([4, 0, -1, 4], dtype=torch.int32, device=DEV)
    x = torch.zeros((B, 512), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(6)
    off = [0, 31, 36, 100, 100]
    for layer in (eager, captured):  # the same prompts
        p = torch.randn((100, 512), generator=torch.Generator().manual_seed(7)).bfloat16().to(DEV)
        idx = torch.zeros(100, dtype=torch.int32, device=DEV)
        layer(p, idx, tables, lengths, i32(off))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    warm = make()
    with torch.cuda.stream(side):
        warm(x, index, tables, lengths)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lengths.add_(1)
        out = captured(x, index, tables, lengths)
    lengths.copy_(i32(start))
    for s in range(steps):
        x.copy_(torch.randn((B, 512), generator=g).bfloat16())
        index.copy_(torch.randint(-1, 5, (B,), generator=g, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert lengths.tolist() == [n + s + 1 for n in start]
        want = eager(x, index, tables, lengths)
        assert torch.equal(out, want)


def test_modules_copy_what_kernels_cannot_read(lin):
    """Views at any element, expanded heads, channels that are not contiguous; refusals of the modules."""
    cache, same = (lin.MXCache(4, 2, 64, 32, device=DEV) for _ in range(2))
    pages, lengths = i32([[0, 1], [3, 2]]), i32([33, 7])
    g = torch.Generator().manual_seed(8)
    flat = torch.randn((4000,), generator=g).bfloat16().to(DEV)
    k = flat[1:1 + 2 * 2 * 64].view(2, 2, 64)
    v = flat[301:301 + 2 * 64].view(2, 1, 64).expand(2, 2, 64)
    q = flat[1000:1000 + 64 * 2 * 4].view(64, 2, 4).permute(1, 2, 0)
    got = cache(q, k, v, pages, lengths)
    want = same(q.contiguous(), k.clone(), v.contiguous(), pages, lengths)
    assert torch.equal(got, want) and torch.equal(cache.kq, same.kq) and torch.equal(cache.vq, same.vq)
    a, b = cache.read(pages, lengths), same.read(pages, lengths)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ValueError):
        lin.MXCache(4, 2, 96, device=DEV)
    with pytest.raises(ValueError):
        lin.MXCache(4, 2, 64, 48, device=DEV)
    layer = lin.MXDecodeLinear(torch.randn((64, 64), device=DEV).bfloat16())
    x = torch.randn((2, 3, 64), device=DEV).bfloat16()
    ad = lin.MXAdapters(torch.randn((2, 8, 64), device=DEV).bfloat16(), torch.randn((2, 64, 8), device=DEV).bfloat16())
    with pytest.raises(ValueError):
        layer(x, ad)
    none = torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    assert torch.equal(layer(x, ad, none), layer(x))
    assert layer(x, ad, none + 1).shape == (2, 3, 64)
    with pytest.raises(ValueError):
        lin.MXAdapters(torch.zeros((2, 8, 64)), torch.zeros((2, 64, 16)))
