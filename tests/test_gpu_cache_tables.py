"""Tables that break the contract: offsets that fall, are negative or too large, lengths and pages that
are nothing of the kind. What the rows get is not said; nothing outside the tensors may be read or
written, and nothing of the cache by a call that only reads it."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BIG, SMALL = 2 ** 31 - 1, -2 ** 31
MARGIN = 1 << 20


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_hadamard32_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.lib()
    return m


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


class Guarded:
    """A tensor with MARGIN bytes before and behind it that must not change."""

    def __init__(self, shape, dtype):
        size = torch.empty((), dtype=dtype).element_size()
        for n in shape:
            size *= n
        self.all = torch.full((2 * MARGIN + size,), 0x5A, dtype=torch.uint8, device=DEV)
        self.own = self.all[MARGIN:MARGIN + size].view(dtype).view(shape)

    def untouched(self):
        return bool((self.all[:MARGIN] == 0x5A).all() and (self.all[-MARGIN:] == 0x5A).all())


def cache_of(n_pages, heads, page, dim, seed):
    shapes = ((n_pages, heads, page, dim), (n_pages, heads, page // 32),
              (n_pages, heads, page // 32, dim, 32), (n_pages, heads, page // 32))
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = [Guarded(s, torch.uint8) for s in shapes]
    for t in out:
        t.own.random_(0, 120, generator=g)
    return out


def calls(mx, offsets, lengths, pages, T, heads=2, group=2, page=32, dim=64):
    """Every entry point with these tables, its outputs guarded."""
    n_pages = 9
    cache = cache_of(n_pages, heads, page, dim, 1)
    tables = (i32(pages), i32(lengths))
    kw = {"offsets": i32(offsets)}
    args = [t.own for t in cache]
    held = [t.clone() for t in args]
    for dtype in (torch.bfloat16, torch.float32):
        q, out = (Guarded((T, heads * group, dim), dtype) for _ in range(2))
        lse = Guarded((T, heads * group), torch.float32)
        k, v = (Guarded((T, heads, dim), dtype) for _ in range(2))
        for t in (q, k, v):
            t.own.normal_()
        before = q.own.clone()
        mx.mx_cache_attention(q.own, *args, *tables, out=out.own, lse=lse.own, **kw)
        mx.mx_cache_read(*args, *tables, k=k.own, v=v.own, **kw)
        torch.cuda.synchronize()
        assert torch.equal(q.own, before)
        assert all(torch.equal(a, b) for a, b in zip(args, held))
        for t in (q, out, lse, k, v, *cache):
            assert t.untouched()
        mx.mx_cache_write(k.own, v.own, *args, *tables, **kw)
        torch.cuda.synchronize()
        for t in (k, v, *cache):
            assert t.untouched()
        for t, was in zip(args, held):
            t.copy_(was)


@pytest.mark.parametrize("seqs", [3, 64, 65, 300])
@pytest.mark.parametrize("width", [2, 70])
def test_any_contents(mx, seqs, width):
    g = torch.Generator().manual_seed(seqs + width)
    T = 200
    pick = lambda choices, n: torch.tensor(choices)[torch.randint(0, len(choices), (n,), generator=g)]  # noqa: E731
    for _ in range(3):
        offsets = pick([0, 0, 5, 31, 32, 100, 199, 200, 201, 5000, -1, -33, BIG, SMALL], seqs + 1)
        lengths = pick([0, 1, 33, 64, 190, 2000, -1, -500, BIG, SMALL], seqs)
        pages = pick([0, 1, 2, 3, 4, 5, 6, 7, 8, 9, -1, BIG, SMALL], seqs * width).view(seqs, width)
        calls(mx, offsets, lengths, pages, T)


def falling(pairs, T):
    """Offsets 0, T, 0, T, ..: `pairs` sequences of all T rows, one of none between each two."""
    return [0, T] * pairs


@pytest.mark.parametrize("pairs,more", [(32, 1), (64, 4), (64, 200)])
def test_sums_of_steps_wrap(mx, pairs, more):
    """Sequences that claim every row give 2^32 steps between them, and the following ones a few: in a
    wave's lanes, in a workgroup's threads, and beyond the first 256 of them."""
    T, group, width, page, dim = (8192 if pairs == 64 else 16384), 8, 65536, 64, 64
    offsets = falling(pairs, T) + [T + 1 + i for i in range(more)]
    rows, seqs = offsets[-1], len(offsets) - 1
    lengths = [width * page if offsets[b + 1] > offsets[b] + 1 else 3 * page for b in range(seqs)]
    # 64 rows an item, 64 tokens a step
    assert pairs * (T * group // 64) * (width * page // 64) == 1 << 32
    cache = cache_of(3, 1, page, dim, 2)
    args = [t.own for t in cache]
    pages = torch.zeros((seqs, width), dtype=torch.int32, device=DEV)
    q, out = (Guarded((rows, group, dim), torch.bfloat16) for _ in range(2))
    lse = Guarded((rows, group), torch.float32)
    q.own.normal_()
    mx.mx_cache_attention(q.own, *args, pages, i32(lengths), offsets=i32(offsets), out=out.own, lse=lse.own)
    torch.cuda.synchronize()
    for t in (q, out, lse, *cache):
        assert t.untouched()
