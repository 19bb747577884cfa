"""CPU checks of the cache's entry points: every refusal of the C ABI (before any HIP call; no pointer
here is dereferenced) and of the binding (before the library)."""
import ctypes
import os

import pytest
import torch

A, B, C, ODD = 0x100000, 0x4000000, 0x8000000, 0x100008
DIMS = dict(n_pages=4, seqs=3, table_width=2, heads=2, dim=64, page_size=64, fmt=0)


@pytest.fixture(scope="module")
def m():
    from mxfp4_block_scaled_hadamard32_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libmx.so not built (run __graft_entry__.build())")
    _lib.lib()
    return _lib


def cache_of(m, **kw):
    v = dict(kq=0x20000000, ks=0x21000000, vq=0x22000000, vs=0x23000000, pages=0x24000000,
             lengths=0x25000000, offsets=None, **DIMS)
    v.update({k: x for k, x in kw.items() if k in v})
    return m.mx_cache(**v)


def call(m, name, **kw):
    c = cache_of(m, **kw) if kw.get("cache", True) else None
    T, heads = kw.get("T", 3), c.heads if c is not None else 2
    row = lambda p, h: m.mx_rows(kw.get(p, {"a": A, "b": B}[p]), kw.get("token", h * 64),  # noqa: E731
                                 kw.get("head", 64))
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    dtype, L = kw.get("dtype", 1), m.lib()
    if name == "mx_cache_attention":
        qh = kw.get("q_heads", 4)
        return L.mx_cache_attention(ref(row("a", qh)), ref(row("b", qh)), kw.get("lse"), dtype, T, qh,
                                    kw.get("scale", 0.125), ref(c), kw.get("workspace", C),
                                    kw.get("size", 1 << 30), None)
    a, b = (None if kw.get(p, 1) is None and p in kw.get("no_rows", "") else row(p, heads) for p in "ab")
    if name == "mx_cache_write":
        return L.mx_cache_write(ref(a), ref(b), dtype, T, ref(c), kw.get("rule", 0), None)
    return L.mx_cache_read(ref(a), ref(b), dtype, T, ref(c), None)


NAMES = ["mx_cache_write", "mx_cache_read", "mx_cache_attention"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("bad,status", [
    (dict(cache=False), "NULL"), (dict(T=-1), "SHAPE"), (dict(seqs=-1, offsets=0x26000000), "SHAPE"),
    (dict(n_pages=-1), "SHAPE"), (dict(table_width=-1), "SHAPE"), (dict(heads=-1), "SHAPE"),
    (dict(T=4), "SHAPE"), (dict(fmt=2), "ARG"), (dict(fmt=-1), "ARG"), (dict(page_size=0), "ARG"),
    (dict(page_size=48), "ARG"), (dict(page_size=2080), "ARG"), (dict(page_size=-32), "ARG"),
    (dict(dim=32), "UNSUPPORTED"), (dict(dim=96), "UNSUPPORTED"), (dict(dim=320), "UNSUPPORTED"),
    (dict(dim=0), "UNSUPPORTED"), (dict(seqs=(1 << 20) + 1, T=(1 << 20) + 1), "UNSUPPORTED"),
    (dict(T=(1 << 24) + 1, offsets=0x26000000), "UNSUPPORTED"), (dict(n_pages=1 << 31), "UNSUPPORTED"),
    (dict(heads=65536, q_heads=65536), "UNSUPPORTED"), (dict(table_width=1 << 31), "UNSUPPORTED"),
    (dict(kq=ODD), "ARG"), (dict(vq=ODD), "ARG"), (dict(pages=0x24000002), "ARG"),
    (dict(lengths=0x25000001), "ARG"), (dict(offsets=0x26000002), "ARG"),
    (dict(kq=None), "NULL"), (dict(ks=None), "NULL"), (dict(vq=None), "NULL"), (dict(vs=None), "NULL"),
    (dict(pages=None), "NULL"), (dict(lengths=None), "NULL"),
    (dict(dtype=2), "ARG"), (dict(dtype=-1), "ARG"), (dict(a=ODD), "ARG"), (dict(b=ODD), "ARG"),
    (dict(a=None), "NULL"), (dict(b=None), "NULL"),
    (dict(head=32), "SHAPE"), (dict(head=68), "SHAPE"), (dict(token=32), "SHAPE"),
    (dict(token=260), "SHAPE"), (dict(token=-256), "SHAPE"), (dict(head=-64), "SHAPE"),
    (dict(token=72, head=80), "SHAPE"), (dict(token=1 << 41), "SHAPE"), (dict(head=1 << 41), "SHAPE"),
])
def test_refusals(m, name, bad, status):
    assert call(m, name, **bad) == getattr(m, "MX_ERR_" + status)


def test_write_and_read_refusals(m):
    for rule in (-1, 2):
        assert call(m, "mx_cache_write", rule=rule) == m.MX_ERR_ARG
    for p in "ab":  # no description of the rows
        for name in NAMES[:2]:
            assert call(m, name, no_rows=p, **{p: None}) == m.MX_ERR_NULL
    for where in (0x20000000, 0x21000000, 0x22000000, 0x23000000):  # rows inside the cache
        for name in NAMES[:2]:
            assert call(m, name, a=where) == m.MX_ERR_ARG
            assert call(m, name, b=where) == m.MX_ERR_ARG
    assert call(m, "mx_cache_read", b=A) == m.MX_ERR_ARG          # k and v
    assert call(m, "mx_cache_read", b=A + 128 * 2) == m.MX_ERR_ARG  # v's rows in k's


def test_attention_refusals(m):
    bad = lambda **kw: call(m, "mx_cache_attention", **kw)  # noqa: E731
    assert bad(q_heads=5) == m.MX_ERR_SHAPE
    assert bad(q_heads=-2) == m.MX_ERR_SHAPE
    assert bad(heads=0) == m.MX_ERR_SHAPE
    assert bad(q_heads=65538) == m.MX_ERR_UNSUPPORTED
    assert bad(table_width=(1 << 31) - 1, page_size=2048, T=3000, seqs=3000) == m.MX_ERR_UNSUPPORTED
    for s in (float("nan"), float("inf"), -float("inf")):
        assert bad(scale=s) == m.MX_ERR_ARG
    assert bad(workspace=None, table_width=40) == m.MX_ERR_NULL
    assert bad(workspace=C + 8) == m.MX_ERR_ARG
    need = m.lib().mx_cache_attention_workspace(3, 4, ctypes.byref(cache_of(m, table_width=40)))
    assert need > 0 and bad(size=need - 1, table_width=40) == m.MX_ERR_ARG
    assert bad(lse=0x30000002) == m.MX_ERR_ARG
    for b in (A, A + 64 * 2, 0x20000000, 0x22000000):  # out on q, out in the cache
        assert bad(b=b) == m.MX_ERR_ARG
    for lse in (A, B, B + 16, 0x21000000):
        assert bad(lse=lse) == m.MX_ERR_ARG


def test_no_ops(m):
    for name in NAMES:
        assert call(m, name, T=0, seqs=0) == m.MX_OK
        assert call(m, name, T=0, offsets=0x26000000, lengths=None, kq=None) == m.MX_OK
        assert call(m, name, T=3, seqs=0, offsets=0x26000000) == m.MX_OK
    assert call(m, "mx_cache_write", n_pages=0, kq=None, ks=None, vq=None, vs=None) == m.MX_OK
    assert call(m, "mx_cache_attention", q_heads=0) == m.MX_OK
    assert call(m, "mx_cache_write", heads=0) == m.MX_OK


def test_workspace_sizes(m):
    size = lambda T, q, **kw: m.lib().mx_cache_attention_workspace(T, q, ctypes.byref(cache_of(m, **kw)))  # noqa: E731
    assert size(0, 4, seqs=0) == 0 and size(3, 0) == 0
    for bad in (dict(dim=32), dict(page_size=33), dict(seqs=-1)):
        assert size(3, 4, **bad) == -1
    assert size(3, 5) == -1 and size(3, -2) == -1 and size(2, 4) == -1
    # a short table: nothing is divided; a long one: every row's place, each segment's sums and statistics
    assert size(3, 4) == 0 and size(3, 4, table_width=17) == 0
    assert size(3, 4, table_width=18) >= 3 * 2 * 16 + 4 * (64 + 2)
    assert size(600, 2, seqs=600) > 0  # many workgroups
    assert m.lib().mx_cache_attention_workspace(3, 4, None) == -1


def test_binding_refuses_before_the_library():
    import mxfp4_block_scaled_hadamard32_amd as mx
    z = lambda *s, dtype=torch.uint8: torch.zeros(s, dtype=dtype)  # noqa: E731
    kq, ks, vq, vs = z(4, 2, 64, 64), z(4, 2, 2), z(4, 2, 2, 64, 32), z(4, 2, 2)
    pages, lengths = z(3, 2, dtype=torch.int32), z(3, dtype=torch.int32)
    x = z(3, 2, 64, dtype=torch.bfloat16)
    for f in (lambda *a: mx.mx_cache_write(x, x, *a), lambda *a: mx.mx_cache_read(*a),
              lambda *a: mx.mx_cache_attention(x, *a)):
        with pytest.raises((ValueError, TypeError)):  # nothing is on a GPU
            f(kq, ks, vq, vs, pages, lengths)
        with pytest.raises((ValueError, TypeError)):
            f(None, ks, vq, vs, pages, lengths)
        with pytest.raises((ValueError, TypeError)):
            f(kq[0], ks, vq, vs, pages, lengths)
    with pytest.raises(TypeError):
        mx.mx_cache_write(None, x, kq, ks, vq, vs, pages, lengths)
    with pytest.raises(TypeError):
        mx.mx_cache_attention([1], kq, ks, vq, vs, pages, lengths)
    with pytest.raises(ValueError):
        mx.mx_cache_attention(x[0], kq, ks, vq, vs, pages, lengths)
    with pytest.raises(ValueError):  # offsets without a number of rows
        mx.mx_cache_read(kq, ks, vq, vs, pages, lengths, offsets=z(4, dtype=torch.int32))


def test_outputs_on_tables(m):
    """Outputs that share a byte with the page table, the lengths or the offsets, which other workgroups
    still read; beside them and between the rows of a strided output they are not refused (without a GPU
    the launch is)."""
    tables = {"pages": (0x24000000, 3 * 2 * 4), "lengths": (0x25000000, 3 * 4), "offsets": (0x26000000, 4 * 4)}
    rows = {"mx_cache_read": 2, "mx_cache_attention": 4}
    for where, size in tables.values():
        for name, heads in rows.items():
            row = heads * 64 * 2
            for out in "ab" if name == "mx_cache_read" else "b":
                kw = dict(offsets=0x26000000)
                for at in (where, where - 3 * row + 16, where - 16 + (size + 15) // 16 * 16):
                    assert call(m, name, **{out: at}, **kw) == m.MX_ERR_ARG, (name, out, at)
                for i in range(3):
                    assert call(m, name, token=1 << 15, **{out: where - (i << 16)}, **kw) == m.MX_ERR_ARG
                for at in (where - 3 * row, where + (size + 15) // 16 * 16):
                    assert call(m, name, **{out: at}, **kw) != m.MX_ERR_ARG, (name, out, at)
                assert call(m, name, token=1 << 15, **{out: where - row - (1 << 16)}, **kw) != m.MX_ERR_ARG
        for at in (where, where - 3 * 4 * 4 + 4, where + size - 4):
            assert call(m, "mx_cache_attention", lse=at, offsets=0x26000000) == m.MX_ERR_ARG
        for at in (where - 3 * 4 * 4, where + size):
            assert call(m, "mx_cache_attention", lse=at, offsets=0x26000000) != m.MX_ERR_ARG
    # heads before tokens: the whole extent counts
    kw = dict(token=64, head=64 * 3, offsets=0x26000000)
    for where, size in tables.values():
        assert call(m, "mx_cache_read", b=where - 128, **kw) == m.MX_ERR_ARG


def test_module_refuses_what_no_call_takes():
    """A cache that every call would refuse is not allocated."""
    from mxfp4_block_scaled_hadamard32_amd.linear import MXCache
    for bad in (dict(page_size=0), dict(page_size=-32), dict(page_size=48), dict(page_size=2080), dict(dim=96),
                dict(dim=0), dict(fmt=2), dict(fmt=-1), dict(scale_rule=2), dict(scale_rule=-1)):
        kw = dict(dim=64, page_size=32)
        kw.update(bad)
        with pytest.raises(ValueError):
            MXCache(2, 1, device="cpu", **kw)
    for page in (32, 2048):
        c = MXCache(2, 3, 128, page, fmt=1, scale_rule=1, device="cpu")
        assert c.kq.shape == (2, 3, page, 128) and c.vs.shape == (2, 3, page // 32)
