"""CPU checks of the norm and few-token product entry points: every refusal of the C ABI (before
any HIP call; no pointer here is dereferenced) and of the binding (before the library)."""
import ctypes
import os

import pytest
import torch

A = ctypes.c_void_p(0x10000)   # aligned, never dereferenced
B = ctypes.c_void_p(0x20000)
ODD = ctypes.c_void_p(0x10004)


@pytest.fixture(scope="module")
def m():
    from mxfp4_block_scaled_hadamard32_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libmx.so not built (run __graft_entry__.build())")
    _lib.lib()
    return _lib


def norm_call(m, name="mx_rmsnorm", **kw):
    v = dict(x=A, ldx=64, residual=A, ldr=64, dtype=1, rows=4, cols=64, gamma=A, gdt=0, eps=1e-5,
             sum=A, lds=64, y=A, ldy=64, rstd=A, fmt=0, opts=m.mx_quant_opts(0, 0, 0, 0, 0),
             codes=A, scales=A)
    v.update(kw)
    o = ctypes.byref(v["opts"]) if v["opts"] is not None else None
    args = [v[k] for k in ("x", "ldx", "residual", "ldr", "dtype", "rows", "cols", "gamma", "gdt",
                           "eps", "sum", "lds", "y", "ldy", "rstd")]
    if name == "mx_rmsnorm_quant":
        args += [o, v["codes"], v["scales"]]
    elif name == "mx_rmsnorm_quant_mxfp8":
        args += [v["fmt"], o, v["codes"], v["scales"]]
    return getattr(m.lib(), name)(*args, None)


@pytest.mark.parametrize("name", ["mx_rmsnorm", "mx_rmsnorm_quant", "mx_rmsnorm_quant_mxfp8"])
@pytest.mark.parametrize("bad,status", [
    (dict(x=None), "NULL"), (dict(gamma=None), "NULL"),
    (dict(rows=-1), "SHAPE"), (dict(cols=-32), "SHAPE"), (dict(cols=48), "SHAPE"),
    (dict(ldx=32), "SHAPE"), (dict(ldx=68), "SHAPE"), (dict(ldr=32), "SHAPE"),
    (dict(lds=68), "SHAPE"), (dict(ldy=32), "SHAPE"),
    (dict(cols=32800, ldx=32800, ldr=32800, lds=32800, ldy=32800), "UNSUPPORTED"),
    (dict(dtype=2), "ARG"), (dict(gdt=-1), "ARG"),
    (dict(eps=-1.0), "ARG"), (dict(eps=float("nan")), "ARG"), (dict(eps=float("inf")), "ARG"),
    (dict(x=ODD), "ARG"), (dict(residual=ODD), "ARG"), (dict(sum=ODD), "ARG"),
    (dict(y=ODD), "ARG"), (dict(gamma=ODD), "ARG"), (dict(rstd=ctypes.c_void_p(0x10002)), "ARG"),
])
def test_norm_refusals(m, name, bad, status):
    assert norm_call(m, name, **bad) == getattr(m, "MX_ERR_" + status)


def test_norm_output_refusals(m):
    assert norm_call(m, y=None) == m.MX_ERR_NULL
    for name in ("mx_rmsnorm_quant", "mx_rmsnorm_quant_mxfp8"):
        assert norm_call(m, name, codes=None) == m.MX_ERR_NULL
        assert norm_call(m, name, scales=None) == m.MX_ERR_NULL
        assert norm_call(m, name, opts=None) == m.MX_ERR_NULL
        assert norm_call(m, name, codes=ODD) == m.MX_ERR_ARG
        for o in ((2, 0, 0), (0, 3, 0), (0, 0, 2)):
            assert norm_call(m, name, opts=m.mx_quant_opts(*o, 0, 0)) == m.MX_ERR_ARG
    assert norm_call(m, "mx_rmsnorm_quant", codes=ctypes.c_void_p(0x10008)) == m.MX_ERR_ARG
    assert norm_call(m, "mx_rmsnorm_quant_mxfp8", fmt=2) == m.MX_ERR_ARG
    # nothing to do: NULLs are fine, nothing is launched
    for kw in (dict(rows=0), dict(cols=0)):
        assert norm_call(m, x=None, gamma=None, y=None, residual=None, sum=None, rstd=None,
                         **kw) == m.MX_OK
    # a leading dimension that goes with no pointer is not looked at
    assert norm_call(m, rows=0, residual=None, ldr=1, sum=None, lds=1) == m.MX_OK


def ptr(address):
    return ctypes.c_void_p(address)


# x, residual, sum and y of 4 rows of 64 bf16 values, 128 bytes apart where nothing else is said
@pytest.mark.parametrize("kw", [
    dict(sum=ptr(0x20000), y=ptr(0x20000)),                                   # both on one buffer
    dict(sum=ptr(0x20000), y=ptr(0x20010)),                                   # a few bytes apart
    dict(x=ptr(0x20000), sum=ptr(0x20000), lds=128),                          # x, other rows
    dict(residual=ptr(0x20000), y=ptr(0x20000), ldy=72),                      # residual, other rows
    dict(x=ptr(0x20000), y=ptr(0x20080)),                                     # a row further
    dict(x=ptr(0x20000), y=ptr(0x1FF80)),                                     # a row before
    dict(x=ptr(0x20000), ldx=128, sum=ptr(0x20070), lds=128),                 # the gap, and a bit
    dict(x=ptr(0x20000), ldx=128, sum=ptr(0x20300), lds=72),                  # into the last row
    dict(x=ptr(0x20000), ldx=128, rows=1 << 20, sum=ptr(0x20000 + (1 << 27)), lds=64),
])
def test_norm_refuses_overlapping_outputs(m, kw):
    v = dict(x=ptr(0x1000000000), residual=ptr(0x2000000000), sum=ptr(0x3000000000),
             y=ptr(0x4000000000))
    v.update(kw)
    for name in ("mx_rmsnorm", "mx_rmsnorm_quant", "mx_rmsnorm_quant_mxfp8"):
        assert norm_call(m, name, **v) == m.MX_ERR_ARG


@pytest.mark.parametrize("kw", [
    dict(dx=ptr(0x20000), dsum=ptr(0x20000), ldds=128),
    dict(dx=ptr(0x20000), dsum=ptr(0x20010)),
    dict(dx=ptr(0x20000), dy=ptr(0x20010)),
    dict(dx=ptr(0x20000), s=ptr(0x20080)),
    dict(dx=ptr(0x20000), s=ptr(0x20000), dgamma=ptr(0x5000000000)),
    dict(dx=ptr(0x20000), dy=ptr(0x20000), lddy=72),
    dict(dx=ptr(0x20000), dy=ptr(0x1FF80), dgamma=ptr(0x5000000000)),
])
def test_backward_refuses_overlapping_outputs(m, kw):
    v = dict(rows=4, dy=ptr(0x1000000000), dsum=ptr(0x2000000000), s=ptr(0x3000000000),
             dx=ptr(0x4000000000), dgamma=None, work=None, size=0)
    v.update(kw)
    assert backward_call(m, **v) == m.MX_ERR_ARG


@pytest.mark.parametrize("kw", [
    dict(N=64, ldy=64), dict(y=ptr(0x10010)), dict(y=ptr(0x1017E)), dict(x=ptr(0x10030)),
    dict(odt=0, T=1, y=ptr(0x1007C)), dict(ldx=128, y=ptr(0x1007E), ldy=128),
])
def test_gemv_refuses_an_output_on_its_input(m, kw):
    assert gemv_call(m, **kw) == m.MX_ERR_ARG


def backward_call(m, **kw):
    v = dict(dy=A, lddy=64, dsum=B, ldds=64, s=A, lds=64, dtype=1, rows=1 << 20, cols=64, gamma=A,
             gdt=0, rstd=A, dx=B, lddx=64, dgamma=A, work=A, size=1 << 20)
    v.update(kw)
    return m.lib().mx_rmsnorm_backward(*v.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(dy=None), "NULL"), (dict(s=None), "NULL"), (dict(gamma=None), "NULL"),
    (dict(rstd=None), "NULL"), (dict(dx=None), "NULL"), (dict(work=None), "NULL"),
    (dict(rows=-1), "SHAPE"), (dict(cols=40), "SHAPE"), (dict(lddy=32), "SHAPE"),
    (dict(ldds=68), "SHAPE"), (dict(lds=32), "SHAPE"), (dict(lddx=32), "SHAPE"),
    (dict(cols=32800, lddy=32800, ldds=32800, lds=32800, lddx=32800), "UNSUPPORTED"),
    (dict(dtype=5), "ARG"), (dict(gdt=5), "ARG"), (dict(dy=ODD), "ARG"), (dict(dsum=ODD), "ARG"),
    (dict(s=ODD), "ARG"), (dict(dx=ODD), "ARG"), (dict(gamma=ODD), "ARG"), (dict(work=ODD), "ARG"),
    (dict(rstd=ctypes.c_void_p(0x10001)), "ARG"), (dict(dgamma=ctypes.c_void_p(0x10002)), "ARG"),
    (dict(size=16), "ARG"), (dict(dx=A), "ARG"),
])
def test_backward_refusals(m, bad, status):
    assert backward_call(m, **bad) == getattr(m, "MX_ERR_" + status)


def test_backward_nothing_to_do(m):
    assert backward_call(m, rows=0, dgamma=None, work=None) == m.MX_OK
    assert backward_call(m, cols=0) == m.MX_OK


def test_backward_workspace_size(m):
    f = m.lib().mx_rmsnorm_backward_workspace
    assert f(0, 64) == 0 and f(4, 0) == 0 and f(-1, 64) == 0 and f(4, 40) == 0
    assert f(4, 65536) == 0
    assert f(1, 32) == 0 and f(4096, 1024) == 0  # small tensors
    for rows, cols in ((4097, 1024), (16384, 8192), (1 << 20, 128), (129, 32768)):
        assert f(rows, cols) % (4 * cols) == 0 and 0 < f(rows, cols) <= min(rows, 1536) * 4 * cols


@pytest.mark.parametrize("rows,cols", [(4097, 32), (8192, 512), (16384, 256), (32768, 128),
                                       (131072, 32)])
def test_backward_of_tall_narrow_tensors_wants_a_workspace(m, rows, cols):
    """Without one, cols / 32 workgroups would walk over all these rows."""
    size = m.lib().mx_rmsnorm_backward_workspace(rows, cols)
    assert size > 0 and size % (4 * cols) == 0 and size <= 1536 * 4 * cols
    ld = dict(lddy=cols, ldds=cols, lds=cols, lddx=cols)
    assert backward_call(m, rows=rows, cols=cols, size=size - 1, **ld) == m.MX_ERR_ARG
    assert backward_call(m, rows=rows, cols=cols, work=None, **ld) == m.MX_ERR_NULL


def gemv_call(m, **kw):
    v = dict(x=A, dtype=1, ldx=64, wq=A, ws=A, gw=1, T=3, N=10, K=64, had=0, mask=0, alpha=0,
             odt=1, y=A, ldy=10, work=None, size=0)
    v.update(kw)
    return m.lib().mx_gemv(*v.values(), None)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), "NULL"), (dict(wq=None), "NULL"), (dict(ws=None), "NULL"),
    (dict(y=None), "NULL"),
    (dict(T=-1), "SHAPE"), (dict(N=-1), "SHAPE"), (dict(K=-32), "SHAPE"), (dict(K=48), "SHAPE"),
    (dict(ldx=32), "SHAPE"), (dict(ldx=66), "SHAPE"), (dict(ldy=9), "SHAPE"),
    (dict(gw=32), "SHAPE"), (dict(gw=2), "ARG"), (dict(gw=0), "ARG"),
    (dict(dtype=2), "ARG"), (dict(odt=2), "ARG"), (dict(had=2), "ARG"),
    (dict(alpha=-127), "ARG"), (dict(alpha=128), "ARG"),
    (dict(x=ODD), "ARG"), (dict(wq=ODD), "ARG"), (dict(y=ctypes.c_void_p(0x10001)), "ARG"),
    (dict(odt=0, y=ctypes.c_void_p(0x10002)), "ARG"),
])
def test_gemv_refusals(m, bad, status):
    assert gemv_call(m, **bad) == getattr(m, "MX_ERR_" + status)


def test_gemv_workspace(m):
    f = m.lib().mx_gemv_workspace
    big = dict(T=16, N=8192, K=28672, ldx=28672, ldy=8192)
    need = f(1, 16, 8192, 28672, 0, 1)
    assert need > 0 and need % (4 * 16 * 8192) == 0
    assert gemv_call(m, work=A, size=need - 1, **big) == m.MX_ERR_ARG
    assert gemv_call(m, work=ctypes.c_void_p(0x10008), size=need, **big) == m.MX_ERR_ARG
    for dtype in (0, 1):
        for had in (0, 1):
            assert f(dtype, 1, 8192, 28672, had, 1) == 0   # one token
            assert f(dtype, 16, 100, 512, had, 1) == 0     # a small product
            assert f(dtype, 0, 8192, 28672, had, 1) == 0


@pytest.mark.parametrize("T,N,K", [((1 << 19) + 1, 128, 4096), (1 << 20, 128, 4096),
                                   (1, (1 << 26) + 1, 32), (16, 1 << 27, 1024),
                                   ((1 << 19) + 1, 32, 0), (1 << 40, 1 << 40, 4096)])
def test_gemv_size_limits(m, T, N, K):
    """The documented limits hold whichever kernel the other sizes would choose."""
    ld = dict(T=T, N=N, K=K, ldx=K, ldy=N)
    assert gemv_call(m, **ld) == m.MX_ERR_UNSUPPORTED
    for dtype in (0, 1):
        for had in (0, 1):
            assert m.lib().mx_gemv_workspace(dtype, T, N, K, had, 1) == 0


def test_gemv_nothing_to_do(m):
    assert gemv_call(m, T=0, x=None, y=None) == m.MX_OK
    assert gemv_call(m, N=0, wq=None, ws=None, y=None) == m.MX_OK


# ------------------------------------------------------------------------------------------------
# the binding
# ------------------------------------------------------------------------------------------------
@pytest.fixture()
def mx(monkeypatch):
    import mxfp4_block_scaled_hadamard32_amd as mod

    def no_library(*a, **k):
        raise AssertionError("the library was reached before the arguments were checked")
    monkeypatch.setattr(mod, "lib", no_library)
    return mod


def test_layers_refuse_what_the_binding_refuses(mx):
    from mxfp4_block_scaled_hadamard32_amd import linear
    layer = linear.MXNormLinear(64, 32, device="cpu")
    for bad, error in ((None, TypeError), ([1.0], TypeError), (torch.zeros(2, 64).half(), TypeError),
                       (torch.tensor(1.0), ValueError), (torch.zeros(64), ValueError),
                       (torch.zeros(2, 64), ValueError), (torch.zeros(1, 2, 64), ValueError)):
        with pytest.raises(error):
            layer(bad)


def test_binding_refuses_host_tensors_and_other_types(mx):
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    g, r = torch.ones(64), torch.ones(2)
    q, s = torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 2), dtype=torch.uint8)
    for call in (lambda: mx.mx_rmsnorm(x, g), lambda: mx.mx_rmsnorm_quant(x, g),
                 lambda: mx.mx_rmsnorm_quant_mxfp8(x, g),
                 lambda: mx.mx_rmsnorm_backward(x, x, g, r), lambda: mx.mx_gemv(x, q, s)):
        with pytest.raises(ValueError):
            call()
    for bad in (x.half(), None, [1.0]):
        for call in (lambda: mx.mx_rmsnorm(bad, g), lambda: mx.mx_rmsnorm_backward(x, bad, g, r),
                     lambda: mx.mx_gemv(bad, q, s)):
            with pytest.raises(TypeError):
                call()
