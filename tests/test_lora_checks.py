"""CPU checks of mx_lora: every refusal of the C ABI (before any HIP call; no pointer here is
dereferenced) and of the binding (before the library)."""
import os

import pytest
import torch

P = {"x": 0x1000000, "a": 0x2000000, "b": 0x3000000, "index": 0x4000000, "scaling": 0x5000000,
     "base": 0x6000000, "out": 0x7000000, "workspace": 0x8000000}


@pytest.fixture(scope="module")
def m():
    from mxfp4_block_scaled_hadamard32_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("libmx.so not built (run __graft_entry__.build())")
    _lib.lib()
    return _lib


def call(m, **kw):
    v = dict(dtype=1, ldx=64, adapters=4, rank=24, base_dtype=0, ldb=100, T=3, N=100, K=64, out_dtype=1,
             ldo=100, size=1 << 30, **P)
    v.update(kw)
    return m.lib().mx_lora(*(v[k] for k in ("x", "dtype", "ldx", "a", "b", "adapters", "rank", "index",
                                            "scaling", "base", "base_dtype", "ldb", "T", "N", "K",
                                            "out_dtype", "out", "ldo", "workspace", "size")), None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), "SHAPE"), (dict(N=-1), "SHAPE"), (dict(K=-8), "SHAPE"), (dict(K=60), "SHAPE"),
    (dict(ldx=56), "SHAPE"), (dict(ldx=68), "SHAPE"), (dict(adapters=-1), "SHAPE"),
    (dict(rank=-8), "SHAPE"), (dict(rank=12), "SHAPE"), (dict(ldo=99), "SHAPE"), (dict(ldb=99), "SHAPE"),
    (dict(dtype=2), "ARG"), (dict(base_dtype=2), "ARG"), (dict(out_dtype=-1), "ARG"),
    (dict(x=P["x"] + 8), "ARG"), (dict(a=P["a"] + 8), "ARG"), (dict(b=P["b"] + 8), "ARG"),
    (dict(index=P["index"] + 2), "ARG"), (dict(scaling=P["scaling"] + 2), "ARG"),
    (dict(base=P["base"] + 2), "ARG"), (dict(out=P["out"] + 1), "ARG"),
    (dict(rank=136), "UNSUPPORTED"), (dict(T=(1 << 21) + 1), "UNSUPPORTED"),
    (dict(N=(1 << 26) + 1, ldo=1 << 27, ldb=1 << 27), "UNSUPPORTED"),
    (dict(K=(1 << 26) + 8, ldx=1 << 27), "UNSUPPORTED"), (dict(adapters=(1 << 26) + 1), "UNSUPPORTED"),
    (dict(x=None), "NULL"), (dict(a=None), "NULL"), (dict(b=None), "NULL"), (dict(index=None), "NULL"),
    (dict(out=None), "NULL"), (dict(workspace=None), "NULL"),
    (dict(workspace=P["workspace"] + 8), "ARG"), (dict(size=3 * 24 * 4 - 1), "ARG"),
    (dict(out=P["x"]), "ARG"), (dict(out=P["x"] + 3 * 128 - 2), "ARG"),       # on x
    (dict(out=P["base"]), "ARG"), (dict(out=P["base"] + 16, out_dtype=0), "ARG"),  # on base, not it
    (dict(out=P["base"], out_dtype=0, ldo=104), "ARG"),
])
def test_refusals(m, bad, status):
    assert call(m, **bad) == getattr(m, "MX_ERR_" + status)


def test_no_ops_and_sizes(m):
    assert call(m, T=0) == m.MX_OK and call(m, N=0) == m.MX_OK
    size = m.lib().mx_lora_workspace
    assert size(1, 3, 100, 64, 4, 24) == 3 * 24 * 4 and size(0, 3, 100, 64, 4, 16) == 3 * 16 * 4
    for none in ((0, 100, 64, 4, 24), (3, 0, 64, 4, 24), (3, 100, 0, 4, 24), (3, 100, 64, 0, 24),
                 (3, 100, 64, 4, 0), (-1, 100, 64, 4, 24), (3, 100, 64, 4, 136)):
        assert size(1, *none) == 0
    assert size(1, 1, 14336, 4096, 8, 64) % (64 * 4) == 0
    assert size(1, 1, 14336, 4096, 8, 16) == 0                      # one kernel
    assert size(1, 17, 14336, 4096, 8, 16) > 0 and size(1, 1, 64, 4104, 8, 16) > 0
    assert size(1, 1, 64, 4096, 8, 24) > 0 and size(1, 16, 16385, 4096, 16, 16) > 0


def test_binding_refuses_before_the_library():
    import mxfp4_block_scaled_hadamard32_amd as mx
    x = torch.zeros((3, 64), dtype=torch.bfloat16)
    a, b = torch.zeros((4, 16, 64), dtype=torch.bfloat16), torch.zeros((4, 100, 16), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        mx.mx_lora(x, a, b, i)  # not on a GPU
    with pytest.raises(TypeError):
        mx.mx_lora(None, a, b, i)


def test_out_on_weights_and_tables(m):
    """An out that shares a byte with a, b, index or scaling would be read while it is written. T, N of
    3 x 100 bf16 in rows of 200 bytes; a has 4 x 24 x 64 values, b 4 x 100 x 24."""
    bytes_of = {"a": 4 * 24 * 64 * 2, "b": 4 * 100 * 24 * 2, "index": 3 * 4, "scaling": 4 * 4}
    for name, size in bytes_of.items():
        for at in (P[name], P[name] + size - 2, P[name] - 3 * 200 + 2):
            assert call(m, out=at) == m.MX_ERR_ARG, (name, at)
        for row in range(3):  # rows of 200 bytes, 1 MiB apart
            for at in (P[name] - 198, P[name] + size - 2):
                assert call(m, out=at - (row << 20), ldo=1 << 19) == m.MX_ERR_ARG, (name, row, at)
        # beside them and between the rows: not refused (without a GPU the launch is)
        for at in (P[name] - 3 * 200, P[name] + size):
            assert call(m, out=at) != m.MX_ERR_ARG, (name, at)
        for at in (P[name] - 200, P[name] + size - (1 << 20), P[name] + size - (2 << 20)):
            assert call(m, out=at, ldo=1 << 19) != m.MX_ERR_ARG, (name, at)
    # in place is no way round it, and nothing is read without adapters
    assert call(m, out=P["b"], base=P["b"], out_dtype=0, base_dtype=0) == m.MX_ERR_ARG
    assert call(m, out=P["b"], adapters=0) != m.MX_ERR_ARG


def test_scaling_stays_fp32():
    """A module's change of type takes the weights along, not the factors, which mx_lora has in fp32."""
    from mxfp4_block_scaled_hadamard32_amd.linear import MXAdapters
    a, b = torch.randn((2, 8, 64)), torch.randn((2, 32, 8))
    s = torch.tensor([1.0 / 3.0, 1e30])
    for change in (lambda m: m.to(torch.bfloat16), lambda m: m.bfloat16(), lambda m: m.double().float(),
                   lambda m: torch.nn.Sequential(m).bfloat16()[0], lambda m: m.to("cpu", torch.bfloat16),
                   lambda m: m.half()):
        ad = MXAdapters(a, b, s)
        got = change(ad)
        assert got.scaling.dtype == torch.float32 and torch.equal(got.scaling, s)
        assert got.a.dtype == got.b.dtype
    assert MXAdapters(a, b).bfloat16().scaling is None and MXAdapters(a, b).bfloat16().a.dtype == torch.bfloat16
    meta = MXAdapters(a, b, s).to("meta")
    assert meta.scaling.device.type == "meta" and meta.a.device.type == "meta"
