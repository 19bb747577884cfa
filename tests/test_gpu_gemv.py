"""Products of a few tokens with MXFP4 weights against float64: fp32 output within
(160 + K / 128) 2^-24 sum|x w|, the documented bound: a step's 128 products, 4 instructions of 33
addends each, lose at most 133 times 2^-24 of their magnitude in the matrix core (further bf16
terms of x add 2^-8 of that), the K / 128 steps are joined by as many fp32 additions at most, and
8 waves or 14 parts by their number. bf16 output is the rounding of such a value. With the
rotation, five fp32 stages round each x' five times: 5 more half steps."""
import numpy as np
import pytest
import torch

import workloads as wl
from tests import norm_reference as ref
from tests.parity import check_gemm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def bound(K):
    return (160 + K / 128) * 2.0 ** -24


MASK = 0x2C6FE9B1


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_hadamard32_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.lib()
    return m


def weights(N, K, g=1, seed=1):
    """Any codes, scale exponents -10 .. 9."""
    rng = np.random.default_rng(seed)
    return (rng.integers(0, 256, (N, K // 2), dtype=np.uint8),
            rng.integers(117, 137, (N // g, K // 32), dtype=np.uint8))


def tokens(T, K, dtype, seed=9):
    return wl.student_t3((T, K), seed=seed).to(DT[dtype])


def expected(orc, x, wq, ws, g, hadamard=0, mask=0, alpha=0, rows=None):
    W = orc.dequantize_f64(wq, ws, wq.shape[0], 2 * wq.shape[1], g, rows)
    X = x.double().numpy()
    if hadamard:
        X = ref.hadamard_f64(X, mask)
    f = 2.0 ** alpha
    return X @ W.T * f, np.abs(X) @ np.abs(W).T * f


def up(*arrays):
    return tuple(torch.from_numpy(a).to(DEV) for a in arrays)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", [(1, 1, 32), (1, 17, 64), (2, 15, 96), (1, 100, 4096),
                                   (3, 256, 160), (15, 33, 2720), (16, 1003, 4128),
                                   (17, 64, 1024), (33, 130, 544), (37, 1003, 4128), (64, 96, 128),
                                   (65, 48, 288), (130, 80, 2048), (1, 4096, 4096),
                                   (5, 14336, 512), (16, 28672, 256), (1, 512, 28672),
                                   (40, 9000, 256), (1, 13000, 8192), (3, 6500, 1056),
                                   (9, 12900, 4128), (20, 12900, 544), (50, 12900, 1600),
                                   (1, 40, 65536), (2, 30, 65536), (16, 6401, 8224),
                                   # products that take a workspace: one and several parts of K,
                                   # a part of a chunk left over, rows and tokens past the end
                                   (2, 4099, 8224), (16, 4096, 8192), (23, 8200, 4128),
                                   (64, 4100, 8256), (33, 33000, 1056), (70, 5000, 8192),
                                   (5, 300, 16416), (20, 1003, 12320), (40, 17, 16384),
                                   (130, 5000, 12832), (2, 1, 65536), (50, 20003, 1696),
                                   (2, 40010, 1056), (20, 40010, 576), (3, 500, 2080),
                                   (2, 300, 4128), (64, 2049, 16416)])
def test_against_float64(mx, orc, T, N, K, dtype):
    x = tokens(T, K, dtype)
    wq, ws = weights(N, K)
    C, Cabs = expected(orc, x, wq, ws, 1)
    dq, ds = up(wq, ws)
    check_gemm(mx.mx_gemv(x.to(DEV), dq, ds, out_dtype=torch.float32), C, Cabs, rel=bound(K))
    check_gemm(mx.mx_gemv(x.to(DEV), dq, ds), C, Cabs, rel=bound(K))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", [(1, 40, 4096), (7, 300, 1056), (16, 5000, 256), (35, 64, 512),
                                   (64, 200, 160), (2, 14000, 96), (3, 500, 2080),
                                   (20, 20003, 1056), (40, 40010, 544),
                                   (1, 13000, 8192), (1, 100, 65536), (20, 13000, 608),
                                   (16, 4100, 8224), (40, 8200, 4128), (3, 33, 8224),
                                   (37, 500, 16416)])
def test_rotated_weights(mx, orc, T, N, K, dtype):
    """Weights as mx_quantize makes them with the signed transform; fp32's five stages on x."""
    w = wl.normal((N, K), 0.02, seed=4).to(torch.bfloat16)
    dq, ds = mx.mx_quantize(w.to(DEV), hadamard=1, sign_mask=MASK, scale_rule=1)
    x = tokens(T, K, dtype)
    C, Cabs = expected(orc, x, dq.cpu().numpy(), ds.cpu().numpy(), 1, 1, MASK, -5)
    # a stage's rounding is relative to its own value, at most the block's sum of |x|: count the
    # five half steps on sum |x| per block times |w|
    W = np.abs(orc.dequantize_f64(dq.cpu().numpy(), ds.cpu().numpy(), N, K, 1))
    A = np.abs(x.double().numpy()).reshape(T, K // 32, 32).sum(2).repeat(32, axis=1) @ W.T / 32
    y = mx.mx_gemv(x.to(DEV), dq, ds, hadamard=1, sign_mask=MASK, alpha_exp=-5,
                   out_dtype=torch.float32)
    check_gemm(y, C, bound(K) * Cabs + 5 * 2.0 ** -24 * A, rel=1.0)
    # bf16 y of bf16 x: 16 bits of each rotated value, half a step is 2^-17
    y16 = mx.mx_gemv(x.to(DEV), dq, ds, hadamard=1, sign_mask=MASK, alpha_exp=-5)
    check_gemm(y16, C, (bound(K) + 2.0 ** -17) * Cabs + 5 * 2.0 ** -24 * A, rel=1.0)
    # the same product as the unrotated layer, up to the quantization of the weights
    plain = x.double() @ w.double().t()
    rel = float((y.double().cpu() - plain).norm() / plain.norm())
    assert rel < 0.25, rel


def some(N, n=48):
    """The first, some middle and the last of N outputs."""
    return np.unique(np.r_[0:min(n, N), N // 2:min(N // 2 + n, N), max(N - n, 0):N])


def check_outputs(orc, y, x, wq, ws, had):
    """y against float64, within the documented bound; wq, ws the rows of y's columns."""
    T, K = x.shape
    C, Cabs = expected(orc, x, wq, ws, 1, had, MASK, -5 * had)
    b = bound(K) * Cabs
    if had:
        if x.dtype == torch.bfloat16 and y.dtype == torch.bfloat16:
            b = b + 2.0 ** -17 * Cabs  # 16 bits of each rotated value
        W = np.abs(orc.dequantize_f64(wq, ws, wq.shape[0], K, 1))  # five fp32 stages, as above
        A = np.abs(x.double().numpy()).reshape(T, K // 32, 32).sum(2).repeat(32, axis=1) @ W.T / 32
        b = b + 5 * 2.0 ** -24 * A
    check_gemm(y, C, b, rel=1.0)


# sizes that between them take each shape of the kernels for rotated tokens, with the number of parts
# of K for two bf16 terms (bf16 tokens and outputs) and for three: the choice is an estimate's, and
# a test that no longer reaches its kernel has to say so
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"),
                                       ("f32", "bf16")])
@pytest.mark.parametrize("T,N,K,parts2,parts3", [
    (38, 24992, 832, 1, 1), (23, 16416, 11232, 3, 1), (30, 2551, 20032, 12, 6),
    (3, 12495, 6784, 5, 5), (16, 28672, 8192, 2, 2), (40, 8200, 8224, 2, 2),
    (64, 2049, 16416, 7, 7), (2, 500, 2080, 0, 0), (1, 7000, 2080, 0, 0), (1, 9700, 1056, 0, 0),
    (1, 17000, 1056, 0, 0), (1, 5000, 28672, 0, 0), (1, 300, 28672, 0, 0)])
def test_every_shape_for_rotated_tokens(mx, orc, T, N, K, parts2, parts3, dtype, out):
    parts = parts2 if (dtype, out) == ("bf16", "bf16") else parts3
    size = mx.lib().mx_gemv_workspace(int(dtype == "bf16"), T, N, K, 1, int(out == "bf16"))
    assert size == (4 * T * N * parts if parts > 1 else 0)
    gen = torch.Generator(device=DEV).manual_seed(T)
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=gen)
    s = torch.randint(117, 137, (N, K // 32), dtype=torch.uint8, device=DEV, generator=gen)
    x = tokens(T, K, dtype)
    y = mx.mx_gemv(x.to(DEV), q, s, hadamard=1, sign_mask=MASK, alpha_exp=-5, out_dtype=DT[out])
    p = torch.from_numpy(some(N, 130)).to(DEV)
    check_outputs(orc, y[:, p], x, q[p].cpu().numpy(), s[p].cpu().numpy(), 1)


# one-token, direct and shared kernels, whole chunks and blocks left over, one part of K and several
KERNELS = [(1, 40, 4128), (1, 9300, 1056), (2, 500, 2080), (6, 40, 1184), (16, 5000, 256),
           (20, 1003, 12320), (16, 4096, 8192), (50, 12900, 1600), (64, 4100, 8256),
           (9, 12900, 4128)]


@pytest.mark.parametrize("had", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", KERNELS)
def test_special_values_in_every_kernel(mx, orc, T, N, K, dtype, had):
    """Infinities and NaNs of a token in its first and last block stay in that token, NaN scales in
    their outputs, zeros give zeros, and the tokens beside them their products."""
    wq, ws = weights(N, K)
    wq[wq & 7 == 0] |= 1  # no zero weights: infinity times zero is a NaN
    wq[wq & 0x70 == 0] |= 0x10
    bad = [5, N - 2]
    ws[5, 0] = ws[N - 2, K // 32 - 1] = 255
    q, s = up(wq, ws)
    cols = some(N)
    W = orc.dequantize_f64(wq[cols], ws[cols], len(cols), K, 1)
    fine = ~np.isin(cols, bad)
    kinds = ["zero", "inf", "-inf", "nan", "late nan", "plain"]
    for shift in range(0, len(kinds), T):
        kind = [kinds[(shift + t) % len(kinds)] for t in range(T)]
        x = tokens(T, K, dtype, seed=shift + 1)
        for t, k in enumerate(kind):
            if k == "zero":
                x[t] = 0.0
            elif k != "plain":
                at = {"inf": 3, "-inf": K - 1, "nan": 20, "late nan": K - 2}[k]
                x[t, at] = float(k.split()[-1])
        for out in (torch.float32, torch.bfloat16):
            y = mx.mx_gemv(x.to(DEV), q, s, hadamard=had, sign_mask=MASK, alpha_exp=-5 * had,
                           out_dtype=out)[:, torch.from_numpy(cols).to(DEV)]
            v = y.double().cpu().numpy()
            assert np.isnan(v[:, ~fine]).all()
            for t, k in enumerate(kind):
                row = v[t, fine]
                if k == "zero":
                    assert (row == 0).all()
                elif k.endswith("nan"):
                    assert np.isnan(row).all()
                elif k.endswith("inf"):
                    if had:
                        assert not np.isfinite(row).any()
                    else:
                        at, sign = (3, 1.0) if k == "inf" else (K - 1, -1.0)
                        assert (row == sign * np.sign(W[fine, at]) * np.inf).all()
            plain = [t for t, k in enumerate(kind) if k == "plain"]
            if plain:
                f = torch.from_numpy(fine)
                check_outputs(orc, y.cpu()[plain][:, f], x[plain], wq[cols[fine]], ws[cols[fine]],
                              had)


@pytest.mark.parametrize("had", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,N,K", KERNELS)
def test_scales_at_the_ends_of_their_range(mx, orc, T, N, K, dtype, had):
    """Bytes 0 (2^-127, bf16 subnormals) to 2 and 250 to 252 in every block, against tokens that
    bring the products into range; 253 and 254 with weights that bf16 holds, and with ones beyond."""
    rng = np.random.default_rng(3)
    wq, _ = weights(N, K)
    cols = some(N)
    p = torch.from_numpy(cols).to(DEV)
    for low, power in ((0, 60), (250, -60)):
        ws = rng.integers(low, low + 3, (N, K // 32), dtype=np.uint8)
        x = tokens(T, K, dtype)
        x = (x.double() * 2.0 ** power).to(x.dtype)
        x[x == 0] = 2.0 ** power
        fine = np.ones(len(cols), dtype=bool)
        if low:
            wq[3] &= 0xDD           # magnitudes 0, 1/2, 2, 3: 3 x 2^126 is below 2^128
            wq[N - 3] &= 0xBB       # magnitudes 0, 1/2, 1, 3/2
            ws[3], ws[N - 3] = 253, 254
            wq[6], ws[6] = 0x11, 250
            wq[6, K // 2 - 1] = 0x17  # one weight of 6 x 2^126 in the last block
            ws[6, K // 32 - 1] = 253
            fine[cols == 6] = False
        q, s = up(wq, ws)
        for out in (torch.float32, torch.bfloat16):
            y = mx.mx_gemv(x.to(DEV), q, s, hadamard=had, sign_mask=MASK, alpha_exp=-5 * had,
                           out_dtype=out)[:, p]
            check_outputs(orc, y[:, torch.from_numpy(fine).to(DEV)], x, wq[cols[fine]],
                          ws[cols[fine]], had)
            if low:
                over = y[:, torch.from_numpy(~fine).to(DEV)]
                assert not torch.isfinite(over).any()
                if dtype == "bf16" and not had:
                    assert (over[:, 0].cpu().float()
                            == torch.sign(x[:, K - 2].float()) * float("inf")).all()


@pytest.mark.parametrize("g", [32, 64])
@pytest.mark.parametrize("T,N,K", [(1, 192, 256), (20, 4096, 320), (20, 8192, 4096),
                                   (1, 6464, 4640), (1, 9664, 320), (1, 16448, 544),
                                   (9, 12864, 320), (3, 6464, 96), (4, 320, 12832)])
def test_tile_scales(mx, orc, g, T, N, K):
    x = tokens(T, K, "bf16")
    wq, ws = weights(N, K, g)
    C, Cabs = expected(orc, x, wq, ws, g)
    dq, ds = up(wq, ws)
    check_gemm(mx.mx_gemv(x.to(DEV), dq, ds, g, out_dtype=torch.float32), C, Cabs, rel=bound(K))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_workspace(mx, orc, dtype):
    """A given workspace (its end untouched), one of another call's leavings, and none at all."""
    T, N, K = 20, 4100, 8256
    x = tokens(T, K, dtype).to(DEV)
    wq, ws = weights(N, K)
    q, s = up(wq, ws)
    size = mx.lib().mx_gemv_workspace(1 if dtype == "bf16" else 0, T, N, K, 0, 0)
    assert size > 0 and size % (4 * T * N) == 0
    y = mx.mx_gemv(x, q, s, out_dtype=torch.float32)
    work = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    for _ in range(2):
        assert torch.equal(mx.mx_gemv(x, q, s, out_dtype=torch.float32, workspace=work[:size]), y)
    assert (work[size:] == 0xFF).all()
    with pytest.raises(mx.MxError):
        mx.mx_gemv(x, q, s, out_dtype=torch.float32, workspace=work[:size - 16])
    # the C entry without one
    out = torch.empty((T, N), device=DEV)
    mx._launch("mx_gemv", x.device, None, x.data_ptr(), 1 if dtype == "bf16" else 0, K,
               q.data_ptr(), s.data_ptr(), 1, T, N, K, 0, 0, 0, 0, out.data_ptr(), N, None, 0)
    C, Cabs = expected(orc, x.cpu(), wq, ws, 1)
    check_gemm(out, C, Cabs, rel=bound(K))
    check_gemm(y, C, Cabs, rel=bound(K))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    z = mx.mx_gemv(x, q, s, out_dtype=torch.float32, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(z, y)


def test_a_workspace_that_is_none(mx):
    """The binding's errors for workspaces of another kind, type, shape or device."""
    x = torch.ones((4, 64), dtype=torch.bfloat16, device=DEV)
    q, s = up(*weights(32, 64))
    g, r = torch.ones(64, device=DEV), torch.ones(4, device=DEV)
    for bad, error in ((b"0" * 64, TypeError), (64, TypeError),
                       (torch.zeros(64, device=DEV), TypeError),
                       (torch.zeros((8, 8), dtype=torch.uint8, device=DEV), ValueError),
                       (torch.zeros(64, dtype=torch.uint8), ValueError),
                       (torch.zeros(64, dtype=torch.uint8, device=DEV)[::2], ValueError)):
        with pytest.raises(error):
            mx.mx_gemv(x, q, s, workspace=bad)
        with pytest.raises(error):
            mx.mx_rmsnorm_backward(x, x, g, r, workspace=bad)


@pytest.mark.parametrize("g", [1, 32, 64])
@pytest.mark.parametrize("dtype,had", [("bf16", 0), ("bf16", 1), ("f32", 0), ("f32", 1)])
@pytest.mark.parametrize("N,K", [(320, 2080),       # few workgroups
                                 (9280, 1056),      # many, short rows
                                 (12352, 28672),    # two or fewer in a compute unit's LDS
                                 (4288, 40032)])    # a single one, K in several segments
def test_shapes_for_one_token(mx, orc, N, K, dtype, had, g):
    x = tokens(1, K, dtype)
    gen = torch.Generator(device=DEV).manual_seed(N)
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV, generator=gen)
    s = torch.randint(117, 137, (N // g, K // 32), dtype=torch.uint8, device=DEV, generator=gen)
    cols = some(N)
    p = torch.from_numpy(cols).to(DEV)
    wq, ws = q[p].cpu().numpy(), s[p // g].cpu().numpy()
    for out in (torch.float32, torch.bfloat16):
        y = mx.mx_gemv(x.to(DEV), q, s, g, hadamard=had, sign_mask=MASK, alpha_exp=-5 * had,
                       out_dtype=out)
        check_outputs(orc, y[:, p], x, wq, ws, had)


@pytest.mark.parametrize("T", [1, 18, 50])
def test_leading_dimensions(mx, orc, T):
    K, N = 288, 77
    x = tokens(T, K, "bf16")
    wq, ws = weights(N, K)
    dq, ds = up(wq, ws)
    wide = torch.full((T, K + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, :K] = x.to(DEV)
    out = torch.full((T + 2, N + 3), 7.0, dtype=torch.float32, device=DEV)
    y = mx.mx_gemv(wide[:, :K], dq, ds, alpha_exp=3, out=out[1:T + 1, :N])
    C, Cabs = expected(orc, x, wq, ws, 1, alpha=3)
    check_gemm(y, C, Cabs, rel=bound(K))
    assert (out[0] == 7).all() and (out[T + 1] == 7).all() and (out[:, N:] == 7).all()
    if T > 1:
        again = mx.mx_gemv(x.to(DEV), dq, ds, alpha_exp=3, out_dtype=torch.float32)
        assert torch.equal(again, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_special_values(mx, dtype):
    """An infinity or NaN in x stays in its token; a NaN scale in its output; zeros give zeros."""
    T, N, K = 6, 40, 160
    wq, ws = weights(N, K)
    wq[wq & 7 == 0] |= 1  # no zero weights: infinity times zero is a NaN
    wq[wq & 0x70 == 0] |= 0x10
    ws[7, 3] = 255
    x = tokens(T, K, dtype)
    x[0] = 0.0
    x[1, 40] = float("inf")
    x[2, 99] = float("nan")
    x[3] = (x[3].float() * 1e30).to(x.dtype)
    x[4] = (x[4].float() * 1e-36).to(x.dtype)
    y = mx.mx_gemv(x.to(DEV), *up(wq, ws), out_dtype=torch.float32).cpu()
    keep = [n for n in range(N) if n != 7]
    assert torch.isnan(y[:, 7]).all()
    assert (y[0, keep] == 0).all()
    assert torch.isinf(y[1, keep]).all()
    assert torch.isnan(y[2]).all()
    assert torch.isfinite(y[3:, keep]).all() and (y[3:, keep] != 0).all()


def test_empty(mx):
    q, s = up(*weights(32, 64))
    x = torch.ones((3, 64), dtype=torch.bfloat16, device=DEV)
    assert mx.mx_gemv(x[:0], q, s).shape == (0, 32)
    assert mx.mx_gemv(x, q[:0], s[:0]).shape == (3, 0)
    out = torch.full((3, 40), 7.0, device=DEV)
    mx.mx_gemv(x[:, :0], q[:, :0].contiguous(), s[:, :0].contiguous(), out=out[:, :32])
    assert (out[:, :32] == 0).all() and (out[:, 32:] == 7).all()


def test_offsets_past_32_bits(mx, orc):
    """Codes of 4.3 GB: the rows at the end against float64; outputs 2^31 elements apart."""
    N, K = (1 << 20) + 7, 8192
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.randint(117, 137, (N, K // 32), dtype=torch.uint8, device=DEV)
    x = tokens(2, K, "bf16")
    buf = torch.empty((1 << 31) + N, dtype=torch.bfloat16, device=DEV)
    out = buf.as_strided((2, N), (1 << 31, 1))
    y = mx.mx_gemv(x.to(DEV), q, s, out=out)
    pick = np.r_[0:64, N // 2:N // 2 + 64, N - 64:N]
    p = torch.from_numpy(pick).to(DEV)
    C, Cabs = expected(orc, x, q[p].cpu().numpy(), s[p].cpu().numpy(), 1)
    check_gemm(y[:, p], C, Cabs, rel=bound(K))


@pytest.mark.parametrize("T,N,K,dtype", [(1 << 19, 17, 64, "bf16"), (1 << 19, 1, 544, "f32"),
                                         (1, 1 << 26, 32, "bf16"), (2, 1 << 26, 64, "bf16")])
def test_the_largest_counts(mx, orc, T, N, K, dtype):
    """As many tokens and rows as the entry takes: the first and last ones against float64."""
    x = torch.randn((T, K), device=DEV).to(DT[dtype])
    q = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=DEV)
    s = torch.randint(117, 137, (N, K // 32), dtype=torch.uint8, device=DEV)
    y = mx.mx_gemv(x, q, s, out_dtype=torch.float32)
    rows, cols = (torch.from_numpy(np.unique(np.r_[0:min(n, 40), max(n - 40, 0):n])).to(DEV)
                  for n in (T, N))
    C, Cabs = expected(orc, x[rows].cpu(), q[cols].cpu().numpy(), s[cols].cpu().numpy(), 1)
    check_gemm(y[rows][:, cols], C, Cabs, rel=bound(K))


def test_streams_and_graph_replays(mx):
    """Three captured products (two of them with workspaces) on streams of their own replayed at once, beside eager calls."""
    K, N = 8192, 4112
    q, s = up(*weights(N, K))
    xs = [torch.zeros((t, K), dtype=torch.bfloat16, device=DEV) for t in (1, 20, 17)]
    for x in xs:
        mx.mx_gemv(x, q, s)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(mx.mx_gemv(x, q, s))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in xs]
    for seed in (1, 2, 3):
        for x in xs:
            x.copy_(tokens(x.shape[0], K, "bf16", seed))
        eager = [mx.mx_gemv(x, q, s) for x in xs]
        torch.cuda.synchronize()
        for o in outs:
            o.fill_(1)
        torch.cuda.synchronize()
        for st, g in zip(streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, outs):
            assert torch.equal(a, b)
