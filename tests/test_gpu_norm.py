"""RMS norm with the residual's addition and block-scaled outputs, and its backward pass.

Forward: y, the sum and rstd against the float64 definition, rounded once (the kernel works in 64
bits, so a value may differ only where the definition itself lies within 2^-40 of a rounding
border); codes and scales bit for bit the oracle's quantization of the unrounded y. Backward:
against the formula in float64 within the count of fp32's roundings, and against differences of
the forward pass."""
import numpy as np
import pytest
import torch

import workloads as wl
from tests import norm_reference as ref
from tests.parity import assert_bytes_equal, bf16_round_f64, host

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
MASK = 0x2C6FE9B1

# every threads-per-row layout, one value beside its border, single rows and odd counts
SHAPES = [(1, 32), (3, 96), (37, 128), (5, 160), (9, 512), (2, 544), (6, 1024), (7, 1056),
          (3, 2048), (5, 2080), (7, 2720), (4, 4096), (2, 4128), (5, 8192), (3, 8224), (2, 16384),
          (3, 16416), (1, 32768), (300, 64)]


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_hadamard32_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.lib()
    return m


def make(rows, cols, dtype, residual, gamma_dtype="f32", seed=5):
    x = wl.student_t3((rows, cols), seed=seed).to(DT[dtype])
    r = wl.normal((rows, cols), 3.0, seed=seed + 1).to(DT[dtype]) if residual else None
    g = (1.0 + wl.normal((1, cols), 0.2, seed=seed + 2)[0]).to(DT[gamma_dtype])
    return x, r, g


def dev(t):
    return None if t is None else t.to(DEV)


def check_rounded(got: torch.Tensor, exact: np.ndarray, slack=2.0 ** -40):
    """got is exact rounded once, exact known to a relative slack."""
    lo, hi = exact - np.abs(exact) * slack, exact + np.abs(exact) * slack
    if got.dtype == torch.bfloat16:
        lo, hi = bf16_round_f64(lo), bf16_round_f64(hi)
    else:
        with np.errstate(over="ignore"):
            lo, hi = lo.astype(np.float32), hi.astype(np.float32)
    v = got.detach().float().cpu().numpy()
    same_nan = np.isnan(v) == np.isnan(exact)
    assert same_nan.all(), np.argwhere(~same_nan)[:4].tolist()
    bad = ~(np.isnan(v) | ((v >= lo) & (v <= hi)))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())


def oracle_codes(orc, fmt, y, hadamard, mask, **kw):
    if hadamard:
        y = ref.hadamard_f64(y, mask)
    w = ref.odd_f32(y)
    if fmt == "fp4":
        return orc.quantize(w, **kw)
    return orc.quantize_fp8(w, fmt=0 if fmt == "e4m3" else 1, **kw)


def quant(mx, fmt, *a, **kw):
    if fmt == "fp4":
        return mx.mx_rmsnorm_quant(*a, **kw)
    return mx.mx_rmsnorm_quant_mxfp8(*a, fmt=0 if fmt == "e4m3" else 1, **kw)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm_against_the_definition(mx, rows, cols, dtype, residual):
    x, r, g = make(rows, cols, dtype, residual, "bf16" if cols % 64 else "f32")
    y, s, rstd = mx.mx_rmsnorm(dev(x), dev(g), dev(r), eps=EPS)
    torch.cuda.synchronize()
    want = ref.stored_sum(x, r)
    assert torch.equal(s.cpu(), want)
    exact, rho = ref.norm_f64(want, g, EPS)
    check_rounded(y, exact)
    check_rounded(rstd, rho)


@pytest.mark.parametrize("rows,cols", [(5, 96), (37, 128), (7, 1056), (3, 2048), (7, 2720),
                                       (5, 8192), (2, 16384), (3, 16416)])
@pytest.mark.parametrize("fmt", ["fp4", "e4m3", "e5m2"])
@pytest.mark.parametrize("rule,rnd,had", [(0, 0, 0), (1, 0, 1), (0, 1, 0), (1, 1, 1)])
def test_codes_are_the_oracles(mx, orc, rows, cols, fmt, rule, rnd, had):
    dtype, residual = ("bf16", True) if cols % 64 == 0 else ("f32", rnd == 0)
    x, r, g = make(rows, cols, dtype, residual)
    kw = dict(scale_rule=rule, hadamard=had, sign_mask=MASK if had else 0, seed=77)
    c, sc, y, s, rstd = quant(mx, fmt, dev(x), dev(g), dev(r), eps=EPS, round=rnd, with_y=True,
                              **kw)
    torch.cuda.synchronize()
    exact, rho = ref.norm_f64(ref.stored_sum(x, r), g, EPS)
    check_rounded(y, exact)
    check_rounded(rstd, rho)
    rc, rs = oracle_codes(orc, fmt, exact, had, MASK, scale_rule=rule, round_mode=rnd, seed=77)
    assert_bytes_equal(sc, rs, "scales")
    assert_bytes_equal(c, rc, "codes")
    # without y the codes are the same
    c2, sc2, y2, _, _ = quant(mx, fmt, dev(x), dev(g), dev(r), eps=EPS, round=rnd, **kw)
    assert y2 is None and torch.equal(c2, c) and torch.equal(sc2, sc)


@pytest.mark.parametrize("cols", [128, 1024, 4096, 8192, 16384])
def test_a_row_does_not_depend_on_its_batch(mx, cols):
    """One row alone (few threads' worth of rows) and the same row among many."""
    x, r, g = make(700, cols, "bf16", True)
    x, r, g = dev(x), dev(r), dev(g)
    c, sc, y, s, rstd = mx.mx_rmsnorm_quant_mxfp8(x, g, r, with_y=True)
    for i in (0, 17, 699):
        c1, sc1, y1, s1, r1 = mx.mx_rmsnorm_quant_mxfp8(x[i:i + 1], g, r[i:i + 1], with_y=True)
        for a, b in ((c, c1), (sc, sc1), (y, y1), (s, s1), (rstd, r1)):
            assert torch.equal(a[i:i + 1], b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(6, 96), (5, 4128)])
def test_leading_dimensions_and_aliasing(mx, rows, cols, dtype):
    x, r, g = (dev(t) for t in make(rows, cols, dtype, True))
    y0, s0, r0 = mx.mx_rmsnorm(x, g, r)
    pad = 24
    wide = [torch.full((rows, cols + pad), 7.0, dtype=x.dtype, device=DEV) for _ in range(4)]
    wx, wr, ws, wy = (w[:, :cols] for w in wide)
    wx.copy_(x)
    wr.copy_(r)
    y, s, _ = mx.mx_rmsnorm(wx, g, wr, sum=ws, y=wy)
    assert y is wy and s is ws and torch.equal(wy, y0) and torch.equal(ws, s0)
    for w in wide:
        assert (w[:, cols:] == 7.0).all()
    # the sum over the residual, y over x
    y, s, rs = mx.mx_rmsnorm(wx, g, wr, sum=wr, y=wx)
    assert torch.equal(wx, y0) and torch.equal(wr, s0) and torch.equal(rs, r0)
    # the sum over x
    wx.copy_(x)
    wr.copy_(r)
    y, s, _ = mx.mx_rmsnorm(wx, g, wr, sum=wx)
    assert torch.equal(wx, s0) and torch.equal(y, y0) and torch.equal(wr, r)


@pytest.mark.parametrize("rows,cols", [(1, 64), (6, 96), (5, 4128)])
def test_rows_that_lie_between_one_another(mx, rows, cols):
    """x, residual, sum and y as the quarters of one buffer's rows, as rows taken in turn, and with
    leading dimensions that differ; outputs that overlap are refused and left alone."""
    x, r, g = (dev(t) for t in make(rows, cols, "bf16", True))
    y0, s0, r0 = mx.mx_rmsnorm(x, g, r)
    buf = torch.zeros((rows, 4 * cols), dtype=x.dtype, device=DEV)
    turns = torch.zeros((rows, 4, cols), dtype=x.dtype, device=DEV)
    for wx, wr, ws, wy in ((buf[:, i * cols:(i + 1) * cols] for i in range(4)),
                           (turns[:, i] for i in range(4))):
        wx.copy_(x)
        wr.copy_(r)
        mx.mx_rmsnorm(wx, g, wr, sum=ws, y=wy)
        assert torch.equal(wx, x) and torch.equal(wr, r)
        assert torch.equal(ws, s0) and torch.equal(wy, y0)
        dx, _ = mx.mx_rmsnorm_backward(wr, ws, g, r0, dsum=wx)
        mx.mx_rmsnorm_backward(wr, ws, g, r0, dsum=wx, dx=wy)
        assert torch.equal(wy, dx)
    # y's short rows inside one long row of x's buffer, between the ends of x's rows
    flat = torch.zeros(8 * rows * cols, dtype=x.dtype, device=DEV)
    wx = flat.as_strided((rows, cols), (4 * cols, 1))
    wx.copy_(x)
    wy = flat.as_strided((min(rows, 2), cols), (cols, 1), cols)
    mx.mx_rmsnorm(wx[:min(rows, 2)], g, r[:min(rows, 2)], y=wy)
    assert torch.equal(wy, y0[:2])
    before = flat.clone()
    with pytest.raises(mx.MxError):
        mx.mx_rmsnorm(wx, g, r, y=flat[16:].as_strided((rows, cols), (4 * cols, 1), 16))
    with pytest.raises(mx.MxError):
        mx.mx_rmsnorm(wx, g, r, sum=wy if rows == 1 else flat[:rows * cols].view(rows, cols), y=wy
                      if rows == 1 else None)
    torch.cuda.synchronize()
    assert torch.equal(flat, before)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_special_rows(mx, orc, dtype):
    """Zero, huge, tiny, infinite and NaN rows; the others are as they are alone."""
    x, _, g = make(8, 256, dtype, False)
    x[0] = 0.0
    x[1] = (x[1].float() * 1e30).to(x.dtype)   # squares past fp32
    x[2] = (x[2].float() * 1e-30).to(x.dtype)  # squares below fp32
    x[3, 5] = float("inf")
    x[4, 200] = float("nan")
    for fmt in ("fp4", "e4m3", "e5m2"):
        c, sc, y, s, rstd = quant(mx, fmt, dev(x), dev(g), eps=EPS, with_y=True)
        torch.cuda.synchronize()
        exact, rho = ref.norm_f64(x, g, EPS)
        check_rounded(y, exact)
        check_rounded(rstd, rho)
        rc, rs = oracle_codes(orc, fmt, exact, 0, 0)
        assert_bytes_equal(sc, rs, "scales")
        assert_bytes_equal(c, rc, "codes")
    assert (host(sc)[0] == 0).all() and (host(sc)[4] == 0xFF).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_rows_and_weights(mx, orc, dtype):
    """y past the types' ranges is infinite (fp32 and bf16 apart from one another), rows near the
    largest and, with eps = 0, the smallest numbers are normalised like others."""
    x, _, g = make(8, 256, dtype, False)
    x = x.clamp(-20.0, 20.0)
    g[3], g[40], g[100] = 3.0e38, -3.0e38, 3.0e-38
    x[1] = (x[1].float() * 1e37).to(x.dtype)
    x[2] = (x[2].float() * 1e-37).to(x.dtype)  # subnormals among them
    x[3] = (x[3].float() * 1e-30).to(x.dtype)
    for eps in (0.0, EPS):
        for fmt in ("fp4", "e4m3", "e5m2"):
            c, sc, y, s, rstd = quant(mx, fmt, dev(x), dev(g), eps=eps, with_y=True)
            torch.cuda.synchronize()
            exact, rho = ref.norm_f64(x, g, eps)
            rho32 = rho.astype(np.float32)
            assert np.allclose(rstd.cpu().numpy(), rho32, rtol=2.0 ** -23, atol=2.0 ** -149)
            # weights below fp32's normal range leave errors that fp32 cannot hold
            big = np.abs(exact) > 2.0 ** -100
            check_rounded(torch.where(torch.from_numpy(big), y.cpu(), torch.zeros_like(y.cpu())),
                          np.where(big, exact, 0.0))
            assert torch.isinf(y[:, 3][y[:, 3].abs() > 3.4e38]).all()
            rc, rs = oracle_codes(orc, fmt, exact, 0, 0)
            assert_bytes_equal(sc, rs, "scales")
            blocks = [b for b in range(8) if b != 3]  # block 3 holds the tiny weight
            width = c.shape[1] // 8
            got, want = host(c).reshape(8, 8, width), rc.reshape(8, 8, width)
            assert np.array_equal(got[:, blocks], want[:, blocks])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_beside_the_borders_of_the_next_rounding(mx, orc, dtype):
    """x = +-1 and eps = 0 make rho exactly 1, so y = +-gamma: weights on a tie of E2M1, E4M3,
    E5M2 and bf16, one fp32 step beside it, and block maxima on and beside a power of two; then
    the same weights with a rho that is no power of two, where y is a step's fraction beside."""
    half = torch.tensor([1.25, 1.75, 2.5, 3.5, 5.0, 0.75, 1.0625, 1.1875, 1.125, 1.375, 1.0 + 2**-8,
                         1.0 + 3 * 2**-8, 0.0625, 6.0, 448.0, 464.0])
    bits = half.view(torch.int32)
    g = torch.cat([(bits + d).view(torch.float32) for d in (-1, 0, 1, 2)])  # 64 weights
    top = torch.full((64,), 1.0).view(torch.int32).repeat(3, 1)
    top = (top + torch.tensor([[-1], [0], [1]], dtype=torch.int32)).view(torch.float32)
    g = torch.cat([g, torch.cat([t * torch.linspace(0.1, 1.0, 64) for t in top])])
    cols = g.numel()
    x = torch.ones((4, cols))
    x[1, ::3] = -1.0
    x[2] *= 3.0
    x[3] *= 0.7
    x = x.to(DT[dtype])
    for fmt in ("fp4", "e4m3", "e5m2"):
        for rule in (0, 1):
            for rnd in (0, 1):
                c, sc, y, s, rstd = quant(mx, fmt, dev(x), dev(g), eps=0.0, with_y=True,
                                          scale_rule=rule, round=rnd, seed=5)
                torch.cuda.synchronize()
                assert float(rstd[0]) == 1.0
                exact, rho = ref.norm_f64(x, g, 0.0)
                exact[:2] = x[:2].double().numpy() * g.double().numpy()
                check_rounded(y, exact)
                rc, rs = oracle_codes(orc, fmt, exact[:2], 0, 0, scale_rule=rule, round_mode=rnd,
                                      seed=5)
                assert_bytes_equal(sc[:2], rs, "scales")
                assert_bytes_equal(c[:2], rc, "codes")


def test_empty(mx):
    g = torch.ones(64, device=DEV)
    y, s, rstd = mx.mx_rmsnorm(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV), g)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    dx, dg = mx.mx_rmsnorm_backward(y, s, g, rstd)
    assert dx.shape == (0, 64) and (dg == 0).all()


def test_offsets_past_32_bits(mx):
    """Rows 2^30 + 64 elements apart, and codes past 2^31 bytes in 2^26 + 5 short rows (more
    workgroups than one launch has); the rows at the end are as they are alone."""
    ld = (1 << 30) + 64
    buf = torch.empty(3 * ld, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((3, 4096), (ld, 1))
    src, _, g = make(3, 4096, "bf16", False)
    x.copy_(src)
    g = dev(g)
    y, _, _ = mx.mx_rmsnorm(x, g, y=x)
    assert y is x
    y0, s0, r0 = mx.mx_rmsnorm(dev(src), g)
    assert torch.equal(x, y0)
    dx0, dg0 = mx.mx_rmsnorm_backward(y0, s0, g, r0)
    _, dg = mx.mx_rmsnorm_backward(x, s0, g, r0)
    dx, _ = mx.mx_rmsnorm_backward(x, s0, g, r0, dx=x, with_dgamma=False)
    assert torch.equal(x, dx0) and torch.equal(dg, dg0)
    del buf, x, y, dx
    rows = (1 << 26) + 5
    x = torch.empty((rows, 32), dtype=torch.bfloat16, device=DEV)
    tail, _, g = make(4096, 32, "bf16", False)
    x[:4096] = tail.to(DEV)
    x[4096:rows - 4096] = 1.0
    x[rows - 4096:] = tail.to(DEV)
    g = dev(g)
    c, sc, y, s, rstd = mx.mx_rmsnorm_quant_mxfp8(x, g, with_y=True)
    c0, sc0, y0, _, r0 = mx.mx_rmsnorm_quant_mxfp8(dev(tail), g, with_y=True)
    for a, b in ((c, c0), (sc, sc0), (y, y0), (rstd, r0)):
        assert torch.equal(a[-4096:], b) and torch.equal(a[:4096], b)
        assert (a[4096:rows - 4096] == a[4096:4097]).all()


# ------------------------------------------------------------------------------------------------
# backward
# ------------------------------------------------------------------------------------------------
def make_backward(rows, cols, dtype, dsum, gamma_dtype="f32", seed=50):
    s, _, g = make(rows, cols, dtype, False, gamma_dtype, seed)
    dy = wl.normal((rows, cols), 1e-2, seed=seed + 7).to(DT[dtype])
    d = wl.normal((rows, cols), 1e-2, seed=seed + 8).to(DT[dtype]) if dsum else None
    rstd = torch.rsqrt((s.float() ** 2).mean(1) + EPS)
    return dy, s, g, rstd, d


def check_backward(dx, dgamma, dy, s, g, rstd, d):
    exact, bound, dg, dgabs = ref.backward_f64(dy, s, g, rstd, d)
    got = dx.float().cpu().numpy().astype(np.float64)
    lo, hi = exact - bound, exact + bound
    if dx.dtype == torch.bfloat16:
        lo, hi = bf16_round_f64(lo), bf16_round_f64(hi)
    bad = ~((got >= lo) & (got <= hi))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())
    # a thread adds at most rows / 64 + 1 rows one after the other (64 slices of the rows, or at
    # least 256 workgroups that share more than 256 rows); then at most 4 lane steps and 16 waves,
    # or 16 rows of a workgroup and a join in 64 bits. z, the product and the last rounding: one each
    n = s.shape[0] // 64 + 1 + 20 + 3
    err = np.abs(dgamma.cpu().numpy().astype(np.float64) - dg)
    assert (err <= n * ref.EPS32 * dgabs).all(), float((err / (dgabs + 1e-300)).max())


@pytest.mark.parametrize("dsum", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", SHAPES + [(2500, 256), (1100, 2720), (20000, 128),
                                                # past 2^22 elements: dgamma by workgroups' sums
                                                (40000, 128), (8300, 512), (4500, 1024),
                                                (2100, 2048), (1600, 2720), (550, 8192),
                                                (530, 8224), (140, 32768), (257, 16416)])
def test_backward_against_the_formula(mx, rows, cols, dtype, dsum):
    dy, s, g, rstd, d = make_backward(rows, cols, dtype, dsum, "bf16" if cols % 64 else "f32")
    dx, dg = mx.mx_rmsnorm_backward(dev(dy), dev(s), dev(g), dev(rstd), dsum=dev(d))
    torch.cuda.synchronize()
    check_backward(dx, dg, dy, s, g, rstd, d)
    again, dg2 = mx.mx_rmsnorm_backward(dev(dy), dev(s), dev(g), dev(rstd), dsum=dev(d))
    assert torch.equal(dx, again) and torch.equal(dg, dg2)
    only, none = mx.mx_rmsnorm_backward(dev(dy), dev(s), dev(g), dev(rstd), dsum=dev(d),
                                        with_dgamma=False)
    assert none is None and torch.equal(only, dx)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(4096, 32), (4097, 32), (4096, 992), (8192, 96),
                                       (131072, 32), (3001, 160)])
def test_backward_of_tall_narrow_tensors(mx, rows, cols, dtype):
    """Both forms of dgamma beside the border between them, and far from it."""
    dy, s, g, rstd, d = make_backward(rows, cols, dtype, True)
    dx, dg = mx.mx_rmsnorm_backward(dev(dy), dev(s), dev(g), dev(rstd), dsum=dev(d))
    torch.cuda.synchronize()
    check_backward(dx, dg, dy, s, g, rstd, d)
    only, _ = mx.mx_rmsnorm_backward(dev(dy), dev(s), dev(g), dev(rstd), dsum=dev(d),
                                     with_dgamma=False)
    assert torch.equal(only, dx)


def test_backward_against_differences(mx):
    """d/dh of L = sum dy y(s + h v, gamma + h w) at 0, by central differences of the forward
    pass in fp32. Its noise is the rounding of y (half a step each) over h and the difference
    formula's own error, which the float64 forward gives."""
    rows, cols, h = 6, 2720, 2.0 ** -7
    dy, s, g, rstd, _ = make_backward(rows, cols, "f32", False)
    v = wl.normal((rows, cols), 1.0, seed=90)
    w = wl.normal((1, cols), 1.0, seed=91)[0]
    _, _, rstd = mx.mx_rmsnorm(dev(s), dev(g), eps=EPS)
    dx, dg = mx.mx_rmsnorm_backward(dev(dy), dev(s), dev(g), rstd)
    got = float((dx.double().cpu() * v.double()).sum() + (dg.double().cpu() * w.double()).sum())
    L, L64, noise = [], [], 0.0
    for sign in (1.0, -1.0):
        sh, gh = s + sign * h * v, g + sign * h * w  # the fp32 points that both sides take
        y = mx.mx_rmsnorm(dev(sh), dev(gh), eps=EPS)[0].double().cpu()
        L.append(float((dy.double() * y).sum()))
        y64, _ = ref.norm_f64(sh, gh, EPS)
        L64.append(float((dy.double().numpy() * y64).sum()))
        noise += float((dy.double() * y).abs().sum()) * ref.EPS32
    fd, fd64 = (L[0] - L[1]) / (2 * h), (L64[0] - L64[1]) / (2 * h)
    exact, bound, dge, dgabs = ref.backward_f64(dy, s, g, rstd, None)
    want = float((exact * v.double().numpy()).sum() + (dge * w.double().numpy()).sum())
    assert abs(fd - fd64) <= noise / (2 * h)
    # truncation: the float64 difference against the float64 gradient, and rstd's half step
    slack = abs(fd64 - want)
    assert slack <= 0.02 * abs(want)
    fp32 = float((bound * np.abs(v.double().numpy())).sum()
                 + 24 * ref.EPS32 * (dgabs * np.abs(w.double().numpy())).sum())
    assert abs(got - fd) <= noise / (2 * h) + slack + fp32


@pytest.mark.parametrize("rows,cols", [(9, 1056), (4100, 1056)])
def test_backward_leading_dimensions_and_aliasing(mx, rows, cols):
    pad = 40
    dy, s, g, rstd, d = (dev(t) for t in make_backward(rows, cols, "bf16", True))
    dx0, dg0 = mx.mx_rmsnorm_backward(dy, s, g, rstd, dsum=d)
    wide = [torch.full((rows, cols + pad), 7.0, dtype=s.dtype, device=DEV) for _ in range(4)]
    for w, t in zip(wide, (dy, s, d)):
        w[:, :cols].copy_(t)
    wdy, ws, wd, wdx = (w[:, :cols] for w in wide)
    dx, dg = mx.mx_rmsnorm_backward(wdy, ws, g, rstd, dsum=wd, dx=wdx)
    assert torch.equal(wdx, dx0) and torch.equal(dg, dg0)
    size = mx.lib().mx_rmsnorm_backward_workspace(rows, cols)
    assert (size > 0) == (rows * cols > 1 << 22)
    work = torch.full((size + 16,), 0xA5, dtype=torch.uint8, device=DEV)
    _, dg = mx.mx_rmsnorm_backward(wdy, ws, g, rstd, dsum=wd, dx=wd, workspace=work[:size])
    assert torch.equal(wd, dx0) and torch.equal(dg, dg0)  # over dsum
    assert (work[size:] == 0xA5).all()
    wd.copy_(d)
    mx.mx_rmsnorm_backward(wdy, ws, g, rstd, dsum=wd, dx=wdy, with_dgamma=False)  # over dy
    assert torch.equal(wdy, dx0)
    with pytest.raises(mx.MxError):
        mx.mx_rmsnorm_backward(wdy, ws, g, rstd, dx=wdy)
    for w in wide:
        assert (w[:, cols:] == 7.0).all()


@pytest.mark.parametrize("rows,cols", [(65, 4096), (1030, 4096)])
def test_streams_and_graph_replays(mx, rows, cols):
    """The norm and its backward pass (without and with a workspace) captured together on a side
    stream, replayed on new inputs beside eager calls."""
    x, r, g = (dev(t) for t in make(rows, cols, "bf16", True))
    dy = dev(wl.normal((rows, cols), 1e-2, seed=3).to(torch.bfloat16))

    def step():
        c, sc, y, s, rstd = mx.mx_rmsnorm_quant_mxfp8(x, g, r, scale_rule=1, hadamard=1,
                                                      sign_mask=MASK, with_y=True)
        dx, dg = mx.mx_rmsnorm_backward(dy, s, g, rstd, dsum=y)
        return c, sc, y, s, rstd, dx, dg

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (11, 22, 33):
        nx, nr, _ = make(rows, cols, "bf16", True, seed=seed)
        x.copy_(nx)
        r.copy_(nr)
        eager = step()
        torch.cuda.synchronize()
        for t in out:
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, out):
            assert torch.equal(a, b)
    # an explicit stream
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
        dx, dg = mx.mx_rmsnorm_backward(dy, eager[3], g, eager[4], dsum=eager[2], stream=side)
    torch.cuda.synchronize()
    assert torch.equal(dx, eager[5]) and torch.equal(dg, eager[6])
