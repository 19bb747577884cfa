"""The norm, the linear layer and the few-token product as they are used together: a training
half-layer (norm, quantized operand, products, both backward passes), the same captured and
replayed, and a decoding step, against the oracle and against the separate calls."""
import numpy as np
import pytest
import torch

import workloads as wl
from tests import norm_reference as ref
from tests.parity import bf16_round_f64, check_gemm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MASK = 0x2C6FE9B1


@pytest.fixture(scope="module")
def mx():
    import mxfp4_block_scaled_hadamard32_amd as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.lib()
    return m


@pytest.fixture(scope="module")
def lin(mx):
    from mxfp4_block_scaled_hadamard32_amd import linear
    return linear


def tensors(T, K, N, seed=1):
    bf = lambda t: t.to(torch.bfloat16).to(DEV)  # noqa: E731
    return (bf(wl.student_t3((T, K), seed=seed)), bf(wl.normal((T, K), 2.0, seed=seed + 1)),
            bf(wl.normal((T, N), 1e-2, seed=seed + 2)), bf(wl.normal((T, K), 1e-2, seed=seed + 3)))


def config(lin, variant):
    if variant == "mxfp8":
        return lin.MXLinearConfig(fmt="mxfp8", seed=40)
    f = lin.QuantSpec(scale_rule=1, round=1, hadamard=1, sign_mask=MASK)
    w = lin.QuantSpec(scale_rule=1, round=0, hadamard=1, sign_mask=0)
    return lin.MXLinearConfig(fprop_q=f, dgrad_q=f, wgrad_q=w, seed=40)


@pytest.mark.parametrize("variant", ["mxfp4", "mxfp8", "off"])
def test_training_half_layer(mx, lin, orc, variant):
    T, K, N = 256, 512, 384
    x, r, dout, dsum = tensors(T, K, N)
    cfg = config(lin, variant)
    if variant == "off":
        cfg.fprop = cfg.dgrad = cfg.wgrad = False
    layer = lin.MXNormLinear(K, N, cfg)
    with torch.no_grad():
        layer.norm.weight.copy_(1.0 + wl.normal((1, K), 0.2, seed=9)[0])
    x.requires_grad_(True)
    r.requires_grad_(True)
    out, s = layer(x, r)
    torch.autograd.backward((out, s), (dout, dsum))
    g, w = layer.norm.weight.detach(), layer.linear.weight.detach()

    # the same step by the separate calls
    xd, rd = x.detach(), r.detach()
    y, s1, rstd = mx.mx_rmsnorm(xd, g, rd)
    assert torch.equal(s1, s)
    f = cfg.fprop_q
    kw = dict(scale_rule=f.scale_rule, round=f.round, hadamard=f.hadamard, sign_mask=f.sign_mask)
    if variant == "mxfp4":
        c, sc, y1, _, _ = mx.mx_rmsnorm_quant(xd, g, rd, seed=40, with_y=True, **kw)
        assert torch.equal(y1, y)
        wq, ws = mx.mx_quantize(w, seed=41, **kw)
        # the forward product against the oracle's exact product of the codes
        C, Cabs = orc.gemm(c.cpu().numpy(), sc.cpu().numpy(), 1, wq.cpu().numpy(),
                           ws.cpu().numpy(), 1, T, N, K, -5)
        check_gemm(out.detach(), C, Cabs)
    elif variant == "off":
        assert torch.equal(out, y @ w.t())
    wy = w.clone().requires_grad_(True)
    yy = y.clone().requires_grad_(True)
    twin = config(lin, variant)
    if variant == "off":
        twin.fprop = twin.dgrad = twin.wgrad = False
    lin.MXLinearFunction.apply(yy, wy, twin).backward(dout)
    assert torch.equal(layer.linear.weight.grad, wy.grad)
    dx, dg = mx.mx_rmsnorm_backward(yy.grad, s1, g, rstd, dsum=dsum)
    assert torch.equal(x.grad, dx) and torch.equal(r.grad, dx)
    assert torch.equal(layer.norm.weight.grad, dg)
    exact, bound, dge, dgabs = ref.backward_f64(yy.grad, s1, g, rstd, dsum)
    got = x.grad.double().cpu().numpy()
    assert ((got >= bf16_round_f64(exact - bound)) & (got <= bf16_round_f64(exact + bound))).all()


def test_norm_module_shapes_and_gradients(lin):
    """[batch][time][K], an expanded gradient, only one of the outputs used, a frozen weight."""
    K = 96
    norm = lin.MXRMSNorm(K)
    x = wl.student_t3((10, K), seed=3).to(DEV).view(2, 5, K).requires_grad_(True)
    r = wl.student_t3((10, K), seed=4).to(DEV).view(2, 5, K).requires_grad_(True)

    def plain(x, r):
        s = x if r is None else x + r
        return s * torch.rsqrt((s * s).mean(-1, keepdim=True) + norm.eps) * norm.weight.double(), s

    for use in ("y", "s", "both", "no residual"):
        res = None if use == "no residual" else r
        x.grad = r.grad = norm.weight.grad = None
        out = norm(x, res)
        y, s = (out, None) if res is None else out
        assert y.shape == x.shape and (s is None or s.shape == x.shape)
        loss = 0.0
        if use != "s":
            loss = loss + y.sum()                # its gradient is an expanded scalar
        if use in ("s", "both"):
            loss = loss + (s * s).sum()
        loss.backward()
        xd = x.detach().double().requires_grad_(True)
        rd = None if res is None else r.detach().double().requires_grad_(True)
        py, ps = plain(xd, rd)
        want = 0.0
        if use != "s":
            want = want + py.sum()
        if use in ("s", "both"):
            want = want + (ps * ps).sum()
        want.backward()
        # the formula's bound (norm_reference.backward_f64), and the gradient 2 s rounded once
        sd, _, rho = (t.detach() for t in (ps, py, 1 / torch.sqrt((ps * ps).mean(-1) + norm.eps)))
        flat = lambda t: t.reshape(10, K)  # noqa: E731
        dy = torch.zeros((10, K)) if use == "s" else torch.ones((10, K))
        ds = flat(2 * sd).float() if use in ("s", "both") else None
        exact, bound, _, _ = ref.backward_f64(dy, flat(sd), norm.weight, rho.reshape(10), ds)
        # s, rstd and 2 s are fp32 in the kernel: half a step each on terms that the bound counts
        assert (np.abs(flat(x.grad).double().cpu().numpy() - flat(xd.grad).cpu().numpy())
                <= 3 * bound + 4 * 2.0 ** -24 * np.abs(exact)).all()
        if res is not None:
            assert torch.equal(r.grad, x.grad)
        if use == "s":
            assert norm.weight.grad is None or (norm.weight.grad == 0).all()
    norm.weight.requires_grad_(False)
    x.grad = norm.weight.grad = None
    norm(x).sum().backward()
    assert x.grad is not None and norm.weight.grad is None


def test_norm_gradient_views_and_second_order(lin):
    """Gradients that are views into a flat buffer at any element; a second derivative is refused."""
    K = 96
    norm = lin.MXRMSNorm(K)
    x = wl.student_t3((10, K), seed=5).to(DEV).requires_grad_(True)
    r = wl.student_t3((10, K), seed=6).to(DEV).requires_grad_(True)
    y, s = norm(x, r)
    flat = wl.normal((10 * K + 1, 2), 1.0, seed=7).to(DEV).t().contiguous()
    dy, ds = (f[1:].view(10, K) for f in flat)
    assert dy.data_ptr() % 16 and ds.data_ptr() % 16
    got = torch.autograd.grad((y, s), (x, r, norm.weight), (dy, ds), retain_graph=True)
    want = torch.autograd.grad((y, s), (x, r, norm.weight), (dy.clone(), ds.clone()),
                               retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    dy = dy.clone().requires_grad_(True)
    dx, = torch.autograd.grad(y, x, dy, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()


@pytest.mark.parametrize("layout", ["flat", "expanded", "odd", "windows", "columns"])
def test_inputs_and_weights_in_any_layout(mx, lin, layout):
    """Inputs and weights that are views into a flat buffer at any element, rows repeated or with
    odd distances: outputs and gradients as for contiguous copies."""
    T, K, N = 64, 128, 96

    def lay(t):
        if layout == "flat":
            v = torch.cat([t.new_zeros(1), t.reshape(-1)])[1:].view(t.shape)
            assert v.data_ptr() % 16
        elif t.dim() == 1:
            v = t
        elif layout == "expanded":
            v = t[:1].expand(t.shape)
        elif layout == "odd":
            v = torch.cat([t, t.new_zeros(t.shape[0], 3)], 1)[:, :K]
        elif layout == "windows":
            v = t.reshape(-1)[:K + 8 * (t.shape[0] - 1)].as_strided(t.shape, (8, 1))
        else:
            v = t.t().contiguous().t()
        return v

    x, r, _, dsum = (t.detach() for t in tensors(T, K, N))
    dout = wl.normal((T, N), 1e-2, seed=8).to(torch.bfloat16).to(DEV)
    gamma = (1.0 + wl.normal((1, K), 0.2, seed=9)[0]).to(DEV)
    layer = lin.MXNormLinear(K, N, lin.MXLinearConfig())
    vx, vr, vg = lay(x), lay(r), lay(gamma)

    def step(x, r, g):
        layer.norm.weight = torch.nn.Parameter(g)
        layer.linear.cfg.seed = 5
        x, r = x.detach().requires_grad_(True), r.detach().requires_grad_(True)
        out, s = layer(x, r)
        y, s2 = layer.norm(x.view(4, -1, K) if x.is_contiguous() else x, r.view(4, -1, K)
                           if x.is_contiguous() else r)
        alone = layer.norm(x)
        grads = torch.autograd.grad((out, s, alone), (x, r, layer.norm.weight,
                                                      layer.linear.weight), (dout, dsum, dsum))
        return (out, s, y.reshape(T, K), s2.reshape(T, K), alone) + grads

    for a, b in zip(step(vx, vr, vg), step(vx.clone(memory_format=torch.contiguous_format),
                                           vr.clone(memory_format=torch.contiguous_format),
                                           vg.clone())):
        assert torch.equal(a, b)
    w = layer.linear.weight.detach()
    decode, plain = lin.MXDecodeLinear(lay(w)), lin.MXDecodeLinear(lay(w).clone(
        memory_format=torch.contiguous_format))
    assert torch.equal(decode.codes, plain.codes)
    assert torch.equal(decode(vx), decode(vx.clone(memory_format=torch.contiguous_format)))


def test_training_step_in_a_graph(lin):
    """Forward and backward of the half-layer captured once and replayed on new inputs; no eager
    graph of the same leaves is alive meanwhile."""
    T, K, N = 128, 512, 256
    layer = lin.MXNormLinear(K, N, lin.MXLinearConfig())
    x, r, dout, dsum = tensors(T, K, N)
    x.requires_grad_(True)
    r.requires_grad_(True)
    leaves = (x, r, layer.norm.weight, layer.linear.weight)

    def step():
        out, s = layer(x, r)
        grads = torch.autograd.grad((out, s), leaves, (dout, dsum))
        return (out.detach(), s.detach()) + grads

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (5, 6, 7):
        with torch.no_grad():
            for t, n in zip((x, r, dout, dsum), tensors(T, K, N, seed)):
                t.copy_(n)
        eager = [t.clone() for t in step()]
        torch.cuda.synchronize()
        for t in captured:
            t.fill_(1)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, captured):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("w_block,hadamard", [(1, 0), (1, 1), (32, 0), (64, 0)])
def test_decoding_step(mx, lin, orc, w_block, hadamard, dtype):
    """norm -> few-token product with a trained layer's weights, one token and five at once."""
    K, N = 1024, 320
    spec = lin.QuantSpec(scale_rule=1, round=1, hadamard=hadamard, sign_mask=MASK if hadamard else 0)
    cfg = lin.MXLinearConfig(fprop_q=spec, dgrad_q=spec, wgrad_q=spec, w_block=w_block)
    layer = lin.MXLinear(K, N, cfg)
    decode = lin.MXDecodeLinear.from_linear(layer)
    norm = lin.MXRMSNorm(K)
    for shape in ((1, K), (5, K), (2, 3, K), (0, K)):
        rows = int(np.prod(shape[:-1]))
        x = wl.student_t3((max(rows, 1), K), seed=3)[:rows].view(shape).to(dtype).to(DEV)
        r = wl.normal((max(rows, 1), K), 2.0, seed=4)[:rows].view(shape).to(dtype).to(DEV)
        with torch.no_grad():
            y, s = norm(x, r)
        out = decode(y)
        assert out.shape == shape[:-1] + (N,) and out.dtype == dtype
        if rows == 0:
            continue
        W = orc.dequantize_f64(decode.codes.cpu().numpy(), decode.scales.cpu().numpy(), N, K,
                               w_block)
        X = y.reshape(rows, K).double().cpu().numpy()
        A = 0.0
        if hadamard:
            A = np.abs(X).reshape(rows, K // 32, 32).sum(2).repeat(32, axis=1) @ np.abs(W).T / 32
            X = ref.hadamard_f64(X, MASK) / 32
        # the product's bound; bf16 tokens that are rotated keep 16 bits
        Cabs = np.abs(X) @ np.abs(W).T * (2.0 ** -16 + 2.0 ** -17) + 5 * 2.0 ** -24 * A
        check_gemm(out.reshape(rows, N), X @ W.T, Cabs, rel=1.0)


def test_decode_layer_refusals(lin):
    with pytest.raises(ValueError):
        lin.MXDecodeLinear(torch.zeros((64, 64), dtype=torch.bfloat16), w_block=8)
    with pytest.raises(ValueError):
        lin.MXDecodeLinear(torch.zeros((64, 64), dtype=torch.bfloat16),
                           lin.QuantSpec(hadamard=1), w_block=32)
    with pytest.raises(ValueError):
        lin.MXDecodeLinear.from_linear(
            lin.MXLinear(128, 128, lin.MXLinearConfig(fmt="mxfp8")))
