"""The normalisation and few-token operators: cases, inputs, plain forms and work.

  norm      RMS norm with the residual's addition and an MXFP8 output (E8M0 scale per 32 values)
  norm_bwd  its backward pass
  gemv      product of a few tokens with MXFP4 weights (E2M1 codes, one E8M0 scale per 32)

Sizes are the hidden, MLP and key widths of the 8B and 70B workloads (4096, 14336; 8192, 28672,
heads of 128), their token counts (8192, 16384), single tokens, and ragged ones.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
EMAX = {"e4m3": 8, "e5m2": 15}
EPS = 1e-5
SIGN_MASK = 0x9E3779B9
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _norm(name, rows, cols, dtype="bf16", residual=True, fmt="e4m3", ceil=False, hadamard=False,
          with_y=False):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "dtype": dtype,
            "residual": residual, "fmt": fmt, "ceil": ceil, "hadamard": hadamard,
            "with_y": with_y}


def _bwd(name, rows, cols, dtype="bf16", dsum=True):
    return {"name": name, "op": "norm_bwd", "rows": rows, "cols": cols, "dtype": dtype,
            "dsum": dsum}


def _gemv(name, T, N, K, dtype="bf16", hadamard=False, tile=1):
    return {"name": name, "op": "gemv", "T": T, "N": N, "K": K, "dtype": dtype,
            "hadamard": hadamard, "tile": tile}


def listed():
    return [
        # one decoded token entering an 8B layer: latency
        _norm("norm_token_8b", 1, 4096),
        # a training step's tokens before the 8B MLP; y is kept for the weight gradient
        _norm("norm_train_8b", 8192, 4096, with_y=True),
        # one GPU's tokens of the 70B model, the truncation-free scale
        _norm("norm_train_70b", 16384, 8192, ceil=True, with_y=True),
        # fp32 activations, ragged width, rotated E5M2 output
        _norm("norm_ragged_f32", 1000, 2720, dtype="f32", residual=False, fmt="e5m2",
              hadamard=True),
        # per-head norm of 64 query heads of 128 for 4096 tokens, no residual
        _norm("norm_heads", 262144, 128, residual=False),
        # backward passes of the training cases, the gradient of the residual stream joining
        _bwd("norm_bwd_8b", 8192, 4096),
        _bwd("norm_bwd_70b", 16384, 8192),
        _bwd("norm_bwd_ragged_f32", 777, 2720, dtype="f32", dsum=False),
        # one token through the 8B up projection and the 70B down projection
        _gemv("gemv_token_8b_up", 1, 14336, 4096),
        _gemv("gemv_token_70b_down", 1, 8192, 28672),
        # a batch of 16 sequences decoding against rotated 70B up weights
        _gemv("gemv_batch_70b_up", 16, 28672, 8192, hadamard=True),
        # a ragged batch in fp32, an odd number of outputs, K an odd number of blocks
        _gemv("gemv_ragged_f32", 37, 1003, 4128, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "gemv"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "gemv":
        tile = rng.choice([1, 1, 32])
        n = _log_int(rng, 17, 28672)
        return {"op": op, "T": _log_int(rng, 1, 64), "N": n if tile == 1 else -(-n // tile) * tile,
                "K": 32 * _log_int(rng, 2, 512), "dtype": dtype,
                "hadamard": tile == 1 and rng.random() < 0.3, "tile": tile}
    cols = 32 * _log_int(rng, 1, 256)
    most = (16384 * 8192) // (2 if dtype == "f32" else 1) // cols
    rows = _log_int(rng, 1, min(most, 262144))
    if op == "norm":
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype,
                "residual": rng.random() < 0.6, "fmt": rng.choice(["e4m3", "e4m3", "e5m2"]),
                "ceil": rng.random() < 0.5, "hadamard": rng.random() < 0.3,
                "with_y": rng.random() < 0.5}
    return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "dsum": rng.random() < 0.5}


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "gemv":
        T, N, K, g = case["T"], case["N"], case["K"], case["tile"]
        return {"bytes": N * K // 2 + N // g * (K // 32) + T * (N + K) * e, "flops": 2 * T * N * K}
    rows, cols = case["rows"], case["cols"]
    n = rows * cols
    if case["op"] == "norm":  # x (, residual in, sum out), codes, scales, (y,) gamma, rstd
        b = n * e * (1 + 2 * case["residual"] + case["with_y"]) + n + n // 32 + 4 * cols + 4 * rows
        return {"bytes": b, "flops": 6 * n + (192 * n // 32 if case["hadamard"] else 0)}
    # dy, s, dx (, gradient of the sum), gamma, its gradient, rstd
    return {"bytes": n * e * (3 + case["dsum"]) + 8 * cols + 4 * rows, "flops": 9 * n}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=F32)


def _hidden(gen, rows, cols, dtype):
    """Hidden states: normal, one channel in 200 (one at least) twenty times the others."""
    x = _randn(gen, rows, cols)
    at = torch.randint(0, cols, (max(1, cols // 200),), generator=gen, device="cuda")
    x[:, at] *= 20.0
    return x.to(dtype)


def _weights(gen, N, K, tile, std):
    """MXFP4 weights ~ N(0, std): floor scales per 1x32 block or tile x tile square, nearest
    codes, two a byte, the even element in the low nibble."""
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((N // tile, K // 32), dtype=torch.uint8, device="cuda")
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = 4096
    for n0 in range(0, N, step):
        n = min(step, N - n0)
        w = _randn(gen, n, K) * std
        amax = w.view(n // tile, tile, K // 32, 32).abs().amax(dim=(1, 3))
        b = ((amax.view(torch.int32) >> 23) - 2).clamp(min=0)
        inv = ((254 - b) << 23).view(F32)
        v = (w.view(n // tile, tile, K // 32, 32) * inv[:, None, :, None]).view(n, K)
        c = torch.bucketize(v.abs(), borders, out_int32=True) | ((v < 0).to(torch.int32) << 3)
        codes[n0:n0 + n] = (c[:, 0::2] | (c[:, 1::2] << 4)).to(torch.uint8)
        scales[n0 // tile:(n0 + n) // tile] = b.to(torch.uint8)
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    dtype = DTYPES[case["dtype"]]
    st = {"case": case}
    if case["op"] == "gemv":
        st["x"] = _hidden(gen, case["T"], case["K"], dtype)
        st["wq"], st["ws"] = _weights(gen, case["N"], case["K"], case["tile"],
                                      0.02 * (32 ** 0.5 if case["hadamard"] else 1.0))
        return st
    rows, cols = case["rows"], case["cols"]
    st["gamma"] = 1.0 + 0.1 * _randn(gen, cols)
    x = _hidden(gen, rows, cols, dtype)
    if case["op"] == "norm":
        st["x"] = x
        st["residual"] = (2.0 * _randn(gen, rows, cols)).to(dtype) if case["residual"] else None
        return st
    st["s"] = x
    st["rstd"] = torch.rsqrt((x.float() ** 2).mean(1) + EPS)
    st["dy"] = (1e-3 * _randn(gen, rows, cols)).to(dtype)
    st["dsum"] = (1e-3 * _randn(gen, rows, cols)).to(dtype) if case["dsum"] else None
    return st


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    return {"norm": _plain_norm, "norm_bwd": _plain_bwd, "gemv": _plain_gemv}[case["op"]](state, case)


def _run_own(st, case):
    import mxfp4_block_scaled_hadamard32_amd as mx
    mask = SIGN_MASK if case.get("hadamard") else 0
    if case["op"] == "norm":
        codes, scales, y, s, rstd = mx.mx_rmsnorm_quant_mxfp8(
            st["x"], st["gamma"], residual=st["residual"], eps=EPS,
            fmt=mx.MX_E4M3 if case["fmt"] == "e4m3" else mx.MX_E5M2,
            scale_rule=mx.MX_SCALE_CEIL if case["ceil"] else mx.MX_SCALE_FLOOR,
            hadamard=int(case["hadamard"]), sign_mask=mask, with_y=case["with_y"])
        return {"codes": codes.view(F8[case["fmt"]]), "scales": scales.view(torch.float8_e8m0fnu),
                "y": y, "sum": s if case["residual"] else None, "rstd": rstd}
    if case["op"] == "norm_bwd":
        dx, dgamma = mx.mx_rmsnorm_backward(st["dy"], st["s"], st["gamma"], st["rstd"],
                                            dsum=st["dsum"])
        return {"dx": dx, "dgamma": dgamma}
    return mx.mx_gemv(st["x"], st["wq"], st["ws"], case["tile"], hadamard=int(case["hadamard"]),
                      sign_mask=mask, alpha_exp=-5 if case["hadamard"] else 0,
                      out_dtype=st["x"].dtype)


def _signs_f32(device):
    bits = torch.arange(32, device=device)
    return 1.0 - 2.0 * ((SIGN_MASK >> bits) & 1).to(F32)


def _rotate_f32(x):
    """Signs and the unnormalised 32-point Walsh-Hadamard transform of each 32-block."""
    i = torch.arange(32, device=x.device)
    a = i[:, None] & i[None, :]
    a = a ^ (a >> 4)
    a = a ^ (a >> 2)
    a = a ^ (a >> 1)
    H = 1.0 - 2.0 * (a & 1).to(F32)
    return ((x.view(-1, 32) * _signs_f32(x.device)) @ H).view(x.shape)


def _plain_norm(st, case):
    s = st["x"].float()
    total = None
    if case["residual"]:
        total = (s + st["residual"].float()).to(st["x"].dtype)  # the stored residual stream
        s = total.float()
    rstd = torch.rsqrt((s * s).mean(1) + EPS)
    y = s * rstd[:, None] * st["gamma"]
    v = _rotate_f32(y) if case["hadamard"] else y
    v = v.view(y.shape[0], -1, 32)
    bits = v.abs().amax(2).view(torch.int32)
    e = (bits >> 23) - EMAX[case["fmt"]]
    if case["ceil"]:
        e = e + ((bits & 0x7FFFFF) > 0x600000)
    e = e.clamp(min=0)
    v = v * ((254 - e) << 23).view(F32)[:, :, None]
    big = LARGEST[case["fmt"]]
    codes = v.clamp(-big, big).view(y.shape).to(F8[case["fmt"]])
    return {"codes": codes, "scales": e.to(torch.uint8).view(torch.float8_e8m0fnu),
            "y": y.to(st["x"].dtype) if case["with_y"] else None, "sum": total, "rstd": rstd}


def _plain_bwd(st, case):
    s, dy = st["s"].float(), st["dy"].float()
    rstd = st["rstd"][:, None]
    z = s * rstd
    u = dy * st["gamma"]
    dx = (u - z * (u * z).mean(1, keepdim=True)) * rstd
    if case["dsum"]:
        dx = dx + st["dsum"].float()
    return {"dx": dx.to(st["s"].dtype), "dgamma": (dy * z).sum(0)}


def _plain_gemv(st, case):
    wq = st["wq"]
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=wq.device, dtype=F32)
    byte = torch.arange(256, device=wq.device)
    pair = torch.stack([grid[byte & 15], grid[byte >> 4]], 1)
    w = pair[wq.int()].view(wq.shape[0], -1, 32)
    # 2^(b - 127): b = 0 is the subnormal 2^-127
    e = st["ws"].float() - 127.0
    scale = torch.exp2(e)
    w = (w * scale.repeat_interleave(case["tile"], 0)[:, :, None]).view(wq.shape[0], -1)
    x = st["x"].float()
    if case["hadamard"]:
        x = _rotate_f32(x) * 2.0 ** -5
    return (x @ w.t()).to(st["x"].dtype)


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------
def _hadamard_f64(x):
    """sum_j (-1)^popcount(i & j) sign_j x_j over each block of 32, as Kronecker factors."""
    h2 = torch.tensor([[1.0, 1.0], [1.0, -1.0]], dtype=torch.float64, device=x.device)
    H = h2
    while H.shape[0] < 32:
        H = torch.kron(H, h2)
    d = torch.tensor([-1.0 if (SIGN_MASK >> j) & 1 else 1.0 for j in range(32)],
                     dtype=torch.float64, device=x.device)
    return (x.reshape(-1, 32) @ (d[:, None] * H)).reshape(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        s = st["x"].double()
        if case["residual"]:
            s = (s + st["residual"].double()).to(st["x"].dtype).double()
        rstd = 1.0 / torch.sqrt(s.square().sum(1) / case["cols"] + EPS)
        y = s.mul(rstd[:, None]).mul_(st["gamma"].double())
        v = _hadamard_f64(y) if case["hadamard"] else y
        v = v.reshape(case["rows"], case["cols"] // 32, 32)
        mant, ex = torch.frexp(v.abs().amax(2))          # mant in [1/2, 1)
        e = ex.double() - 1 - EMAX[case["fmt"]]
        if case["ceil"]:
            e = e + (mant > 0.875).double()              # largest / 2^(emax + 1)
        scale = torch.exp2(e)
        big = LARGEST[case["fmt"]]
        # the one rounding, to 3 or 2 mantissa bits: steps of 2^(exponent - bits), those of the
        # least normal exponent below it; torch.round takes ties to even
        v = (v / scale[:, :, None]).clamp(-big, big).reshape(case["rows"], case["cols"])
        bits, least = (3, -6) if case["fmt"] == "e4m3" else (2, -14)
        step = torch.exp2(((torch.frexp(v).exponent - 1).clamp_(min=least) - bits).double())
        v = torch.round(v / step).mul_(step).clamp_(-big, big)
        return {"codes": v, "scales": scale, "y": y if case["with_y"] else None,
                "sum": s if case["residual"] else None, "rstd": rstd}
    if case["op"] == "norm_bwd":
        s, dy, r = st["s"].double(), st["dy"].double(), st["rstd"].double()[:, None]
        z = s.mul_(r)
        dgamma = (dy * z).sum(0)
        u = dy.mul_(st["gamma"].double())
        c = (u * z).sum(1, keepdim=True) / case["cols"]
        dx = u.sub_(z.mul_(c)).mul_(r)
        return {"dx": dx + st["dsum"].double() if case["dsum"] else dx, "dgamma": dgamma}
    x = st["x"].double()
    if case["hadamard"]:
        x = _hadamard_f64(x) / 32.0
    out = torch.empty((case["T"], case["N"]), dtype=torch.float64, device=x.device)
    for n0 in range(0, case["N"], 4096):
        q = st["wq"][n0:n0 + 4096]
        c = torch.stack([q & 15, q >> 4], 2).reshape(q.shape[0], -1)
        m = (c & 7).double()
        # magnitude: m / 2 below 2, else (2 + (m & 1)) 2^(floor(m / 2) - 2)
        mag = torch.where(m < 2, m / 2, (2 + m % 2) * torch.exp2(torch.floor(m / 2) - 2))
        w = torch.where(c >= 8, -mag, mag).reshape(q.shape[0], -1, 32)
        rows = torch.arange(n0, n0 + q.shape[0], device=x.device) // case["tile"]
        w = w * torch.exp2(st["ws"].double() - 127)[rows][:, :, None]
        out[:, n0:n0 + 4096] = x @ w.reshape(q.shape[0], -1).t()
    return out
