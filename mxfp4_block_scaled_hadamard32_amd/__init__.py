"""MXFP4 block-scaled Hadamard-32 hot path for AMD MI355X (gfx950).

Python face of the C ABI in include/mx.h (libmx.so). Each function marshals torch tensors (device
memory, current HIP stream) into one library call; the quantizer, dequantizer and GEMMs all run
in the library's HIP kernels.

  mx_quantize     1x32 blocks, optional 32-point Hadamard rotation with random signs, floor or
                  ceil E8M0 scale, RNE or Philox stochastic rounding, packed E2M1 codes
  mx_quantize_2d  32x32 transposition-invariant blocks, plus the transposed K-major copy
  mx_dequantize   codes * 2^(scale-127), optional inverse rotation
  mx_gemm_fprop / mx_gemm_dgrad / mx_gemm_wgrad   block-scaled MXFP4 GEMMs, fp32 accumulate
  mx_gemm_fprop_quant   Fprop whose output tile is quantized (1x32 along N) in the epilogue
  mx_quantize_2d_blocks   8x8, 32x32 or 64x64 tiles (64x64 scales in the GEMM layout, g = 64)
  mx_scale_mismatch_map   per-element scale exponent of the row block minus the column block
  mx_quantize_mxfp8 / mx_gemm_mxfp8   MXFP8 (E4M3 / E5M2 elements, the same E8M0 block scales)
                  quantize and block-scaled GEMM, for the query / key projections
  mx_rmsnorm / mx_rmsnorm_quant / mx_rmsnorm_quant_mxfp8   RMS norm with the residual's addition,
                  its result in the input's type and / or quantized in 1x32 blocks
  mx_rmsnorm_backward   gradients of the norm's input and weight
  mx_gemv         product of a few tokens (bf16 / fp32, not quantized) with MXFP4 weights
  mx_cache_write / mx_cache_read   keys and values into a paged cache of 8-bit codes with one scale
                  for 32 tokens of a head, and back
  mx_cache_attention   causal attention of each sequence's newest tokens over that cache
  mx_lora         low-rank adapters, each token its own, beside a shared projection

Each takes the stream to run on (None: the current one). Outputs that a call allocates belong to the
current stream's pool, scratch to that of the stream it runs on: a caller who passes another stream
lets it wait for the current one before the call, and the current one for it before the outputs are
used or freed.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _lib
from ._lib import (MX_BF16, MX_E4M3, MX_E5M2, MX_F32, MX_ROUND_RNE, MX_ROUND_SR, MX_SCALE_CEIL,
                   MX_SCALE_FLOOR, MxError, check, lib, mx_quant_opts)

__all__ = ["mx_quantize", "mx_quantize_2d", "mx_dequantize", "mx_gemm_fprop", "mx_gemm_dgrad",
           "mx_gemm_wgrad", "mx_gemm_fprop_quant", "mx_quantize_mxfp8", "mx_gemm_mxfp8", "mx_quantize_2d_blocks",
           "mx_scale_mismatch_map", "mx_rmsnorm", "mx_rmsnorm_quant", "mx_rmsnorm_quant_mxfp8",
           "mx_rmsnorm_backward", "mx_gemv", "mx_cache_write", "mx_cache_read",
           "mx_cache_attention", "mx_lora", "MxError",
           "MX_SCALE_FLOOR", "MX_SCALE_CEIL", "MX_ROUND_RNE", "MX_ROUND_SR", "MX_E4M3", "MX_E5M2",
           "lib"]


def _stream(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return MX_BF16
    if x.dtype == torch.float32:
        return MX_F32
    raise TypeError("mx_quantize takes bfloat16 or float32 input")


def _src(x: torch.Tensor):
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("expected a 2-D CUDA tensor with contiguous rows")
    return x.shape[0], x.shape[1], x.stride(0)


def _buf(t, name: str, shape, dtypes, device, rows_only: bool = False):
    """Checks a caller-supplied buffer before its address goes to a kernel: a tensor on `device`
    with one of `dtypes` and exactly `shape`, contiguous (rows_only: only its rows contiguous,
    for outputs with a leading dimension). Raises ValueError / TypeError otherwise."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape
            and t.device == device and t.is_contiguous()):
        return t  # what nearly every call has; the rest finds out what is wrong
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != torch.device(device):
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if rows_only:
        if t.dim() != 2 or (t.numel() > 0 and (t.stride(1) != 1 or t.stride(0) < shape[1])):
            raise ValueError(f"{name} must have contiguous rows")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


_U8 = (torch.uint8,)


def _codes_out(t, name, shape, device):
    """A code or scale output: allocated when None, else checked."""
    if t is None:
        return torch.empty(shape, dtype=torch.uint8, device=device)
    return _buf(t, name, shape, _U8, device)


def _operand(q, s, g: int, name: str, k_bytes_per_elem: float = 0.5):
    """A packed GEMM operand (codes [rows][K * bytes per element], scales [rows / g][K / 32])
    on a CUDA device; returns (rows, K)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 2 or not q.is_cuda:
        raise ValueError(f"{name} codes must be a 2-D CUDA tensor")
    rows, width = q.shape
    if (k_bytes_per_elem == 0.5 and g == 1 and q.dtype is torch.uint8 and q.is_contiguous()
            and isinstance(s, torch.Tensor) and s.dtype is torch.uint8
            and s.shape == (rows, width // 16) and s.device == q.device and s.is_contiguous()):
        return rows, 2 * width  # what nearly every call has; the rest finds out what is wrong
    K = int(round(width / k_bytes_per_elem))
    _buf(q, f"{name} codes", tuple(q.shape), _U8, q.device)
    if int(g) not in (1, 32, 64) or rows % int(g):
        raise ValueError(f"{name} scale granularity {g} does not divide its {rows} rows")
    _buf(s, f"{name} scales", (rows // int(g), K // 32), _U8, q.device)
    return rows, K


def _opts(scale_rule, round, hadamard, sign_mask, seed) -> mx_quant_opts:
    return mx_quant_opts(int(scale_rule), int(round), int(hadamard), int(sign_mask) & 0xFFFFFFFF,
                         int(seed) & 0xFFFFFFFFFFFFFFFF)


def mx_quantize(x: torch.Tensor, axis: int = 1, scale_rule: int = MX_SCALE_FLOOR,
                round: int = MX_ROUND_RNE, hadamard: int = 0, sign_mask: int = 0, seed: int = 0,
                codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                stream=None):
    """1x32 quantize. axis=1 -> codes [rows][cols/2], scales [rows][cols/32];
    axis=0 -> codes [cols][rows/2], scales [cols][rows/32] (K-major layout of x^T)."""
    rows, cols, ld = _src(x)
    shape_c = (rows, cols // 2) if axis == 1 else (cols, rows // 2)
    shape_s = (rows, cols // 32) if axis == 1 else (cols, rows // 32)
    codes = _codes_out(codes, "codes", shape_c, x.device)
    scales = _codes_out(scales, "scales", shape_s, x.device)
    o = _opts(scale_rule, round, hadamard, sign_mask, seed)
    check(lib().mx_quantize(_ptr(x), _dtype_code(x), rows, cols, ld, int(axis), ctypes.byref(o),
                            _ptr(codes), _ptr(scales), _stream(stream)), "mx_quantize")
    return codes, scales


def mx_quantize_2d(x: torch.Tensor, scale_rule: int = MX_SCALE_CEIL, round: int = MX_ROUND_RNE,
                   seed: int = 0, transposed: bool = True, codes=None, scales=None, codes_t=None,
                   scales_t=None, stream=None):
    """32x32 quantize -> (codes [rows][cols/2], scales [rows/32][cols/32],
    codes_t [cols][rows/2], scales_t [cols/32][rows/32]); the last two are None unless
    transposed."""
    rows, cols, ld = _src(x)
    dev = x.device
    codes = _codes_out(codes, "codes", (rows, cols // 2), dev)
    scales = _codes_out(scales, "scales", (rows // 32, cols // 32), dev)
    if transposed:
        codes_t = _codes_out(codes_t, "codes_t", (cols, rows // 2), dev)
        scales_t = _codes_out(scales_t, "scales_t", (cols // 32, rows // 32), dev)
    else:
        codes_t = scales_t = None
    o = _opts(scale_rule, round, 0, 0, seed)
    check(lib().mx_quantize_2d(_ptr(x), _dtype_code(x), rows, cols, ld, ctypes.byref(o),
                               _ptr(codes), _ptr(scales), _ptr(codes_t), _ptr(scales_t),
                               _stream(stream)), "mx_quantize_2d")
    return codes, scales, codes_t, scales_t


def mx_dequantize(codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int,
                  block_rows: int = 1, inv_hadamard: int = 0, sign_mask: int = 0,
                  out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    if not isinstance(codes, torch.Tensor) or not codes.is_cuda:
        raise ValueError("codes must be a CUDA tensor")
    rows, cols, block_rows = int(rows), int(cols), int(block_rows)
    if block_rows not in (1, 32) or rows % block_rows:
        raise ValueError("block_rows must be 1 or 32 and divide rows")
    dev = codes.device
    _buf(codes, "codes", (rows, cols // 2), _U8, dev)
    _buf(scales, "scales", (rows // block_rows, cols // 32), _U8, dev)
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float32, device=dev)
    _buf(out, "out", (rows, cols), (torch.float32,), dev)
    check(lib().mx_dequantize(_ptr(codes), _ptr(scales), rows, cols, int(block_rows),
                              int(inv_hadamard), int(sign_mask) & 0xFFFFFFFF, _ptr(out),
                              _stream(stream)), "mx_dequantize")
    return out


def _out(out, rows, cols, out_dtype, device):
    if out is None:
        out = torch.empty((rows, cols), dtype=out_dtype, device=device)
    _buf(out, "out", (rows, cols), (torch.bfloat16, torch.float32), device, rows_only=True)
    code = MX_BF16 if out.dtype == torch.bfloat16 else MX_F32
    return out, code


def _gemm(name, aq, as_, ga, bq, bs, gb, alpha_exp, out_dtype, out, stream):
    M, K = _operand(aq, as_, ga, "A")
    N, Kb = _operand(bq, bs, gb, "B")
    if Kb != K or bq.device != aq.device:
        raise ValueError("operands disagree on the reduction length or the device")
    out, code = _out(out, M, N, out_dtype, aq.device)
    check(getattr(lib(), name)(_ptr(aq), _ptr(as_), int(ga), _ptr(bq), _ptr(bs), int(gb), M, N, K,
                               int(alpha_exp), code, _ptr(out), out.stride(0), _stream(stream)),
          name)
    return out


def mx_gemm_fprop(xq, xs, gx, wq, ws, gw, alpha_exp=0, out_dtype=torch.bfloat16, out=None,
                  stream=None):
    """Y[T][N] = 2^alpha sum_k X[t][k] W[n][k]; xq [T][K/2], wq [N][K/2]."""
    return _gemm("mx_gemm_fprop", xq, xs, gx, wq, ws, gw, alpha_exp, out_dtype, out, stream)


def mx_gemm_dgrad(dyq, dys, gdy, wtq, wts, gwt, alpha_exp=0, out_dtype=torch.bfloat16, out=None,
                  stream=None):
    """dX[T][K] = 2^alpha sum_n dY[t][n] Wt[k][n]; dyq [T][N/2], wtq [K][N/2]."""
    return _gemm("mx_gemm_dgrad", dyq, dys, gdy, wtq, wts, gwt, alpha_exp, out_dtype, out, stream)


def mx_gemm_wgrad(dytq, dyts, gdy, xtq, xts, gx, alpha_exp=0, out_dtype=torch.bfloat16, out=None,
                  stream=None):
    """dW[N][K] = 2^alpha sum_t dYt[n][t] Xt[k][t]; dytq [N][T/2], xtq [K][T/2]."""
    return _gemm("mx_gemm_wgrad", dytq, dyts, gdy, xtq, xts, gx, alpha_exp, out_dtype, out, stream)


def mx_gemm_fprop_quant(xq, xs, gx, wq, ws, gw, alpha_exp=0, scale_rule=MX_SCALE_FLOOR,
                        round=MX_ROUND_RNE, hadamard=0, sign_mask=0, seed=0, codes=None,
                        scales=None, stream=None):
    """Y = 2^alpha X W^T in fp32, quantized in the GEMM epilogue along its rows (1x32 blocks
    along N, options as for mx_quantize) -> (codes [T][N/2], scales [T][N/32])."""
    T, K = _operand(xq, xs, gx, "X")
    N, Kw = _operand(wq, ws, gw, "W")
    if Kw != K or wq.device != xq.device:
        raise ValueError("operands disagree on the reduction length or the device")
    codes = _codes_out(codes, "codes", (T, N // 2), xq.device)
    scales = _codes_out(scales, "scales", (T, N // 32), xq.device)
    o = _opts(scale_rule, round, hadamard, sign_mask, seed)
    check(lib().mx_gemm_fprop_quant(_ptr(xq), _ptr(xs), int(gx), _ptr(wq), _ptr(ws), int(gw), T, N,
                                    K, int(alpha_exp), ctypes.byref(o), _ptr(codes), _ptr(scales),
                                    _stream(stream)), "mx_gemm_fprop_quant")
    return codes, scales


def mx_quantize_mxfp8(x: torch.Tensor, fmt: int = MX_E4M3, axis: int = 1,
                      scale_rule: int = MX_SCALE_FLOOR, round: int = MX_ROUND_RNE,
                      hadamard: int = 0, sign_mask: int = 0, seed: int = 0,
                      codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                      stream=None):
    """1x32 MXFP8 quantize (fmt MX_E4M3 or MX_E5M2). axis=1 -> codes [rows][cols] (one byte per
    element), scales [rows][cols/32]; axis=0 -> codes [cols][rows], scales [cols][rows/32]."""
    rows, cols, ld = _src(x)
    shape_c = (rows, cols) if axis == 1 else (cols, rows)
    shape_s = (rows, cols // 32) if axis == 1 else (cols, rows // 32)
    codes = _codes_out(codes, "codes", shape_c, x.device)
    scales = _codes_out(scales, "scales", shape_s, x.device)
    o = _opts(scale_rule, round, hadamard, sign_mask, seed)
    check(lib().mx_quantize_mxfp8(_ptr(x), _dtype_code(x), rows, cols, ld, int(axis), int(fmt),
                                  ctypes.byref(o), _ptr(codes), _ptr(scales), _stream(stream)),
          "mx_quantize_mxfp8")
    return codes, scales


def mx_gemm_mxfp8(aq, as_, afmt, bq, bs, bfmt, alpha_exp=0, out_dtype=torch.bfloat16, out=None,
                  stream=None):
    """C[M][N] = 2^alpha sum_k A[m][k] B[n][k]; aq [M][K], bq [N][K] MXFP8 codes of formats
    afmt / bfmt, scales [M][K/32], [N][K/32]."""
    M, K = _operand(aq, as_, 1, "A", 1.0)
    N, Kb = _operand(bq, bs, 1, "B", 1.0)
    if Kb != K or bq.device != aq.device:
        raise ValueError("operands disagree on the reduction length or the device")
    out, code = _out(out, M, N, out_dtype, aq.device)
    check(lib().mx_gemm_mxfp8(_ptr(aq), _ptr(as_), int(afmt), _ptr(bq), _ptr(bs), int(bfmt), M, N,
                              K, int(alpha_exp), code, _ptr(out), out.stride(0), _stream(stream)),
          "mx_gemm_mxfp8")
    return out


def mx_quantize_2d_blocks(x: torch.Tensor, block: int = 32, scale_rule: int = MX_SCALE_CEIL,
                          round: int = MX_ROUND_RNE, seed: int = 0, transposed: bool = True,
                          codes=None, scales=None, codes_t=None, scales_t=None, stream=None):
    """BxB tiles (block 8, 32 or 64) -> (codes, scales, codes_t, scales_t); scales [rows/8]
    [cols/8] for 8, [rows/32][cols/32] for 32, [rows/64][cols/32] (GEMM layout) for 64; the
    transposed pair is None unless transposed."""
    rows, cols, ld = _src(x)
    dev = x.device
    B = int(block)
    shape_s = {8: (rows // 8, cols // 8), 32: (rows // 32, cols // 32), 64: (rows // 64, cols // 32)}
    shape_st = {8: (cols // 8, rows // 8), 32: (cols // 32, rows // 32), 64: (cols // 64, rows // 32)}
    if B not in shape_s:
        raise ValueError("block must be 8, 32 or 64")
    codes = _codes_out(codes, "codes", (rows, cols // 2), dev)
    scales = _codes_out(scales, "scales", shape_s[B], dev)
    if not transposed:
        codes_t = scales_t = None
    else:
        codes_t = _codes_out(codes_t, "codes_t", (cols, rows // 2), dev)
        scales_t = _codes_out(scales_t, "scales_t", shape_st[B], dev)
    o = _opts(scale_rule, round, 0, 0, seed)
    check(lib().mx_quantize_2d_blocks(_ptr(x), _dtype_code(x), rows, cols, ld, B, ctypes.byref(o),
                                      _ptr(codes), _ptr(scales), _ptr(codes_t), _ptr(scales_t),
                                      _stream(stream)), "mx_quantize_2d_blocks")
    return codes, scales, codes_t, scales_t


def mx_scale_mismatch_map(x: torch.Tensor, scale_rule: int = MX_SCALE_FLOOR, out=None,
                          stream=None) -> torch.Tensor:
    """int8 [rows][cols]: scale exponent of each element's 1x32 row block minus that of its 1x32
    column block (saturated; -128 for non-finite blocks)."""
    rows, cols, ld = _src(x)
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.int8, device=x.device)
    _buf(out, "out", (rows, cols), (torch.int8,), x.device)
    check(lib().mx_scale_mismatch_map(_ptr(x), _dtype_code(x), rows, cols, ld, int(scale_rule),
                                      _ptr(out), _stream(stream)), "mx_scale_mismatch_map")
    return out


# the current stream of a device as an address, without a Stream object (3 us on the host)
_current_raw_stream = torch._C._cuda_getCurrentRawStream


def _launch(name, device, stream, *args):
    """One library call on `stream` (None: the device's current stream), with the tensors' device
    current during the call."""
    raw = _current_raw_stream(device.index) if stream is None else stream.cuda_stream
    if device.index == torch.cuda.current_device():
        status = getattr(_lib.lib(), name)(*args, raw)
    else:
        with torch.cuda.device(device):
            status = getattr(_lib.lib(), name)(*args, raw)
    if status:
        check(status, name)


def _rows(t, name: str):
    """A 2-D CUDA tensor of bf16 or fp32 with contiguous rows; returns (rows, cols, ld). The
    stride of a single row says nothing, so its leading dimension is its length."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _CODE:
        raise TypeError(f"{name} must be bfloat16 or float32")
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{name} must be a 2-D CUDA tensor with contiguous rows")
    rows, cols = t.shape
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name} must be a 2-D CUDA tensor with contiguous rows")
    return rows, cols, ld if rows > 1 else cols


def _rows_like(t, name: str, x):
    """Another [rows][cols] operand of x's shape, type and device; returns its ld."""
    if (isinstance(t, torch.Tensor) and t.dtype is x.dtype and t.shape == x.shape
            and t.device == x.device and t.is_contiguous()):
        return t.shape[1]
    rows, cols, ld = _rows(t, name)
    if (rows, cols) != tuple(x.shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(x.shape)}")
    if t.dtype != x.dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {x.dtype}")
    if t.device != x.device:
        raise ValueError(f"{name} is on {t.device}, expected {x.device}")
    return ld


def _scratch(size: int, device, stream):
    """size bytes from the pool of the stream that uses them: what is allocated there next comes
    after that use."""
    if stream is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=torch.uint8, device=device)


def _workspace(t, device) -> int:
    """Bytes of a caller's workspace, after the checks of _buf."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    _buf(t, "workspace", (t.numel(),), _U8, device)
    return t.numel()


def _data(t):
    return None if t is None else t.data_ptr()


_CODE = {torch.bfloat16: MX_BF16, torch.float32: MX_F32}
_FLOATS = (torch.bfloat16, torch.float32)
_F32 = (torch.float32,)


def _norm_args(x, gamma, residual, eps, sum, y, with_y, rstd):
    """Checks the norm's tensors and allocates the outputs that are not given; returns the leading
    arguments of the C calls and (y, s, rstd)."""
    rows, cols, ldx = _rows(x, "x")
    dev = x.device
    _buf(gamma, "gamma", (cols,), _FLOATS, dev)
    ldr = lds = ldy = 0
    s = x
    if residual is not None:
        ldr = _rows_like(residual, "residual", x)
        if sum is None:
            sum, lds = torch.empty(rows, cols, dtype=x.dtype, device=dev), cols
        else:
            lds = _rows_like(sum, "sum", x)
        s = sum
    elif sum is not None:
        lds = _rows_like(sum, "sum", x)
    if y is not None:
        ldy = _rows_like(y, "y", x)
    elif with_y:
        y, ldy = torch.empty(rows, cols, dtype=x.dtype, device=dev), cols
    if rstd is None:
        rstd = torch.empty(rows, dtype=torch.float32, device=dev)
    else:
        _buf(rstd, "rstd", (rows,), _F32, dev)
    args = (x.data_ptr(), ldx, _data(residual), ldr, _CODE[x.dtype], rows, cols, gamma.data_ptr(),
            _CODE[gamma.dtype], eps, _data(sum), lds, _data(y), ldy, rstd.data_ptr())
    return args, (y, s, rstd)


def mx_rmsnorm(x, gamma, residual=None, eps: float = 1e-5, sum=None, y=None, rstd=None,
               stream=None):
    """RMS norm of s = x + residual by rows: y = s / sqrt(mean(s^2) + eps) * gamma.
    x, residual [rows][cols] bf16 or fp32 (cols a multiple of 32, at most 32768), gamma [cols]
    bf16 or fp32 -> (y, s, rstd [rows] fp32); s is x itself without a residual."""
    args, out = _norm_args(x, gamma, residual, eps, sum, y, True, rstd)
    _launch("mx_rmsnorm", x.device, stream, *args)
    return out


def _norm_quant(name, fmt, width, x, gamma, residual, eps, o, with_y, codes, scales, sum, y, rstd,
                stream):
    args, out = _norm_args(x, gamma, residual, eps, sum, y, with_y, rstd)
    rows, cols, dev = args[5], args[6], x.device
    if codes is None:
        codes = torch.empty(rows, cols // width, dtype=torch.uint8, device=dev)
    else:
        _buf(codes, "codes", (rows, cols // width), _U8, dev)
    if scales is None:
        scales = torch.empty(rows, cols // 32, dtype=torch.uint8, device=dev)
    else:
        _buf(scales, "scales", (rows, cols // 32), _U8, dev)
    _launch(name, dev, stream, *args, *fmt, ctypes.byref(o), codes.data_ptr(), scales.data_ptr())
    return (codes, scales) + out


def mx_rmsnorm_quant(x, gamma, residual=None, eps: float = 1e-5, scale_rule: int = MX_SCALE_FLOOR,
                     round: int = MX_ROUND_RNE, hadamard: int = 0, sign_mask: int = 0,
                     seed: int = 0, with_y: bool = False, codes=None, scales=None, sum=None,
                     y=None, rstd=None, stream=None):
    """mx_rmsnorm with its result in MXFP4, 1x32 blocks along the row -> (codes [rows][cols/2],
    scales [rows][cols/32], y or None, s, rstd). y is written with with_y or when a buffer is
    given."""
    return _norm_quant("mx_rmsnorm_quant", (), 2, x, gamma, residual, eps,
                       _opts(scale_rule, round, hadamard, sign_mask, seed), with_y, codes, scales,
                       sum, y, rstd, stream)


def mx_rmsnorm_quant_mxfp8(x, gamma, residual=None, eps: float = 1e-5, fmt: int = MX_E4M3,
                           scale_rule: int = MX_SCALE_FLOOR, round: int = MX_ROUND_RNE,
                           hadamard: int = 0, sign_mask: int = 0, seed: int = 0,
                           with_y: bool = False, codes=None, scales=None, sum=None, y=None,
                           rstd=None, stream=None):
    """mx_rmsnorm with its result in MXFP8 (fmt MX_E4M3 or MX_E5M2), 1x32 blocks along the row ->
    (codes [rows][cols], scales [rows][cols/32], y or None, s, rstd)."""
    return _norm_quant("mx_rmsnorm_quant_mxfp8", (int(fmt),), 1, x, gamma, residual, eps,
                       _opts(scale_rule, round, hadamard, sign_mask, seed), with_y, codes, scales,
                       sum, y, rstd, stream)


def mx_rmsnorm_backward(dy, s, gamma, rstd, dsum=None, with_dgamma: bool = True, dx=None,
                        dgamma=None, workspace=None, stream=None):
    """Gradients of mx_rmsnorm from dy, the stored sum s, rstd and (optionally) the gradient dsum
    that reaches the sum from further on -> (dx, of x and of residual alike; dgamma [cols] fp32,
    None without with_dgamma). workspace: a uint8 buffer of at least
    lib().mx_rmsnorm_backward_workspace(rows, cols) bytes, allocated per call when None."""
    rows, cols, lds = _rows(s, "s")
    dev = s.device
    lddy = _rows_like(dy, "dy", s)
    ldds = 0 if dsum is None else _rows_like(dsum, "dsum", s)
    _buf(gamma, "gamma", (cols,), _FLOATS, dev)
    _buf(rstd, "rstd", (rows,), _F32, dev)
    if dx is None:
        dx, lddx = torch.empty(rows, cols, dtype=s.dtype, device=dev), cols
    else:
        lddx = _rows_like(dx, "dx", s)
    size = 0
    if with_dgamma:
        if dgamma is None:
            dgamma = torch.empty(cols, dtype=torch.float32, device=dev)
        else:
            _buf(dgamma, "dgamma", (cols,), _F32, dev)
        if workspace is not None:
            size = _workspace(workspace, dev)
        else:
            size = lib().mx_rmsnorm_backward_workspace(rows, cols)
            if size:  # small tensors want none
                workspace = _scratch(size, dev, stream)
    else:
        dgamma = workspace = None
    _launch("mx_rmsnorm_backward", dev, stream, dy.data_ptr(), lddy, _data(dsum), ldds,
            s.data_ptr(), lds, _CODE[s.dtype], rows, cols, gamma.data_ptr(), _CODE[gamma.dtype],
            rstd.data_ptr(), dx.data_ptr(), lddx, _data(dgamma), _data(workspace), size)
    return dx, dgamma


def mx_gemv(x, wq, ws, gw: int = 1, hadamard: int = 0, sign_mask: int = 0, alpha_exp: int = 0,
            out_dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """y[T][N] = 2^alpha x W^T for a few tokens x [T][K] (bf16 or fp32, not quantized) and MXFP4
    weights wq [N][K/2], ws [N/gw][K/32]; hadamard = 1 rotates x as mx_quantize does (for weights
    quantized rotated, with alpha_exp = -5). workspace: a uint8 buffer of at least
    lib().mx_gemv_workspace(...) bytes, allocated per call when None and wanted."""
    T, K, ldx = _rows(x, "x")
    N, Kw = _operand(wq, ws, gw, "W")
    dev = x.device
    if Kw != K or wq.device != dev:
        raise ValueError("operands disagree on the reduction length or the device")
    if out is None and out_dtype in _CODE:
        out, code, ldy = torch.empty(T, N, dtype=out_dtype, device=dev), _CODE[out_dtype], N
    else:
        out, code = _out(out, T, N, out_dtype, dev)
        ldy = out.stride(0) if T > 1 else N
    dtype, size = _CODE[x.dtype], 0
    if workspace is not None:
        size = _workspace(workspace, dev)
    elif T > 1:  # one token wants none
        size = lib().mx_gemv_workspace(dtype, T, N, K, hadamard, code)
        if size:
            workspace = _scratch(size, dev, stream)
    _launch("mx_gemv", dev, stream, x.data_ptr(), dtype, ldx, wq.data_ptr(), ws.data_ptr(), gw, T,
            N, K, hadamard, sign_mask & 0xFFFFFFFF, alpha_exp, code, out.data_ptr(), ldy,
            _data(workspace), size)
    return out


_I32 = (torch.int32,)
# mx_cache and mx_rows of mx.h as bytes: a third of the time that ctypes structures take
_pack_cache = struct.Struct("@7P3q4i").pack
_pack_rows = struct.Struct("@P2q").pack


def _cache(kq, ks, vq, vs, pages, lengths, offsets, T, fmt):
    """Checks a cache and the tables of a call with T rows; returns its C view, its heads and dim and
    the device's index."""
    u8, i32 = torch.uint8, torch.int32
    try:
        n, H, P, D = kq.shape
        B, width = pages.shape
        at, block = kq.get_device(), (n, H, P >> 5)
        good = (kq.dtype is u8 and ks.dtype is u8 and vq.dtype is u8 and vs.dtype is u8
                and pages.dtype is i32 and lengths.dtype is i32 and P & 31 == 0
                and ks.shape == block and vs.shape == block and vq.shape == block + (D, 32)
                and lengths.shape == (B,) and at >= 0 and ks.get_device() == at
                and vq.get_device() == at and vs.get_device() == at and pages.get_device() == at
                and lengths.get_device() == at and kq.is_contiguous() and ks.is_contiguous()
                and vq.is_contiguous() and vs.is_contiguous() and pages.is_contiguous()
                and lengths.is_contiguous())
        if offsets is None:
            good, table = good and T == B, 0
        else:
            good = (good and offsets.dtype is i32 and offsets.shape == (B + 1,)
                    and offsets.get_device() == at and offsets.is_contiguous())
            table = offsets.data_ptr()
    except (AttributeError, TypeError, ValueError):
        good = False
    if not good:
        _cache_refusal(kq, ks, vq, vs, pages, lengths, offsets, T)
    return _pack_cache(kq.data_ptr(), ks.data_ptr(), vq.data_ptr(), vs.data_ptr(),
                       pages.data_ptr(), lengths.data_ptr(), table, n, B, width, H, D, P,
                       fmt), H, D, at


def _cache_refusal(kq, ks, vq, vs, pages, lengths, offsets, T):
    """Says what is wrong with a cache and its tables."""
    if not isinstance(kq, torch.Tensor) or kq.dim() != 4 or not kq.is_cuda:
        raise ValueError("kq must be a CUDA tensor [pages][heads][page][dim]")
    n, H, P, D = kq.shape
    dev = kq.device
    if P % 32:
        raise ValueError("a page holds a multiple of 32 tokens")
    _buf(kq, "kq", (n, H, P, D), _U8, dev)
    _buf(vq, "vq", (n, H, P // 32, D, 32), _U8, dev)
    _buf(ks, "ks", (n, H, P // 32), _U8, dev)
    _buf(vs, "vs", (n, H, P // 32), _U8, dev)
    if not isinstance(pages, torch.Tensor) or pages.dim() != 2:
        raise ValueError("pages must be a tensor [sequences][pages]")
    B, width = pages.shape
    _buf(pages, "pages", (B, width), _I32, dev)
    _buf(lengths, "lengths", (B,), _I32, dev)
    if offsets is not None:
        _buf(offsets, "offsets", (B + 1,), _I32, dev)
    raise ValueError(f"{T} rows for {B} sequences: offsets say which are whose")


def _heads(t, name: str, heads, dim, at, like=None):
    """A [T][heads][dim] tensor of bf16 or fp32 on device `at` with contiguous channels (like: of that
    one's shape and type); returns its C view."""
    try:
        _, n, d = t.shape
        token, head, one = t.stride()
        if (t.dtype in _CODE and d == dim and one == 1 and t.get_device() == at
                and (n == heads if like is None else t.shape == like.shape and t.dtype is like.dtype)):
            return _pack_rows(t.data_ptr(), token, head)
    except (AttributeError, TypeError, ValueError):
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _CODE:
        raise TypeError(f"{name} must be bfloat16 or float32")
    if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name} must be [tokens][heads][dim] with contiguous channels")
    if like is not None and t.dtype != like.dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {like.dtype}")
    want = ("T", heads, dim) if like is None else tuple(like.shape)
    if t.shape[2] != dim or t.shape[1] != want[1] or (like is not None and tuple(t.shape) != want):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {want}")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{at}")


def _row_count(t, name):
    try:
        T, heads, _ = t.shape
        return T, heads
    except (AttributeError, TypeError, ValueError):
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    raise ValueError(f"{name} must be [tokens][heads][dim]")


_current_device = torch._C._cuda_getDevice


def _call(function, at, stream, *args):
    """_launch for a device's index and a function of the library."""
    raw = _current_raw_stream(at) if stream is None else stream.cuda_stream
    if at == _current_device():
        status = function(*args, raw)
    else:
        with torch.cuda.device(at):
            status = function(*args, raw)
    if status:
        check(status, function.__name__)


def mx_cache_write(k, v, kq, ks, vq, vs, pages, lengths, offsets=None, fmt: int = MX_E4M3,
                   scale_rule: int = MX_SCALE_FLOOR, stream=None) -> None:
    """Quantizes keys and values [T][heads][dim] (bf16 or fp32, any distance of tokens and heads) into
    a cache: kq [pages][heads][page][dim], vq [pages][heads][page / 32][dim][32] codes, ks, vs
    [pages][heads][page / 32] scales, all uint8. pages [B][..] int32 is the page table, lengths [B]
    int32 counts the sequences' tokens with these; rows offsets[b] .. offsets[b + 1] (int32, [B + 1])
    are the newest of sequence b, without offsets row b is. A block of 32 tokens whose scale has to
    grow rounds its older codes again; it keeps that scale when the tokens that needed it are written
    over (refused drafts), unless it is written from its first slot on."""
    T = _row_count(k, "k")[0]
    c, H, D, at = _cache(kq, ks, vq, vs, pages, lengths, offsets, T, fmt)
    rk = _heads(k, "k", H, D, at)
    rv = _heads(v, "v", H, D, at, k)
    _call(_lib.lib().mx_cache_write, at, stream, rk, rv, _CODE[k.dtype], T, c, scale_rule)


def mx_cache_read(kq, ks, vq, vs, pages, lengths, offsets=None, rows=None, fmt: int = MX_E4M3,
                  out_dtype=torch.bfloat16, k=None, v=None, stream=None):
    """Keys and values of the sequences' newest tokens back from a cache (as for mx_cache_write) ->
    (k, v), [rows][heads][dim] of out_dtype. rows: how many there are, offsets[B] (without offsets one
    for each sequence); rows of no sequence are left as they are, rows without a token are zeros."""
    if k is None and rows is None:
        if offsets is not None:
            raise ValueError("with offsets, rows (or k and v) says how many rows there are")
        rows = lengths.shape[0] if isinstance(lengths, torch.Tensor) and lengths.dim() == 1 else 0
    T = rows if k is None else _row_count(k, "k")[0]
    c, H, D, at = _cache(kq, ks, vq, vs, pages, lengths, offsets, T, fmt)
    if k is None and v is None:
        if out_dtype not in _CODE:
            raise TypeError("out_dtype must be bfloat16 or float32")
        k = torch.empty((T, H, D), dtype=out_dtype, device=kq.device)
        v = torch.empty_like(k)
    elif k is None or v is None:
        raise ValueError("k and v are given together")
    rk, rv = _heads(k, "k", H, D, at), _heads(v, "v", H, D, at, k)
    _call(_lib.lib().mx_cache_read, at, stream, rk, rv, _CODE[k.dtype], T, c)
    return k, v


def mx_cache_attention(q, kq, ks, vq, vs, pages, lengths, offsets=None, scale=None,
                       fmt: int = MX_E4M3, out=None, lse=None, with_lse: bool = False,
                       workspace=None, stream=None):
    """Causal attention of each sequence's newest tokens over its cache (as for mx_cache_write): q
    [T][query heads][dim] bf16 or fp32, query head h over head h / (query heads / heads) of the cache,
    each row over the tokens up to its own -> out of q's shape and type, or (out, lse [T][query heads]
    fp32) with with_lse or an lse buffer. Prompts and single tokens are faster in calls of their own.
    scale: dim ** -0.5 when None. workspace: a uint8 buffer of at
    least lib().mx_cache_attention_workspace(...) bytes, allocated per call when None."""
    T, heads = _row_count(q, "q")
    c, _, D, at = _cache(kq, ks, vq, vs, pages, lengths, offsets, T, fmt)
    rq = _heads(q, "q", heads, D, at)
    dev = kq.device
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    ro = _heads(out, "out", heads, D, at, q)
    if lse is not None:
        _buf(lse, "lse", (T, heads), _F32, dev)
    elif with_lse:
        lse = torch.empty((T, heads), dtype=torch.float32, device=dev)
    L = _lib.lib()
    if workspace is not None:
        size = _workspace(workspace, dev)
    else:
        size = L.mx_cache_attention_workspace(T, heads, c)
        if size > 0:
            workspace = _scratch(size, dev, stream)
    _call(L.mx_cache_attention, at, stream, rq, ro, _data(lse), _CODE[q.dtype], T, heads,
          D ** -0.5 if scale is None else scale, c, _data(workspace), size)
    return out if lse is None else (out, lse)


def mx_lora(x, a, b, index, base=None, scaling=None, out_dtype=None, out=None, workspace=None,
            stream=None):
    """out[t] = base[t] + scaling[e] b[e] (a[e] x[t]) with e = index[t], each token's own adapter: x
    [T][K], a [E][rank][K], b [E][N][rank] bf16 or fp32 of one type (K and rank multiples of 8, rank
    at most 128), index [T] int32 (outside [0, E): base alone), base [T][N] bf16 or fp32 or None
    (zeros), scaling [E] fp32 or None (ones) -> out [T][N] of out_dtype (base's type when None, x's
    without a base). out may be base itself. workspace: a uint8 buffer of at least
    lib().mx_lora_workspace(...) bytes, allocated per call when None and wanted."""
    try:
        T, K = x.shape
        E, rank, _ = a.shape
        N, at, dtype = b.shape[1], x.get_device(), x.dtype
        ldx, one = x.stride()
        good = (dtype in _CODE and at >= 0 and (one == 1 or K <= 1) and a.dtype is dtype
                and b.dtype is dtype and a.shape == (E, rank, K) and b.shape == (E, N, rank)
                and a.get_device() == at and b.get_device() == at and a.is_contiguous()
                and b.is_contiguous() and index.dtype is torch.int32 and index.shape == (T,)
                and index.get_device() == at and index.is_contiguous()
                and (scaling is None or scaling.dtype is torch.float32 and scaling.shape == (E,)
                     and scaling.get_device() == at and scaling.is_contiguous())
                and (base is None or base.dtype in _CODE and base.shape == (T, N)
                     and base.get_device() == at and (base.stride(1) == 1 or N <= 1)))
    except (AttributeError, IndexError, TypeError, ValueError):
        good = False
    if not good:
        _lora_refusal(x, a, b, index, base, scaling)
    base_code = ldb = 0
    if base is not None:
        base_code, ldb = _CODE[base.dtype], base.stride(0) if T > 1 else N
    if out is None:
        if out_dtype is None:
            out_dtype = dtype if base is None else base.dtype
        if out_dtype not in _CODE:
            raise TypeError("out_dtype must be bfloat16 or float32")
        out, code, ldo = torch.empty((T, N), dtype=out_dtype, device=x.device), _CODE[out_dtype], N
    else:
        out, code = _out(out, T, N, out_dtype, x.device)
        ldo = out.stride(0) if T > 1 else N
    L = _lib.lib()
    if workspace is not None:
        size = _workspace(workspace, x.device)
    else:
        size = L.mx_lora_workspace(_CODE[dtype], T, N, K, E, rank)
        if size:
            workspace = _scratch(size, x.device, stream)
    _call(L.mx_lora, at, stream, x.data_ptr(), _CODE[dtype], ldx if T > 1 and K else K, a.data_ptr(),
          b.data_ptr(), E, rank, index.data_ptr(), _data(scaling), _data(base), base_code, ldb, T, N,
          K, code, out.data_ptr(), ldo, _data(workspace), size)
    return out


def _lora_refusal(x, a, b, index, base, scaling):
    """Says what is wrong with the operands of mx_lora."""
    T, K, _ = _rows(x, "x")
    dev, same = x.device, (x.dtype,)
    for t, name in ((a, "a"), (b, "b")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != 3:
            raise ValueError(f"{name} must have three dimensions")
    E, rank, N = a.shape[0], a.shape[1], b.shape[1]
    _buf(a, "a", (E, rank, K), same, dev)
    _buf(b, "b", (E, N, rank), same, dev)
    _buf(index, "index", (T,), _I32, dev)
    if scaling is not None:
        _buf(scaling, "scaling", (E,), _F32, dev)
    rows, cols, _ = _rows(base, "base")
    if (rows, cols) != (T, N):
        raise ValueError(f"base has shape {tuple(base.shape)}, expected {(T, N)}")
    raise ValueError(f"base is on {base.device}, expected {dev}")
