"""float64 definitions of the norm and its gradients, for the tests of the HIP kernels."""
import numpy as np
import torch

EPS32 = 2.0 ** -24  # half a step of fp32


def stored_sum(x: torch.Tensor, residual) -> torch.Tensor:
    """x + residual, rounded to their type (one fp32 addition)."""
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def norm_f64(s: torch.Tensor, gamma: torch.Tensor, eps: float):
    """(y, rho) of the stored sum s, float64."""
    s = s.detach().cpu().double().numpy()
    g = gamma.detach().cpu().double().numpy()
    with np.errstate(all="ignore"):
        rho = 1.0 / np.sqrt((s * s).sum(1) / s.shape[1] + np.float64(np.float32(eps)))
        return s * rho[:, None] * g, rho


def hadamard_f64(y: np.ndarray, sign_mask: int) -> np.ndarray:
    """Signs, then the unnormalised 32-point transform of every block, float64."""
    i = np.arange(32)
    H = np.array([[(-1.0) ** bin(a & b).count("1") for a in i] for b in i])
    d = np.array([-1.0 if (sign_mask >> j) & 1 else 1.0 for j in i])
    return ((y.reshape(-1, 32) * d) @ H).reshape(y.shape)


def odd_f32(y: np.ndarray) -> np.ndarray:
    """float64 -> float32 toward zero, the last bit set when bits were dropped: a rounding of the
    result to 22 bits or fewer is the rounding of y."""
    y = np.ascontiguousarray(y, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        h = y.astype(np.float32)
    b = h.view(np.uint32).copy()
    fin = np.isfinite(h)
    d = h.astype(np.float64)
    b[fin & (np.abs(d) > np.abs(y))] -= 1
    b[fin & (d != y)] |= 1
    return b.view(np.float32)


def backward_f64(dy, s, gamma, rstd, dsum):
    """(dx, bound on fp32's error in dx, dgamma, sum |dy z|) in float64. The bound counts half
    steps: u, z and the products one each; the mean is a sum of at most 32 terms in a thread, 6
    lane steps and 16 waves, each addend with 3 roundings, so 64 of them on mean |u z|; the last
    operations 2 on the result."""
    f = lambda t: t.detach().cpu().double().numpy()  # noqa: E731
    dy, s, g, r = f(dy), f(s), f(gamma), f(rstd)[:, None]
    u, z = dy * g, s * r
    n = s.shape[1]
    c = (u * z).sum(1, keepdims=True) / n
    cabs = np.abs(u * z).sum(1, keepdims=True) / n
    dx = r * (u - z * c)
    bound = EPS32 * r * (4 * np.abs(u) + np.abs(z) * (6 * np.abs(c) + 64 * cabs))
    if dsum is not None:
        dx = dx + f(dsum)
    bound += 2 * EPS32 * np.abs(dx)
    return dx, bound, (dy * z).sum(0), np.abs(dy * z).sum(0)
