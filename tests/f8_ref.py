"""8-bit floating point with a scale per block of 128, the norm and its gradients
from their definitions, in 64 bits on the CPU."""
import numpy as np
import torch

U = 2.0 ** -23     # a whole fp32 step per sum: whatever the matrix core's own rounding is
LARGEST = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}
GRID = {torch.float8_e4m3fn: (3, -6), torch.float8_e5m2: (2, -14)}    # fraction bits, least normal exponent
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def blocks(n):
    return -(-n // 128)


def round8(v, dtype):
    """v to the nearest 8-bit value, ties to even, saturating (float64 numpy)."""
    bits, least = GRID[dtype]
    v = np.clip(v, -LARGEST[dtype], LARGEST[dtype])
    e = np.maximum(np.frexp(v)[1] - 1, least) - bits
    return np.ldexp(np.rint(np.ldexp(v, -e)), e)


def spread(scales, R, K, block_rows):
    """A scale per element."""
    return np.repeat(np.repeat(scales, block_rows, axis=0)[:R], 128, axis=1)[:, :K]


def quotients(x, block_rows, dtype):
    """(quotients that are rounded to 8 bits, scales in float32) of x [R, K]
    float64; blocks with a non-finite element give NaN scales and zeros."""
    R, K = x.shape
    L = LARGEST[dtype]
    p = np.zeros((-(-R // block_rows) * block_rows, blocks(K) * 128))
    p[:R, :K] = x
    b = p.reshape(-1, block_rows, blocks(K), 128)
    m = np.abs(b).max(axis=(1, 3))                       # NaN stays NaN
    bad = ~np.isfinite(m)
    mm = np.maximum(np.where(bad, 1.0, m), L * 2.0 ** -126)
    full = spread(mm, R, K, block_rows)
    q = np.where(spread(bad, R, K, block_rows), 0.0, np.nan_to_num(x, nan=0.0, posinf=0.0, neginf=0.0) * L / full)
    s = (mm.astype(np.float32) / np.float32(L)).astype(np.float64)
    s[bad] = np.nan
    return q, s


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy() if t.dtype not in LARGEST else \
        t.detach().cpu().to(torch.float32).double().numpy()


def values(data, scales):
    """8-bit elements times their scales, float64."""
    v, s = f64(data), f64(scales)
    R, K = v.shape
    return v * spread(s, R, K, 1 if s.shape[0] == R else 128)


def product(a, sa, b, sb, dtype):
    """(C, tolerance) of gemm_f8_scaled: fp32 sums over K products and the
    blocks' scaled sums (two roundings of the scale, one of the sum); for a 16-bit
    C each 8 consecutive products cut at 2^-13 of their largest, so that seven of
    them are off by that much at most; the output's half step."""
    x, y = values(a, sa), values(b, sb)
    c, mag = x @ y.T, np.abs(x) @ np.abs(y).T
    tol = (a.shape[1] + 4 * blocks(a.shape[1]) + 8) * U * mag
    if dtype != torch.float32:
        for k in range(0, a.shape[1], 8):
            xs, ys = np.abs(x[:, k:k + 8]), np.abs(y[:, k:k + 8])
            top = np.zeros_like(c)
            for i in range(xs.shape[1]):
                np.maximum(top, np.outer(xs[:, i], ys[:, i]), out=top)
            tol += 7 * 2.0 ** -13 * top
    return c, tol + half_step(np.abs(c) + tol, dtype)


def half_step(v, dtype):
    f = torch.finfo(dtype)
    return v * (f.eps / 2) + f.tiny * f.eps / 2


def assert_near(got, want, tol, what=""):
    d = np.abs(f64(got) - want)
    bad = ~(d <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(np.where(np.isnan(d), np.inf, d - tol))}"


def norm(x, residual, w, eps):
    """(h rounded to x's dtype, y float64, relative error that fp32 leaves y)."""
    h = x.cpu()
    if residual is not None:
        h = (h.float() + residual.cpu().float()).to(x.dtype)
    v = f64(h)
    K = v.shape[1]
    r = 1 / np.sqrt((v * v).sum(axis=1, keepdims=True) / K + eps)
    # the sum of K squares, each addition half a step, goes into r by half; a
    # few more roundings of r and of y, some of them whole steps
    return h, v * r * f64(w), (K / 2 + 16) * 2.0 ** -24


def norm_grad(dy, h, w, eps, dh):
    """(dx, tolerance, dw, tolerance) but for the outputs' rounding."""
    y, v, wt = f64(dy), f64(h), f64(w)
    R, K = v.shape
    r = 1 / np.sqrt((v * v).sum(axis=1, keepdims=True) / K + eps)
    g = y * wt
    c, mag = (g * v).sum(axis=1, keepdims=True), (np.abs(g) * np.abs(v)).sum(axis=1, keepdims=True)
    dx = r * (g - v * r * r * c / K)
    e = (K + 32) * 2.0 ** -24
    tol = 2 * e * r * (np.abs(g) + np.abs(v) * r * r * mag / K)
    if dh is not None:
        dx = dx + f64(dh)
        tol = tol + 2.0 ** -23 * (np.abs(f64(dh)) + np.abs(dx))
    dw = (y * v * r).sum(axis=0)
    return dx, tol, dw, (R + K + 32) * 2.0 ** -24 * (np.abs(y) * np.abs(v) * r).sum(axis=0)
