"""Norm and projection with all their gradients in 8 bits, as a training step runs
them: the projection's weight gradient takes the norm's result in blocks along the
tokens, formed again from h."""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
from f8_ref import E5M2, f64
from gpu_util import DEV, say
from test_f8_scaled import BF16, F16, F32, randn

pytestmark = pytest.mark.gpu
EPS = 1e-6


def step(x, residual, weight, w, dy, dh):
    """(y, h, dx, dweight, dw) of y = norm(x + residual) . w^T."""
    a, sa, h = g.rms_norm_f8(x, weight, EPS, residual=residual)
    y = g.gemm_f8_scaled(a, sa, *g.quantize_f8(w, 128), dtype=x.dtype)
    da = g.gemm_f8_scaled(*g.quantize_f8(dy, dtype=E5M2), *g.quantize_f8(w.t(), 128), dtype=x.dtype)
    dx, dweight = g.rms_norm_backward(da, h, weight, EPS, dh=dh)
    v = h.float()
    n = (v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS) * weight.float()).to(h.dtype)
    dw = g.gemm_f8_scaled(*g.quantize_f8(dy.t(), dtype=E5M2), *g.quantize_f8(n.t()), dtype=F32)
    return y, h, dx, dweight, dw


def off(got, want, most):
    d = np.linalg.norm(f64(got) - want)
    assert d <= most, (d, most)


@pytest.mark.parametrize("T,K,N", [(1, 256, 130), (70, 515, 300), (300, 640, 260), (1030, 1024, 512)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_training_step(T, K, N, dtype):
    say(f"layer {T}x{K}x{N} {dtype}")
    x, r = randn(T, K, dtype=dtype, seed=1), randn(T, K, dtype=dtype, seed=2)
    weight, w = 1 + 0.2 * randn(K, dtype=F32, seed=3), randn(N, K, dtype=dtype, seed=4, scale=K ** -0.5)
    dy, dh = randn(T, N, dtype=dtype, seed=5, scale=0.1), randn(T, K, dtype=dtype, seed=6, scale=0.1)
    y, h, dx, dweight, dw = step(x, r, weight, w, dy, dh)
    H, W, G, D, DH = f64(h), f64(w), f64(weight), f64(dy), f64(dh)
    s = 1 / np.sqrt((H * H).mean(axis=1, keepdims=True) + EPS)
    n = H * s * G
    # A product's factors are off by half a step each, 2^-4 of an element in E4M3 and 2^-3 in
    # E5M2, to either side by chance, so that the squares of the terms add up; results and
    # the 16-bit norm add a half step of 2^-8 at most.
    size = lambda p, q: np.linalg.norm(np.sqrt((p * p) @ (q * q)))
    off(y, n @ W.T, (2 * 2.0 ** -4 + 2.0 ** -7) * size(n, W.T))
    off(dw, D.T @ n, (2.0 ** -4 + 2.0 ** -3 + 2.0 ** -7) * size(D.T, n))
    # dx and dweight are linear in dy w: dx takes an error of it to at most s |weight| times
    # itself (the part along h only shrinks), dweight to at most sqrt(T) max |h s| times
    da = D @ W
    e = (2.0 ** -4 + 2.0 ** -3 + 2.0 ** -7) * size(D, W)
    q = da * G
    want = s * (q - H * s * s * (q * H).mean(axis=1, keepdims=True)) + DH
    off(dx, want, e * np.max(s * np.abs(G)) + 2.0 ** -8 * np.linalg.norm(want))
    off(dweight, (da * H * s).sum(axis=0), e * np.sqrt(T) * np.max(np.abs(H * s)) + 1e-5 * np.linalg.norm(da))
