"""Activations silu(g) u of a mixture-of-experts layer over a range of
magnitudes: the definition is a real number at any of them, so the layer has
to hold as many significant bits of a small or a large one as of one near 1."""
import math

import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
import moe_ref
import mx4_ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -23     # a whole fp32 step per operation
# What the layer keeps of an activation: two bfloat16 parts, each rounded to
# nearest, so at most 2^-8 of 2^-8 of it is lost.
PARTS = 2.0 ** -16


def layer64(x, p, up, down, eps, tiny):
    """y and its tolerance for one expert per token (weight p): x [T, H], up
    [2I, H], down [H, I], float64.  No absolute term but the formats' least
    steps: everything scales with the activations."""
    I = down.shape[1]
    z, absz = x @ up.T, np.abs(x) @ np.abs(up).T
    dz = (x.shape[1] + 8) * U * absz
    gate, u, dg, du = z[:, :I], z[:, I:], dz[:, :I], dz[:, I:]
    with np.errstate(over="ignore"):
        s = gate / (1 + np.exp(-gate))
    a = s * u
    # silu' below 1.1; exp, the division and the product take a few fp32 steps,
    # and exp's argument is off by dg, which 1.1 dg counts
    da = 1.1 * dg * np.abs(u) + np.abs(s) * du + 1.1 * dg * du + (PARTS + 8 * U) * np.abs(a)
    y = p * (a @ down.T)
    # two parts of an activation times at most two of a weight: sums of up to 4 I terms
    mag = (np.abs(a) + da) @ np.abs(down).T
    tol = p * (da @ np.abs(down).T) + (4 * I + 32) * U * p * mag
    return y, tol + (np.abs(y) + tol) * (eps / 2) + tiny / 2


def run(T, E, H, I, dtype, weights, scale_up, scale_down, seed, k=1):
    rng = np.random.default_rng(seed % 1000)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(dtype)
    if weights == "16":
        up = torch.from_numpy(rng.standard_normal((E, 2 * I, H)) * (H ** -0.5 * scale_up)).to(dtype)
        down = torch.from_numpy(rng.standard_normal((E, H, I)) * (I ** -0.5 * scale_down)).to(dtype)
        up64, down64, du, dd = up.double().numpy(), down.double().numpy(), up.to(DEV), down.to(DEV)
    else:
        def make(n, kk, scale):
            lo = 120 + round(math.log2(scale))
            d, s = mx4_ref.random_codes(rng, E * n, kk, lo, lo + 3)
            q = g.MX4(torch.from_numpy(d).to(DEV).view(E, n, -1), torch.from_numpy(s).to(DEV).view(E, n, -1), kk)
            return q, mx4_ref.values(d, s, kk).reshape(E, n, kk)
        (du, up64), (dd, down64) = make(2 * I, H, scale_up), make(H, I, scale_down)
    choice = rng.integers(0, E, T)
    logits = torch.full((T, E), -1e30)
    logits[torch.arange(T), torch.from_numpy(choice)] = 0.0
    y = g.gemm_moe(x.to(DEV), logits.to(DEV), du, dd, k).double().cpu().numpy()
    info = torch.finfo(dtype)
    x64 = x.double().numpy()
    for t in range(T):
        want, tol = layer64(x64[t:t + 1], 1.0, up64[choice[t]], down64[choice[t]], info.eps,
                            info.smallest_normal * info.eps)
        err = np.abs(y[t:t + 1] - want)
        assert (np.abs(want) < info.max / 2).all() and (np.abs(want) > info.smallest_normal).mean() > 0.8, "inputs"
        bad = ~(err <= tol)
        assert not bad.any(), f"token {t}: {bad.sum()} of {bad.size} outside, worst error " \
                              f"{(err / np.abs(want)).max()} of the value"


# T, E, H, I: few rows a load and not, whole and partial groups, one and two
# strips of columns, split sums, both numbers of token tiles
SHAPES = [(1, 3, 64, 64), (4, 8, 200, 130), (16, 2, 128, 96), (12, 4, 6150, 70), (33, 2, 96, 160), (64, 3, 6200, 70),
          (16, 40, 1000, 400), (40, 40, 1000, 400)]


@pytest.mark.parametrize("T,E,H,I", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("power", [-9, -7, -5, 0, 6, 9])
def test_activations_of_any_size(T, E, H, I, dtype, power):
    """gate and up of about 2^power: silu(g) u of 2^(2 power - 1) for negative
    powers, of 2^(2 power) for half of the others; the down weights bring Y back."""
    say(f"moe range T={T} E={E} H={H} I={I} {dtype} 2^{power}")
    back = min(9, -2 * power) if power < 0 else -2 * power
    run(T, E, H, I, dtype, "16", 2.0 ** power, 2.0 ** max(back, -10), T + E + power)


@pytest.mark.parametrize("T,E,H,I", [(4, 8, 200, 130), (33, 2, 96, 160)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("power", [-12, 8])
def test_activations_of_any_size_mx4(T, E, H, I, dtype, power):
    say(f"moe range mx4 T={T} E={E} H={H} I={I} {dtype} 2^{power}")
    run(T, E, H, I, dtype, "mx4", 2.0 ** power, 2.0 ** (-2 * power - 4), T + E + power)


@pytest.mark.parametrize("T", [1, 20])
def test_one_large_activation(T):
    """Past binary16's range, beside a zero weight and a small one."""
    H, I = 32, 40
    up = torch.zeros((1, 2 * I, H), dtype=torch.float16)
    up[0, 3, 0], up[0, I + 3, 0] = 600.0, 700.0          # 420000
    up[0, 5, 0], up[0, I + 5, 0] = 2.0, 1.0
    down = torch.zeros((1, H, I), dtype=torch.float16)
    down[0, 1, 3], down[0, 2, 5], down[0, 4, 3], down[0, 4, 5] = 2.0 ** -10, 1.0, 2.0 ** -8, 1.0
    x = torch.zeros((T, H), dtype=torch.float16)
    x[:, 0] = 1.0
    say(f"moe one large activation {T}")
    y = g.gemm_moe(x.to(DEV), torch.zeros((T, 1), device=DEV), up.to(DEV), down.to(DEV), 1).double().cpu()
    s = 2.0 / (1 + math.exp(-2.0))
    want = torch.zeros((T, H), dtype=torch.float64)
    want[:, 1], want[:, 2], want[:, 4] = 420000 / 1024, s, 420000 / 256 + s
    # two parts, one sum, the output's rounding
    assert ((y - want).abs() <= want * (PARTS + 16 * U + 2.0 ** -11)).all()
