"""MX FP4 products at the ends of the scales' range, and with a last block
whose codes past K are garbage at a scale that makes them huge."""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
import mx4_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def mx4(data, scales, K):
    return g.MX4(torch.from_numpy(np.ascontiguousarray(data)).to(DEV),
                 torch.from_numpy(np.ascontiguousarray(scales)).to(DEV), K)


def garbage_tail(rng, R, K, scale):
    """A random matrix whose last block has zeros up to K, the largest codes
    behind it and the given scale."""
    data, scales = ref.random_codes(rng, R, K, 120, 126)
    last = 32 * (K // 32)
    data[:, last // 2:] = 0x77
    data[:, last // 2: K // 2] = 0
    if K % 2:
        data[:, K // 2] = 0x70
    scales[:, -1] = scale
    assert (ref.values(data, scales, K)[:, last:] == 0).all()
    return data, scales


@pytest.mark.parametrize("M,N", [(1, 40), (1, 7000), (4, 70), (12, 70), (16, 6200), (30, 50), (33, 3100), (64, 9000), (300, 50)])
@pytest.mark.parametrize("K", [40, 161, 300, 1001])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_codes_past_the_end_count_as_absent(M, N, K, dtype):
    rng = np.random.default_rng(M + N + K)
    x = torch.from_numpy(rng.standard_normal((M, K))).to(dtype)
    say(f"mx4 tail a16 {M}x{N}x{K} {dtype}")
    for scale in (140, 253, 254):
        b = garbage_tail(rng, N, K, scale)
        clean = (b[0].copy(), b[1])
        clean[0][:, 16 * (K // 32):] = 0
        got = g.gemm_mx4(x.to(DEV), mx4(*b, K))
        assert torch.isfinite(got).all(), f"scale {scale}"
        assert torch.equal(got, g.gemm_mx4(x.to(DEV), mx4(*clean, K))), f"scale {scale}"


@pytest.mark.parametrize("M,N", [(1, 40), (20, 70), (300, 300), (1600, 1801)])
@pytest.mark.parametrize("K", [40, 161, 300])
def test_codes_past_the_end_count_as_absent_mx4(M, N, K):
    rng = np.random.default_rng(M + N + K)
    a = ref.random_codes(rng, M, K, 120, 126)
    say(f"mx4 tail {M}x{N}x{K}")
    for scale in (140, 253, 254):
        b = garbage_tail(rng, N, K, scale)
        clean = (b[0].copy(), b[1])
        clean[0][:, 16 * (K // 32):] = 0
        qa, qb, qc = mx4(*a, K), mx4(*b, K), mx4(*clean, K)
        for got, want in ((g.gemm_mx4(qa, qb, dtype=torch.bfloat16), g.gemm_mx4(qa, qc, dtype=torch.bfloat16)),
                          (g.gemm_mx4(qb, qa, dtype=torch.bfloat16), g.gemm_mx4(qc, qa, dtype=torch.bfloat16))):
            assert torch.isfinite(got).all() and torch.equal(got, want), f"scale {scale}"


@pytest.mark.parametrize("T,E,k", [(2, 9, 2), (12, 4, 2), (40, 6, 2)])
@pytest.mark.parametrize("H,I", [(40, 72), (300, 161), (6150, 40)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_codes_past_the_end_in_experts(T, E, k, H, I, dtype):
    rng = np.random.default_rng(T + H + I)
    x = torch.from_numpy(rng.standard_normal((T, H))).to(dtype).to(DEV)
    logits = torch.from_numpy(rng.standard_normal((T, E))).float().to(DEV)

    def stack(n, kk, scale, clean):
        d, s = garbage_tail(np.random.default_rng(n + kk), E * n, kk, scale)
        if clean:
            d = d.copy()
            d[:, 16 * (kk // 32):] = 0
        return g.MX4(torch.from_numpy(d).to(DEV).view(E, n, -1), torch.from_numpy(s).to(DEV).view(E, n, -1), kk)

    say(f"moe tail {T} {E} {H} {I} {dtype}")
    for scale in (140, 254):
        y, z = (g.gemm_moe(x, logits, stack(2 * I, H, scale, c), stack(H, I, scale, c), k) for c in (False, True))
        # (a NaN equals nothing; with H 6150, sums of the definition itself pass binary16's range)
        assert torch.equal(y, z), f"scale {scale}"


@pytest.mark.parametrize("scales,power", [((0, 0), 90), ((0, 2), 90), ((1, 1), 90), ((3, 20), 80), ((245, 252), -110),
                                          ((252, 252), -120)])
@pytest.mark.parametrize("M,N", [(1, 40), (20, 48), (40, 6150)])
def test_bfloat16_activations_at_extreme_scales(scales, power, M, N):
    """The least scales (subnormal weights) and the largest that the quantiser
    gives, with activations that bring the sums back."""
    rng = np.random.default_rng(scales[0] + M)
    K = 200
    b = ref.random_codes(rng, N, K, *scales)
    x = torch.from_numpy(rng.standard_normal((M, K)) * 2.0 ** power).to(torch.bfloat16)
    say(f"mx4 extreme scales {scales} {M}x{N}")
    got = g.gemm_mx4(x.to(DEV), mx4(*b, K)).double().cpu().numpy()
    av, bv = x.double().numpy(), ref.values(*b, K)
    info = torch.finfo(torch.bfloat16)
    tol = ref.product_tolerance(av @ bv.T, np.abs(av) @ np.abs(bv).T, K + 8, info.eps, info.smallest_normal * info.eps)
    assert (np.abs(got - av @ bv.T) <= tol).all()


@pytest.mark.parametrize("sa,sb", [((254, 254), (0, 0)), ((250, 254), (0, 5)), ((0, 3), (250, 254)), ((127, 127), (235, 235)),
                                   ((1, 1), (220, 230))])
@pytest.mark.parametrize("M,N", [(3, 40), (70, 50), (1600, 1801)])
def test_mx4_products_at_extreme_scales(sa, sb, M, N):
    """Two scales multiply before anything is rounded: each may be extreme."""
    rng = np.random.default_rng(sa[0] + M)
    K = 200
    a, b = ref.random_codes(rng, M, K, *sa), ref.random_codes(rng, N, K, *sb)
    say(f"mx4 extreme scales {sa} {sb} {M}x{N}")
    got = g.gemm_mx4(mx4(*a, K), mx4(*b, K), dtype=torch.bfloat16).double().cpu().numpy()
    av, bv = ref.values(*a, K), ref.values(*b, K)
    info = torch.finfo(torch.bfloat16)
    want = av @ bv.T
    tol = ref.product_tolerance(want, np.abs(av) @ np.abs(bv).T, K + 8, info.eps, info.smallest_normal * info.eps)
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.parametrize("M", [1, 20, 40])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_weights_past_fp32_beside_16_bits(M, dtype):
    """Scales 253 and 254, which the quantiser never gives: values below 2^128
    are exact, the others infinite when dequantised, and no finite output hides
    them."""
    K = 32
    x = torch.full((M, K), 2.0 ** -14, dtype=dtype, device=DEV)
    data, scales = np.zeros((16, 16), dtype=np.uint8), np.full((16, 1), 253, dtype=np.uint8)
    data[:, 3] = np.arange(16)                # code n of weight row n at k = 6
    say(f"mx4 largest scales {M} {dtype}")
    for scale in (253, 254):
        scales[:] = scale
        q = mx4(data, scales, K)
        values = g.dequantize_mx4(q, torch.float32)[:, 6].double().cpu()
        exact = torch.from_numpy(ref.values(data, scales, K)[:, 6])
        assert torch.equal(values, torch.where(exact.abs() < 2.0 ** 128, exact, exact * torch.inf))
        want = (values * 2.0 ** -14).to(dtype).expand(M, 16)
        got = g.gemm_mx4(x, q).cpu()
        held = torch.isfinite(values)
        assert torch.equal(got[:, held], want[:, held]) and not torch.isfinite(got[:, ~held]).any()
    # the product of two MX4 matrices multiplies the scales first
    small = mx4(np.full((M, 16), 0x22, dtype=np.uint8), np.full((M, 1), 27, dtype=np.uint8), K)   # 1.0 at 2^-100
    got = g.gemm_mx4(small, q, dtype=torch.bfloat16).double().cpu()
    assert torch.equal(got, (exact * 2.0 ** -100).expand(M, 16))
