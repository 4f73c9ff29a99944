"""Products scaled by blocks where a row's scale times a column's leaves float32's
normal range, though the block's sum brings the result back into it: every
kernel, row and square blocks, every output type, against 64 bits."""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
import f8_ref as ref
from f8_ref import E4M3, E5M2, f64
from gpu_util import DEV, say
from test_f8_scaled import BF16, F16, F32, VARIANTS, taken

pytestmark = pytest.mark.gpu

# Least and largest scales that quantisation makes, and some between them.
SCALES = [2.0 ** -126, 1.5 * 2.0 ** -126, 1.3 * 2.0 ** -100, 1.7 * 2.0 ** -63, 1.3 * 2.0 ** -20, 1.1, 1.9 * 2.0 ** 30,
          1.3 * 2.0 ** 64, 1.7 * 2.0 ** 100, 1.9 * 2.0 ** 119]


def codes(R, K, dtype, seed, unit):
    """Whole numbers of up to 4 times `unit`, all of them 8-bit values, so that a
    block's sum is exact; rows start 16-byte aligned, with NaN codes behind K."""
    ld = -(-K // 16) * 16 + 16
    data = torch.full((R, ld), 0x7F, dtype=torch.uint8, device=DEV).view(dtype)[:, :K]
    data.copy_((torch.from_numpy(np.random.default_rng(seed).integers(-4, 5, (R, K))).float() * unit).to(dtype))
    return data


def check(c, a, sa, b, sb, dtype, what):
    """Each block's sum meets its scales with two roundings, each addition is
    rounded once, and no step is finer than 2^-149; past float32's largest value a
    sum is not finite."""
    x, y = ref.values(a, sa), ref.values(b, sb)
    want, mag, n = x @ y.T, np.abs(x) @ np.abs(y).T, sa.shape[1]
    got = f64(c)
    top = float(torch.finfo(dtype).max)
    tol = (3 * n + 8) * 2.0 ** -24 * mag + (n + 1) * 2.0 ** -149
    tol = tol + ref.half_step(np.abs(want) + tol, dtype)
    small = (mag < 2.0 ** 127) & (np.abs(want) + tol < top)
    # (the sum of K products in float64 is itself off by up to K 2^-53 of their magnitudes)
    large = np.abs(want) > 2 * top + a.shape[1] * 2.0 ** -52 * mag
    assert small.sum() > 0
    bad = small & ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {small.sum()} off, first {got[bad][0]} for {want[bad][0]}"
    bad = large & ~(got == np.copysign(np.inf, want))
    assert not bad.any(), f"{what}: {bad.sum()} of {large.sum()} not infinite, first {got[bad][0]} for {want[bad][0]}"


FORMS = [(E4M3, E4M3, 2.0 ** -9, 2.0 ** -9), (E4M3, E4M3, 64.0, 64.0), (E5M2, E4M3, 2.0 ** -16, 1.0),
         (E4M3, E5M2, 1.0, 8192.0), (E5M2, E5M2, 2.0 ** -16, 2.0 ** -16), (E5M2, E5M2, 8192.0, 8192.0)]


@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("brows", [1, 128])
@pytest.mark.parametrize("variant", VARIANTS)
def test_every_pair_of_scales(form, brows, variant):
    """Every scale of SCALES on a row meets every one on a block of columns."""
    fa, fb, ua, ub = FORMS[form]
    n = len(SCALES)
    M, N, K = 70, 128 * n if brows == 128 else 16 * n, 300
    a, b = codes(M, K, fa, 1, ua), codes(N, K, fb, 2, ub)
    s = torch.tensor(SCALES, dtype=F32)
    sa = s[torch.arange(M) % n][:, None].repeat(1, ref.blocks(K)).to(DEV)
    sb = s[torch.arange(N // brows) % n][:, None].repeat(1, ref.blocks(K)).to(DEV)
    for dtype in (F32, BF16, F16):
        if taken(variant, brows, dtype):
            what = f"f8 scaled range {form} {brows} {variant} {dtype}"
            say(what)
            check(g.gemm_f8_scaled(a, sa, b, sb, dtype=dtype, variant=variant), a, sa, b, sb, dtype, what)


@pytest.mark.parametrize("size", [(40, 256, 640), (300, 512, 1300)])
@pytest.mark.parametrize("brows", [1, 128])
@pytest.mark.parametrize("variant", VARIANTS)
def test_blocks_of_zeros_under_any_scale(size, brows, variant):
    """A block whose products are all zero adds nothing, whatever its scales: rows
    of A hold zeros where B's block has its scale, and their other blocks lie at
    2^-110 or at 1."""
    M, N, K = size
    say(f"f8 scaled zeros {size} {brows} {variant}")
    a, b = codes(M, K, E4M3, 3, 1.0), codes(N, K, E4M3, 4, 1.0)
    a[:, 128:256] = 0
    a[M // 2:M // 2 + 3] = 0                               # whole rows too
    sa, sb = torch.ones(M, ref.blocks(K)), torch.ones(N // brows, ref.blocks(K))
    sa[::2] = 2.0 ** -110
    sa[:, 1], sb[:, 1] = 1.5 * 2.0 ** 100, 1.5 * 2.0 ** 90
    sa[M // 2:M // 2 + 3] = 2.0 ** -126
    sa, sb = sa.to(DEV), sb.to(DEV)
    for dtype in (F32, BF16, F16):
        if taken(variant, brows, dtype):
            c = g.gemm_f8_scaled(a, sa, b, sb, dtype=dtype, variant=variant)
            check(c, a, sa, b, sb, dtype, f"{variant} {dtype}")
            assert not c[M // 2:M // 2 + 3].any()


@pytest.mark.parametrize("variant", VARIANTS)
def test_rows_of_large_results_leave_the_others_as_they_are(variant):
    """Results on both sides of 2^88, non-finite rows and columns among them: every
    other element keeps its bits."""
    say(f"f8 scaled large rows {variant}")
    M, N, K = 150, 384, 700
    for brows, dtype in ((128, BF16), (1, F32)):
        if not taken(variant, brows, dtype):
            continue
        a, b = codes(M, K, E4M3, 5, 1.0), codes(N, K, E4M3, 6, 1.0)
        rng = np.random.default_rng(7)
        sa = torch.from_numpy(2.0 ** rng.uniform(-8, 8, (M, ref.blocks(K)))).float().to(DEV)
        sb = torch.from_numpy(2.0 ** rng.uniform(-8, 8, (N // brows, ref.blocks(K)))).float().to(DEV)
        clean = g.gemm_f8_scaled(a, sa, b, sb, dtype=dtype, variant=variant)
        sa[20] *= 2.0 ** 80
        sa[21] *= 2.0 ** 100
        sa[100, 3] = float("nan")
        c = g.gemm_f8_scaled(a, sa, b, sb, dtype=dtype, variant=variant)
        keep = torch.ones(M, dtype=torch.bool, device=DEV)
        keep[[20, 21, 100]] = False
        assert torch.equal(c[keep], clean[keep]) and torch.isnan(c[100]).all()
        rows = slice(20, 22)
        check(c[rows], a[rows], sa[rows], b, sb, dtype, f"{variant} {dtype}")
        again = g.gemm_f8_scaled(a, sa, b, sb, dtype=dtype, variant=variant)
        assert torch.equal(c[keep], again[keep]) and torch.equal(c[rows], again[rows])


@pytest.mark.parametrize("size", [(1, 203, 300), (37, 203, 300), (150, 391, 700)])
@pytest.mark.parametrize("brows", [1, 128])
@pytest.mark.parametrize("variant", VARIANTS)
def test_large_results_into_views(size, brows, variant):
    """Sums that are formed again, with strides of their own in scales and output, whose
    surroundings stay as they were; infinities where float32 ends."""
    M, N, K = size
    say(f"f8 scaled large views {size} {brows} {variant}")
    a, b = codes(M, K, E5M2, 8, 1.0), codes(N, K, E4M3, 9, 1.0)
    n = ref.blocks(K)
    sa, sb = torch.ones(2 * n, 3 * M, device=DEV).t()[::3, ::2], torch.ones(n, -(-N // brows), device=DEV).t()
    sa[::2] = 1.25 * 2.0 ** 70
    sa[::3] = 1.25 * 2.0 ** 110
    sb[::2] = 1.5 * 2.0 ** 14
    for dtype in (F32, BF16, F16)[:2 if M == 1 else 3]:     # (a row of infinities in float16)
        if taken(variant, brows, dtype):
            buf = torch.full((M + 2, N + 5), 7.0, dtype=dtype, device=DEV)
            out = buf[1:M + 1, 3:3 + N]
            c = g.gemm_f8_scaled(a, sa, b, sb, out=out, variant=variant)
            check(c.contiguous(), a, sa, b, sb, dtype, f"{variant} {dtype}")
            out.fill_(7.0)
            assert (buf == 7).all()
