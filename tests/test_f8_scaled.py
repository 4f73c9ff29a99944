"""Quantisation to 8 bits by blocks of 128, products scaled by blocks, the norm
that feeds them and its gradients, against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
import f8_ref as ref
from f8_ref import E4M3, E5M2, f64
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def randn(*shape, dtype=BF16, seed=0, scale=1.0):
    gen = torch.Generator(device="cpu")
    gen.manual_seed(seed)
    return (torch.randn(*shape, generator=gen) * scale).to(dtype).to(DEV)


def rows8(R, K, dtype, seed, scale=1.0, pad=16, poison=True):
    """8-bit rows that start 16-byte aligned, with NaN codes behind K."""
    ld = -(-K // 16) * 16 + pad
    buf = torch.full((R, ld), 0x7F, dtype=torch.uint8, device=DEV).view(dtype) if poison else \
        torch.zeros(R, ld, dtype=torch.uint8, device=DEV).view(dtype)
    data = buf[:, :K]
    data.copy_(randn(R, K, dtype=F32, seed=seed, scale=scale))
    return data


def scales_of(R, K, seed, low=-6, high=2):
    gen = torch.Generator(device="cpu")
    gen.manual_seed(seed)
    return torch.exp2(torch.rand(R, ref.blocks(K), generator=gen) * (high - low) + low).to(DEV)


# ---- quantisation

SHAPES = [(1, 1), (3, 7), (1, 128), (2, 129), (5, 127), (4, 2048), (2, 2056), (33, 333), (130, 130), (128, 256),
          (257, 385), (9, 4100)]


@pytest.mark.parametrize("R,K", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,order,f8", [(1, "rows", E4M3), (1, "columns", E4M3), (128, "rows", E4M3),
                                           (128, "columns", E5M2), (1, "rows", E5M2), (1, "spread", E4M3),
                                           (128, "spread", E4M3), (1, "columns", E5M2)])
def test_quantize(R, K, dtype, rows, order, f8):
    say(f"quantize {R}x{K} {dtype} {rows} {order} {f8}")
    x = randn(R, K, dtype=dtype, seed=R * K, scale=3.0)
    x[R // 2, K // 2] *= 64
    if order == "columns":
        x = x.t().contiguous().t()
    elif order == "spread":
        x = x.repeat_interleave(2, dim=0).repeat_interleave(3, dim=1)[::2, ::3]
    q, s = ref.quotients(f64(x), rows, f8)
    data, scales = g.quantize_f8(x, rows, f8)
    assert data.shape == x.shape and data.dtype == f8 and scales.dtype == F32
    assert data.data_ptr() % 16 == 0 and (R == 1 or data.stride(0) % 16 == 0)
    assert np.array_equal(f64(scales), s)
    if dtype != F32:
        assert np.array_equal(f64(data), ref.round8(q, f8))
    else:
        # the quotient takes two roundings in float32
        lo, hi = ref.round8(q * (1 - 2.0 ** -22), f8), ref.round8(q * (1 + 2.0 ** -22), f8)
        assert np.all((f64(data) >= np.minimum(lo, hi)) & (f64(data) <= np.maximum(lo, hi)))


@pytest.mark.parametrize("dtype,f8", [(F16, E4M3), (F16, E5M2), (BF16, E4M3), (BF16, E5M2)])
def test_quantize_every_16_bit_value_against_many_maxima(dtype, f8):
    """Blocks of one maximum and values below it: every tie that 16-bit numbers
    can make is met exactly."""
    say(f"quantize ties {dtype} {f8}")
    gen = torch.Generator(device="cpu")
    gen.manual_seed(5)
    bits = torch.randint(0, 1 << 16, (4096, 256), generator=gen, dtype=torch.int32).to(torch.int16)
    x = bits.view(dtype)
    top = torch.finfo(dtype)
    x = torch.where(torch.isfinite(x), x, torch.ones_like(x))
    m = x[:, :1].abs().float().clamp(min=float(top.tiny))
    # magnitudes within four binades below the row's first
    x = (torch.sign(x.float()) * m * torch.exp2(-4 * torch.rand(4096, 256, generator=gen))).to(dtype)
    x[:, 0] = m[:, 0].to(dtype)
    x[:, 128] = m[:, 0].to(dtype)
    q, s = ref.quotients(f64(x), 1, f8)
    ties = int((np.abs(ref.round8(q * (1 + 2e-7), f8) - ref.round8(q * (1 - 2e-7), f8)) > 0).sum())
    assert ties > 100          # of a million elements, counted by the definition alone
    data, scales = g.quantize_f8(x.to(DEV), 1, f8)
    assert np.array_equal(f64(scales), s)
    assert np.array_equal(f64(data), ref.round8(q, f8))


@pytest.mark.parametrize("rows,order", [(1, "rows"), (1, "columns"), (128, "rows"), (128, "columns")])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_quantize_extremes(rows, order, dtype):
    say(f"quantize extremes {rows} {order} {dtype}")
    R, K = 8 * 128 + 3, 300
    x = randn(R, K, dtype=dtype, seed=3)
    top = float(torch.finfo(dtype).max)
    for i, v in enumerate((0.0, float(torch.finfo(dtype).smallest_normal) / 4, top, float("nan"), float("inf"),
                           -float("inf"), 2.0 ** -120 if dtype != F16 else 2.0 ** -24)):
        x[128 * i:128 * i + 128, 128:256] = 0.0
        x[128 * i + 5, 130] = v
        if v == v and abs(v) < top:
            x[128 * i + 5, 140] = v / 2
    if order == "columns":
        x = x.t().contiguous().t()
    q, s = ref.quotients(f64(x), rows, E4M3)
    data, scales = g.quantize_f8(x, rows)
    assert np.array_equal(f64(scales), s, equal_nan=True)
    if dtype != F32:
        assert np.array_equal(f64(data), ref.round8(q, E4M3))
    else:
        lo, hi = ref.round8(q * (1 - 2.0 ** -22), E4M3), ref.round8(q * (1 + 2.0 ** -22), E4M3)
        assert np.all((f64(data) >= np.minimum(lo, hi)) & (f64(data) <= np.maximum(lo, hi)))


@pytest.mark.parametrize("rows,order", [(1, "rows"), (1, "columns"), (128, "rows"), (128, "columns")])
def test_quantize_into_given_outputs(rows, order):
    say(f"quantize out {rows} {order}")
    R, K = 200, 333
    x = randn(R, K, seed=8)
    if order == "columns":
        x = x.t().contiguous().t()
    want, ws = g.quantize_f8(x, rows)
    buf = torch.full((R, 401), 0x55, dtype=torch.uint8, device=DEV)
    sr = R if rows == 1 else 2
    sbuf = torch.full((3, 2 * sr), -7.0, device=DEV)
    out = (buf.view(E4M3)[:, 3:3 + K], sbuf.t()[::2])
    got = g.quantize_f8(x, rows, out=out)
    assert got[0] is out[0] and got[1] is out[1]
    assert torch.equal(out[0].view(torch.uint8), want.view(torch.uint8)) and torch.equal(out[1], ws)
    assert (buf[:, :3] == 0x55).all() and (buf[:, 3 + K:] == 0x55).all() and (sbuf[:, 1::2] == -7).all()


def test_quantize_blocks_of_the_transpose_are_those_of_the_matrix():
    x = randn(300, 500, seed=4)
    a, sa = g.quantize_f8(x, 128)
    b, sb = g.quantize_f8(x.t(), 128)
    assert torch.equal(sa, sb.t()) and torch.equal(a.view(torch.uint8), b.view(torch.uint8).t())


# ---- products

SIZES = [(1, 1, 1), (1, 5, 130), (2, 3, 127), (1, 2048, 128), (3, 129, 256), (16, 64, 640), (17, 65, 129), (48, 200, 1000),
         (64, 256, 2048), (65, 127, 257), (100, 300, 384), (128, 128, 1280), (129, 257, 515), (256, 256, 128),
         (300, 520, 1037), (512, 512, 512)]


def check_product(a, sa, b, sb, dtype, what, **kw):
    say(what)
    c = g.gemm_f8_scaled(a, sa, b, sb, dtype=dtype, **kw)
    want, tol = ref.product(a, sa, b, sb, dtype)
    assert c.dtype == dtype
    ref.assert_near(c, want, tol, what)
    return c


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("fa,fb,brows,dtype", [(E4M3, E4M3, 128, BF16), (E4M3, E4M3, 1, F16), (E5M2, E4M3, 1, F32),
                                               (E4M3, E5M2, 128, F32), (E5M2, E5M2, 128, F16)])
def test_product(M, N, K, fa, fb, brows, dtype):
    a, b = rows8(M, K, fa, 1), rows8(N, K, fb, 2)
    sa, sb = scales_of(M, K, 3), scales_of(-(-N // brows), K, 4)
    check_product(a, sa, b, sb, dtype, f"f8 scaled {M}x{N}x{K} {fa} {fb} {brows} {dtype}")


VARIANTS = list(g.f8_scaled.VARIANTS)


def taken(variant, brows, dtype):
    return variant != "tile256x256" or (brows == 128 and dtype != F32)


def whole(R, K, dtype, seed):
    """Whole numbers of up to 4 in 8 bits, with NaN codes behind K."""
    data = rows8(R, K, dtype, seed)
    data.copy_(torch.from_numpy(np.random.default_rng(seed).integers(-4, 5, (R, K))).float())
    return data


def rounded(c, dtype):
    """Whole numbers below 2^24 to dtype, once."""
    return f64(torch.from_numpy(c).float().to(dtype))


@pytest.mark.parametrize("M,N,K", [(1, 100, 700), (31, 70, 128), (70, 130, 300), (200, 300, 900), (513, 700, 1281)])
@pytest.mark.parametrize("brows", [1, 128])
@pytest.mark.parametrize("variant", VARIANTS)
def test_exact_on_whole_numbers(M, N, K, brows, variant):
    """Whole numbers of up to 4 and scales of 1, 2 and 4: every sum is exact, so
    every bit of a result is."""
    a, b = whole(M, K, E4M3, 1), whole(N, K, E5M2, 2)
    rng = np.random.default_rng(M + N)
    sa = torch.from_numpy(2.0 ** rng.integers(0, 3, (M, ref.blocks(K)))).float().to(DEV)
    sb = torch.from_numpy(2.0 ** rng.integers(0, 3, (-(-N // brows), ref.blocks(K)))).float().to(DEV)
    want, _ = ref.product(a, sa, b, sb, F32)
    for dtype in (F32, F16, BF16):
        if taken(variant, brows, dtype):
            say(f"f8 scaled exact {M}x{N}x{K} {brows} {variant} {dtype}")
            c = g.gemm_f8_scaled(a, sa, b, sb, dtype=dtype, variant=variant)
            assert np.array_equal(f64(c), rounded(want, dtype))


@pytest.mark.parametrize("K", [1, 16, 17, 127, 128, 129, 255, 256, 384, 500, 512, 640, 641, 1025, 1153, 2049, 2176])
@pytest.mark.parametrize("variant", VARIANTS)
def test_every_number_of_blocks(K, variant):
    """Rings that are longer than K, and K's end at every place of them."""
    say(f"f8 scaled blocks {K} {variant}")
    M, N = 90, 150
    a, b = whole(M, K, E5M2, 3), whole(N, K, E4M3, 4)
    rng = np.random.default_rng(K)
    sa = torch.from_numpy(2.0 ** rng.integers(0, 3, (M, ref.blocks(K)))).float().to(DEV)
    sb = torch.from_numpy(2.0 ** rng.integers(0, 3, (2, ref.blocks(K)))).float().to(DEV)
    want, _ = ref.product(a, sa, b, sb, F32)
    assert np.array_equal(f64(g.gemm_f8_scaled(a, sa, b, sb, dtype=BF16, variant=variant)), rounded(want, BF16))


@pytest.mark.parametrize("variant", VARIANTS)
@pytest.mark.parametrize("fa,fb", [(E4M3, E4M3), (E4M3, E5M2), (E5M2, E4M3), (E5M2, E5M2)])
def test_every_code_times_every_code(fa, fb, variant):
    """Row m has code m at one place, so C is the table of products, each exact in
    float32: subnormal and non-finite codes included."""
    say(f"f8 scaled codes {fa} {fb} {variant}")
    K, at = 200, 150
    a, b = torch.zeros(256, 208, dtype=torch.uint8), torch.zeros(256, 208, dtype=torch.uint8)
    a[:, at] = b[:, at] = torch.arange(256).to(torch.uint8)
    a, b = a.to(DEV).view(fa)[:, :K], b.to(DEV).view(fb)[:, :K]
    one = torch.ones(256, 2, device=DEV)
    with np.errstate(invalid="ignore"):
        table = np.outer(f64(a)[:, at], f64(b)[:, at])
    for dtype, sb in ((F32, one), (BF16, one[:2])):
        if taken(variant, sb.shape[0] // 256 or 128, dtype):
            c = g.gemm_f8_scaled(a, one, b, sb, dtype=dtype, variant=variant)
            want = f64(torch.from_numpy(table).float().to(dtype))
            assert np.array_equal(f64(c), want, equal_nan=True)


@pytest.mark.parametrize("variant", VARIANTS[1:])
@pytest.mark.parametrize("M,N,K", [(300, 400, 1100), (70, 260, 2000)])
def test_variants_within_tolerance(M, N, K, variant):
    a, b = rows8(M, K, E4M3, 1), rows8(N, K, E4M3, 2)
    for brows in (1, 128):
        sa, sb = scales_of(M, K, 3), scales_of(-(-N // brows), K, 4)
        for dtype in (F32, F16, BF16):
            if taken(variant, brows, dtype):
                check_product(a, sa, b, sb, dtype, f"f8 scaled {M}x{N}x{K} {brows} {variant} {dtype}", variant=variant)


def test_variants_that_do_not_take_the_call():
    a, b, s = rows8(8, 128, E4M3, 1), rows8(8, 128, E4M3, 2), torch.ones(8, 1, device=DEV)
    for sb, dtype in ((s, BF16), (s[:1], F32)):
        with pytest.raises(g.GemmError):
            g.gemm_f8_scaled(a, s, b, sb, dtype=dtype, variant="tile256x256")
    with pytest.raises(KeyError):
        g.gemm_f8_scaled(a, s, b, s, variant="tile1x1")


@pytest.mark.parametrize("M,N,K", [(1, 300, 700), (20, 300, 700), (200, 300, 700)])
def test_strides_of_operands_scales_and_output(M, N, K):
    a, b = rows8(M, K, E4M3, 1, pad=48), rows8(N, K, E4M3, 2, pad=160)
    sa = scales_of(2 * ref.blocks(K), 128 * 3 * M, 3).t()[::3, ::2][:M]
    sb = scales_of(ref.blocks(K), 128 * N, 4).t()
    assert sa.shape == (M, ref.blocks(K)) and sb.shape == (N, ref.blocks(K))
    for dtype in (BF16, F32):
        for pad, off in ((0, 0), (3, 1), (8, 8)):
            buf = torch.full((M + 2, N + pad + off), 7.0, dtype=dtype, device=DEV)
            out = buf[1:M + 1, off:off + N]
            c = check_product(a, sa, b, sb, dtype, f"f8 scaled strides {M} {dtype} {pad} {off}", out=out)
            assert c is out
            buf[1:M + 1, off:off + N] = 7.0
            assert (buf == 7).all()


@pytest.mark.parametrize("M,N,K", [(1, 200, 300), (40, 200, 300), (260, 200, 300)])
def test_non_finite_elements_and_scales_stay_in_their_rows(M, N, K):
    say(f"f8 scaled nan {M}")
    a, b = rows8(M, K, E4M3, 1), rows8(N, K, E4M3, 2)
    sa, sb = scales_of(M, K, 3), scales_of(N, K, 4)
    clean = g.gemm_f8_scaled(a, sa, b, sb, dtype=F32)
    a[M // 2, 200] = float("nan")
    sb[77, 1] = float("nan")
    sb[78, 2] = float("inf")
    c = g.gemm_f8_scaled(a, sa, b, sb, dtype=F32)
    assert torch.isnan(c[M // 2]).all() and torch.isnan(c[:, 77]).all() and not torch.isfinite(c[:, 78]).any()
    keep = torch.ones_like(c, dtype=torch.bool)
    keep[M // 2], keep[:, 77], keep[:, 78] = False, False, False
    assert torch.equal(c[keep], clean[keep])


@pytest.mark.parametrize("fa", [E4M3, E5M2])
def test_scales_over_the_whole_range(fa):
    """Blocks of 2^-60 beside blocks of 2^60: the large ones must not drown in an
    intermediate overflow nor the small ones, alone in their row, vanish."""
    M, N, K = 64, 200, 512
    a, b = rows8(M, K, fa, 1), rows8(N, K, E4M3, 2)
    sa = torch.exp2(torch.linspace(-60, 60, M, device=DEV)[:, None] * torch.ones(1, 4, device=DEV))
    sb = torch.exp2(torch.linspace(50, -50, N, device=DEV)[:, None] * torch.ones(1, 4, device=DEV))
    check_product(a, sa, b, sb, F32, f"f8 scaled range {fa}")


def test_linear_layer_and_its_gradients():
    """y = x w^T, dx = dy w, dw = dy^T x, all in 8 bits, against the product of the
    values that the 8 bits stand for; and against differences of <y, dy>, which
    is linear in x and w, within what 8 bits leave."""
    T, N, K = 300, 260, 390
    x, w, dy = randn(T, K, seed=1), randn(N, K, seed=2, scale=0.05), randn(T, N, seed=3, scale=0.01)
    qx, qw, qd = g.quantize_f8(x), g.quantize_f8(w, 128), g.quantize_f8(dy, dtype=E5M2)
    y = check_product(*qx, *qw, BF16, "linear")
    dx = check_product(*qd, *g.quantize_f8(w.t(), 128), BF16, "linear dx")
    dw = check_product(*g.quantize_f8(dy.t(), dtype=E5M2), *g.quantize_f8(x.t()), F32, "linear dw")
    for got, a, b in ((y, x, w.t()), (dx, dy, w), (dw, dy.t(), x)):
        # relative steps 2^-4 and 2^-3 (and 2^-9 of the output), on the 2-norm; roundings of both sides add up
        want = f64(a) @ f64(b)
        mag = np.sqrt((f64(a) ** 2) @ (f64(b) ** 2))
        assert np.linalg.norm(f64(got) - want) <= (2.0 ** -4 + 2.0 ** -3 + 2.0 ** -8) * np.linalg.norm(mag)
    d = randn(T, K, seed=9, dtype=F32).double()
    slope = float(((d.cpu() @ w.double().cpu().t()) * dy.double().cpu()).sum())
    assert abs(float((dx.double().cpu() * d.cpu()).sum()) - slope) <= 0.2 * float(dx.double().norm() * d.norm()) / 8


# ---- the norm

NORMS = [(1, 1), (1, 7), (3, 128), (5, 129), (4, 511), (9, 1024), (7, 1025), (16, 2051), (3, 7168), (2, 16384), (2, 16392),
         (1, 40001), (1, 65536), (1030, 64)]


@pytest.mark.parametrize("R,K", NORMS)
@pytest.mark.parametrize("dtype,wt,res,f8", [(BF16, F32, True, E4M3), (F16, F16, False, E4M3), (F16, F32, True, E5M2),
                                             (BF16, BF16, False, E5M2)])
def test_norm(R, K, dtype, wt, res, f8):
    say(f"norm {R}x{K} {dtype} {wt} {res} {f8}")
    x, w = randn(R, K, dtype=dtype, seed=R + K), (1 + 0.3 * randn(K, dtype=F32, seed=5)).to(wt)
    r = randn(R, K, dtype=dtype, seed=6, scale=2.0) if res else None
    if R > 2:
        x[1] = 0
        if res:
            r[1] = 0
    h, y, e = ref.norm(x, r, w, 1e-6)
    data, scales, got = g.rms_norm_f8(x, w, 1e-6, residual=r, dtype=f8)
    assert torch.equal(got.cpu(), h) and (res or got is x)
    q, s = ref.quotients(y, 1, f8)
    assert np.all(np.abs(f64(scales) - s) <= s * (e + 2.0 ** -23))
    lo, hi = ref.round8(q * (1 - 2 * e - 2.0 ** -21), f8), ref.round8(q * (1 + 2 * e + 2.0 ** -21), f8)
    assert np.all((f64(data) >= np.minimum(lo, hi)) & (f64(data) <= np.maximum(lo, hi)))


def test_norm_views_and_in_place():
    say("norm views")
    R, K = 37, 515
    x, r = randn(R, K + 9, seed=1)[:, 4:4 + K], randn(R, K + 1, seed=2)[:, 1:]
    w = randn(K, dtype=F32, seed=3)
    want = g.rms_norm_f8(x.contiguous(), w, residual=r.contiguous())
    buf = torch.full((R, 800), 0x55, dtype=torch.uint8, device=DEV)
    sbuf = torch.zeros(ref.blocks(K), R, device=DEV)
    hbuf = torch.full((R, K + 6), 3.0, dtype=BF16, device=DEV)
    got = g.rms_norm_f8(x, w, residual=r, out=(buf.view(E4M3)[:, 5:5 + K], sbuf.t()), h=hbuf[:, 2:2 + K])
    for a, b in zip(want, got):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    assert (buf[:, :5] == 0x55).all() and (buf[:, 5 + K:] == 0x55).all()
    assert (hbuf[:, :2] == 3).all() and (hbuf[:, 2 + K:] == 3).all()
    for t in ("x", "r"):
        xs, rs = x.contiguous(), r.contiguous()
        into = xs if t == "x" else rs
        got = g.rms_norm_f8(xs, w, residual=rs, h=into)
        assert got[2] is into and torch.equal(into, want[2]) and torch.equal(got[1], want[1])


def test_norm_rows_with_non_finite_elements():
    say("norm nan")
    x, w = randn(6, 400, seed=1), torch.ones(400, device=DEV)
    clean = g.rms_norm_f8(x, w)
    x[2, 3], x[4, 300] = float("nan"), float("inf")
    data, scales, _ = g.rms_norm_f8(x, w)
    # an infinite mean square leaves zeros, and a NaN where the infinity was
    assert torch.isnan(scales[2]).all() and torch.isnan(scales[4, 2]) and (scales[4, :2] == 2.0 ** -126).all()
    assert (data[2].float() == 0).all() and (data[4].float() == 0).all()
    for i in (0, 1, 3, 5):
        assert torch.equal(scales[i], clean[1][i]) and torch.equal(data[i].float(), clean[0][i].float())


GRADS = NORMS + [(700, 300), (2500, 130), (600, 1200)]


@pytest.mark.parametrize("R,K", GRADS)
@pytest.mark.parametrize("dtype,wt,res", [(BF16, F32, True), (F16, F16, False)])
def test_norm_backward(R, K, dtype, wt, res):
    say(f"norm backward {R}x{K} {dtype} {wt} {res}")
    h, w = randn(R, K, dtype=dtype, seed=R + K, scale=2.0), (1 + 0.3 * randn(K, dtype=F32, seed=5)).to(wt)
    dy, dh = randn(R, K, dtype=dtype, seed=7, scale=0.1), randn(R, K, dtype=dtype, seed=8, scale=0.1) if res else None
    if R > 2:
        h[1] = 0
    dx, dw = g.rms_norm_backward(dy, h, w, 1e-6, dh=dh)
    assert dx.dtype == dtype and dw.dtype == wt
    wx, tx, ww, tw = ref.norm_grad(dy, h, w, 1e-6, dh)
    ref.assert_near(dx, wx, tx + ref.half_step(np.abs(wx) + tx, dtype), "dx")
    ref.assert_near(dw, ww, tw + ref.half_step(np.abs(ww) + tw, wt), "dw")


def test_norm_backward_against_differences():
    """The change of <y, dy> + <h, dh> along a direction, by central differences
    of the norm's own formula in 64 bits."""
    say("norm differences")
    R, K, eps = 7, 200, 1e-3
    h, w = randn(R, K, dtype=F16, seed=1), randn(K, dtype=F32, seed=2)
    dy, dh = randn(R, K, dtype=F16, seed=3), randn(R, K, dtype=F16, seed=4)
    dx, dw = g.rms_norm_backward(dy, h, w, eps, dh=dh)
    H, W, Y, D = f64(h), f64(w), f64(dy), f64(dh)

    def loss(v, wt):
        return float((v / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps) * wt * Y).sum() + (v * D).sum())

    rng = np.random.default_rng(1)
    for _ in range(8):
        u, t = rng.standard_normal((R, K)), 1e-5
        slope = (loss(H + t * u, W) - loss(H - t * u, W)) / (2 * t)
        # half steps of 2^-11 on dx, random against u
        assert abs(slope - (f64(dx) * u).sum()) <= 2.0 ** -11 * np.linalg.norm(f64(dx)) * 6 + 1e-5 * abs(slope)
        u = rng.standard_normal(K)
        slope = (loss(H, W + t * u) - loss(H, W - t * u)) / (2 * t)
        assert abs(slope - (f64(dw) * u).sum()) <= 1e-5 * np.linalg.norm(f64(dw)) * 6 + 1e-6 * abs(slope)


def test_norm_backward_views_in_place_and_workspace():
    say("norm backward views")
    R, K = 70, 515
    dy, h = randn(R, K + 9, seed=1)[:, 4:4 + K], randn(R, K + 1, seed=2)[:, 1:]
    dh, w = randn(R, K + 2, seed=3)[:, :K], randn(K, dtype=F32, seed=4)
    dx, dw = g.rms_norm_backward(dy.contiguous(), h.contiguous(), w, dh=dh.contiguous())
    buf = torch.full((R, K + 5), 3.0, dtype=BF16, device=DEV)
    ws = torch.empty(g.rms_norm_backward_workspace_bytes(R, K), dtype=torch.uint8, device=DEV)
    gx, gw = g.rms_norm_backward(dy, h, w, dh=dh, out=buf[:, 1:1 + K], workspace=ws)
    assert torch.equal(gx, dx) and torch.equal(gw, dw) and (buf[:, 0] == 3).all() and (buf[:, 1 + K:] == 3).all()
    for i in range(2):
        a, b = dy.contiguous(), dh.contiguous()
        into = (a, b)[i]
        gx, gw = g.rms_norm_backward(a, h, w, dh=b, out=into)
        assert gx is into and torch.equal(gx, dx) and torch.equal(gw, dw)


def test_norm_into_linear_layer():
    """As a model uses them: the sum with the residual, the norm, the projection."""
    say("norm and linear")
    T, H, N = 70, 640, 300
    x, r, w = randn(T, H, seed=1), randn(T, H, seed=2), 1 + 0.2 * randn(H, dtype=F32, seed=3)
    p = g.quantize_f8(randn(N, H, seed=4, scale=H ** -0.5), 128)
    data, scales, h = g.rms_norm_f8(x, w, residual=r)
    c = check_product(data, scales, *p, BF16, "norm and linear")
    _, y, _ = ref.norm(x, r, w, 1e-6)
    want = y @ ref.values(*p).T
    mag = np.sqrt((y ** 2) @ (ref.values(*p).T ** 2))
    assert np.linalg.norm(f64(c) - want) <= (2.0 ** -4 + 2.0 ** -8) * np.linalg.norm(mag)
