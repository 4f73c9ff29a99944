"""8-bit floating point (OCP E4M3 and E5M2) with a float32 scale for each block
of 128: quantisation and products.  Argument marshalling for
include/gemm_f8_scaled.h; the computation runs in the HIP library.

    quantize_f8(x)                                  -> data [R, K], scales
    gemm_f8_scaled(a, a_scales, b, b_scales)        -> C [M, N] = a . b^T

data is a float8_e4m3fn or float8_e5m2 tensor; scales is float32, either [R,
ceil(K/128)], one for each 128 consecutive elements of a row ("row blocks"), or
[ceil(R/128), ceil(K/128)], one for each 128 rows x 128 elements ("square
blocks").  An element's value is its 8-bit value times its block's scale.

A linear layer y = x . w^T keeps its activations in row blocks and its weights
in square blocks.  Those are the same blocks of the transposed weights, so
dx = dy . w takes quantize_f8(w.t(), 128) as b; and dw = dy^T . x takes both
operands in row blocks along the tokens, quantize_f8(dy.t()) and
quantize_f8(x.t()).

A stream by argument: as the package says.
"""
import torch

from ._lib import F8sArgs, F8sQuantizeArgs, lib, packer
from .mx4 import FORMATS, _call, _check_stream, _keep, _new2

BLOCK = 128
FORMATS8 = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}

# Kernels that a call may be given to (enum gemm_f8s_variant).
VARIANTS = {name: i for i, name in enumerate(("auto", "strip16x16", "strip16x32", "strip32x16", "strip32x32", "strip64x32",
                                              "strip64x64", "tile64x128", "tile128x128", "tile256x256"))}

_c_quantize, _c_product = lib.gemm_f8s_quantize, lib.gemm_f8s
_quantize_args, _product_args = packer(F8sQuantizeArgs), packer(F8sArgs)


def _new_f8(R, K, dtype, device, stream):
    """[R, K] in 8 bits whose rows start 16-byte aligned, as the products want
    them."""
    pitch = -(-K // 16) * 16
    data = _new2(R, pitch, dtype, device, stream)
    return data if pitch == K else data[:, :K]


def _check_f8_out(data, scales, dtype, device, R, K, block_rows):
    if data.dtype != dtype or data.device != device or data.shape != (R, K) or \
            (data.stride(1) != 1 and K > 1) or (data.stride(0) < K and R > 1):
        raise ValueError("out's data must be a row-major [R, K] tensor of dtype on the inputs' device")
    if scales.dtype != torch.float32 or scales.device != device or \
            scales.shape != (-(-R // block_rows), -(-K // BLOCK)) or min(scales.stride()) <= 0:
        raise ValueError("out's scales must be a float32 tensor of a scale per block, with positive strides, on the "
                         "inputs' device")


def quantize_f8(x, rows=1, dtype=torch.float8_e4m3fn, out=None, stream=None):
    """(data, scales) of x [R, K] (float16, bfloat16 or float32, any positive
    strides) in blocks of `rows` (1 or 128) rows x 128 elements.

    With m the block's largest magnitude and L dtype's largest value (448 for
    float8_e4m3fn, 57344 for float8_e5m2) the scale is m / L, at least 2^-126;
    elements are multiplied by L / m and rounded to nearest, ties to even.  A block
    with an infinity or a NaN gets a NaN scale and zero elements.
    data has rows that start 16-byte aligned.  out: a pair (data, scales), data
    with any row stride, scales with any positive strides that keep them apart."""
    fmt, fmt8, device = FORMATS.get(x.dtype), FORMATS8.get(dtype), x.device
    if fmt is None:
        raise TypeError("expected float16, bfloat16 or float32")
    if fmt8 is None:
        raise TypeError("dtype must be float8_e4m3fn or float8_e5m2")
    if x.ndim != 2 or device.type != "cuda":
        raise ValueError("expected an [R, K] matrix on a GPU")
    if rows != 1 and rows != BLOCK:
        raise ValueError("blocks have 1 or 128 rows")
    R, K = x.shape
    sr, sk = x.stride()
    if R <= 0 or K <= 0:
        raise ValueError("empty shape")
    if sr <= 0 or sk <= 0:
        raise ValueError("strides must be positive")
    if stream is not None:
        _check_stream(stream, device)
    if out is None:
        blocks = -(-K // BLOCK)
        data = _new_f8(R, K, dtype, device, stream)
        scales = _new2(R if rows == 1 else -(-R // BLOCK), blocks, torch.float32, device, stream)
        pitch, ss_r, ss_k = -(-K // 16) * 16, blocks, 1
    else:
        data, scales = out
        _check_f8_out(data, scales, dtype, device, R, K, rows)
        pitch, (ss_r, ss_k) = data.stride(0) if R > 1 else K, scales.stride()
    _call(device, stream, _c_quantize, _quantize_args(x.data_ptr(), sr, sk, R, K, data.data_ptr(), pitch,
                                                      scales.data_ptr(), ss_r, ss_k, fmt, fmt8, rows))
    if stream is not None:
        _keep(stream, x, data, scales)
    return data, scales


def gemm_f8_scaled(a, a_scales, b, b_scales, out=None, dtype=None, variant="auto", stream=None):
    """C [M, N] = a . b^T of 8-bit a [M, K] in row blocks and b [N, K] (weights as
    rows) in row or square blocks, each float8_e4m3fn or float8_e5m2, with float32
    sums; C in dtype (float16, bfloat16 or float32; bfloat16, or out's).

    b_scales [N, ceil(K/128)] are row blocks', [ceil(N/128), ceil(K/128)] square
    blocks'; both scales with any positive strides (up to 2^21 from row to row).  a
    and b have unit stride along K, and rows that start 16-byte aligned (as
    quantize_f8 makes them), at most 2^23 bytes apart.

    Sums are float32; for a 16-bit C the FP8 matrix instructions cut products that
    are added together at 2^-13 of the largest of eight (1 to 3 in 10^5 of a sum of
    random products), for a float32 C nothing is cut, at about half the rate (and
    rounded by the caller, that is a 16-bit result without cuts).  Scales may be any
    float32, also where the product of two is not one; results above 2^88 are formed
    twice, the second time slowly.

    variant: a kernel by its tile (VARIANTS), for measurements; all compute the
    same."""
    fmt_a, fmt_b, device = FORMATS8.get(a.dtype), FORMATS8.get(b.dtype), a.device
    if fmt_a is None or fmt_b is None or a_scales.dtype != torch.float32 or b_scales.dtype != torch.float32:
        raise TypeError("a and b must be float8_e4m3fn or float8_e5m2, with float32 scales")
    if a.ndim != 2 or b.ndim != 2 or a_scales.ndim != 2 or b_scales.ndim != 2:
        raise ValueError("expected matrices a, a_scales, b and b_scales")
    if device.type != "cuda" or b.device != device or a_scales.device != device or b_scales.device != device:
        raise ValueError("inputs must share one GPU device")
    if stream is not None:
        _check_stream(stream, device)
    (M, K), (N, Kb) = a.shape, b.shape
    if K != Kb or M <= 0 or N <= 0 or K <= 0:
        raise ValueError("incompatible or empty shape")
    blocks, brows = -(-K // BLOCK), b_scales.shape[0]
    if a_scales.shape != (M, blocks) or b_scales.shape[1] != blocks or brows not in (N, -(-N // BLOCK)):
        raise ValueError("scales must be [M, ceil(K/128)] for a, [N, ceil(K/128)] or [ceil(N/128), ceil(K/128)] for b")
    (lda, ka), (ldb, kb) = a.stride(), b.stride()
    sa, sb = a_scales.stride(), b_scales.stride()
    if K > 1 and (ka != 1 or kb != 1):
        raise ValueError("a and b must have unit stride along K")
    if min(sa) <= 0 or min(sb) <= 0 or lda <= 0 or ldb <= 0:
        raise ValueError("strides must be positive")
    if out is None:
        dtype = dtype or torch.bfloat16
        if dtype not in FORMATS:
            raise TypeError("dtype must be float16, bfloat16 or float32")
        out, ldc = _new2(M, N, dtype, device, stream), N
    else:
        if out.dtype not in FORMATS or (dtype is not None and out.dtype != dtype):
            raise TypeError("out must be float16, bfloat16 or float32, and of dtype where that is given")
        if out.device != device or out.shape != (M, N) or (out.stride(1) != 1 and N > 1) or \
                (out.stride(0) < N and M > 1):
            raise ValueError("out must be a row-major [M, N] tensor on the inputs' device")
        ldc = out.stride(0) if M > 1 else N
    _call(device, stream, _c_product,
          _product_args(a.data_ptr(), lda, a_scales.data_ptr(), *sa, b.data_ptr(), ldb, b_scales.data_ptr(), *sb,
                        out.data_ptr(), ldc, M, N, K, fmt_a, fmt_b, 1 if brows == N else BLOCK, FORMATS[out.dtype],
                        VARIANTS[variant]))
    if stream is not None:
        _keep(stream, a, a_scales, b, b_scales, out)
    return out
