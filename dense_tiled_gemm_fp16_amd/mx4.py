"""Microscaled 4-bit floating point (OCP MX FP4): quantisation and products
with 4-bit weights.  Argument marshalling for include/gemm_mx4.h; the
computation runs in the HIP library.

    MX4(data, scales, K)          -> a matrix (or a stack of them) in 4 bits
    quantize_mx4(x)               -> MX4 of x [R, K] or [G, R, K], along the last axis
    dequantize_mx4(q, dtype)      -> its values
    gemm_mx4(a, b)                -> C [M, N] = a . b^T, b MX4 [N, K], a MX4 [M, K]
                                     or float16 / bfloat16 [M, K]
    gemm_mx4_workspace_bytes(M, N, K)
"""
import contextlib

import torch

from ._lib import GEMM_OK, lib

# Element formats of the C calls (enum gemm_mx4_format).
FORMATS = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
BLOCK = 32


def _error(rc):
    from . import GemmError
    return GemmError(rc)


def _device(device):
    """The device made current for a call; nothing to do where it is already."""
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _stream(stream, device):
    return (stream if stream is not None else torch.cuda.current_stream(device)).cuda_stream


class MX4:
    """A matrix in microscaled 4-bit floating point, [R, K] or a stack
    [G, R, K], quantised along K in blocks of 32.

    data    uint8 [..., R, 16 * ceil(K/32)]: element k in the low (even k) or
            high (odd k) half of byte k/2; a sign bit and +-{0, 0.5, 1, 1.5, 2,
            3, 4, 6}
    scales  uint8 [..., R, ceil(K/32)]: the block's factor is 2^(scale - 127),
            255 a NaN

    Both have unit stride along the last axis; data rows start 16-byte aligned.
    Slices of rows and of the stack are views (q[g], q[g, r0:r1], q[r0:r1])."""

    def __init__(self, data, scales, K):
        blocks = -(-K // BLOCK)
        if data.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("data and scales must be uint8")
        if data.ndim not in (2, 3) or scales.ndim != data.ndim or scales.shape[:-1] != data.shape[:-1]:
            raise ValueError("data and scales must be [R, ...] or [G, R, ...] with the same rows")
        if K <= 0 or data.shape[-1] != 16 * blocks or scales.shape[-1] != blocks:
            raise ValueError("data must have 16 * ceil(K/32) columns and scales ceil(K/32)")
        if data.device != scales.device:
            raise ValueError("data and scales must share one device")
        if data.stride(-1) != 1 or (scales.stride(-1) != 1 and blocks > 1):
            raise ValueError("data and scales must have unit stride along the last axis")
        self.data, self.scales, self.K = data, scales, K

    @property
    def shape(self):
        return torch.Size((*self.data.shape[:-1], self.K))

    @property
    def ndim(self):
        return self.data.ndim

    @property
    def device(self):
        return self.data.device

    def __getitem__(self, rows):
        return MX4(self.data[rows], self.scales[rows], self.K)

    def __repr__(self):
        return f"MX4(shape={tuple(self.shape)}, device={self.device})"


def quantize_mx4(x, out=None, stream=None):
    """x [R, K] or [G, R, K] (float16, bfloat16 or float32, any positive
    strides) in MX4, quantised along K.

    A block's scale is 2^(floor(log2 m) - 2), m its largest magnitude (at least
    2^-127); elements round to nearest, ties to the even code, and saturate at
    6 scales.  A block with an infinity or a NaN becomes NaN.  The elements
    past K of the last block are zero.  out: an MX4 of x's shape with
    contiguous data and scales."""
    if x.dtype not in FORMATS:
        raise TypeError("expected float16, bfloat16 or float32")
    if x.ndim not in (2, 3) or not x.is_cuda:
        raise ValueError("expected an [R, K] matrix or a [G, R, K] stack on a GPU")
    if min(x.shape) <= 0:
        raise ValueError("empty shape")
    if min(x.stride()) <= 0:
        raise ValueError("strides must be positive")
    K = x.shape[-1]
    blocks = -(-K // BLOCK)
    if out is None:
        out = MX4(torch.empty((*x.shape[:-1], 16 * blocks), dtype=torch.uint8, device=x.device),
                  torch.empty((*x.shape[:-1], blocks), dtype=torch.uint8, device=x.device), K)
    elif out.shape != x.shape or out.device != x.device or not out.data.is_contiguous() or \
            not out.scales.is_contiguous():
        raise ValueError("out must be an MX4 of x's shape on its device, contiguous")
    G, sg = (x.shape[0], x.stride(0)) if x.ndim == 3 else (1, 1)
    with _device(x.device):
        rc = lib.gemm_mx4_quantize(x.data_ptr(), FORMATS[x.dtype], sg, x.stride(-2), x.stride(-1), G,
                                   x.shape[-2], K, out.data.data_ptr(), out.scales.data_ptr(),
                                   _stream(stream, x.device))
    if rc != GEMM_OK:
        raise _error(rc)
    return out


def dequantize_mx4(q, dtype=torch.bfloat16, out=None, stream=None):
    """The values of an MX4 matrix or stack, each rounded once to dtype
    (float16, bfloat16 or float32).  out: of q's shape, contiguous, or for a
    matrix row-major with any row stride."""
    if dtype not in FORMATS:
        raise TypeError("dtype must be float16, bfloat16 or float32")
    if not q.data.is_cuda or min(q.shape) <= 0:
        raise ValueError("expected a non-empty MX4 on a GPU")
    if out is None:
        out = torch.empty(q.shape, dtype=dtype, device=q.device)
    elif out.dtype != dtype or out.device != q.device or out.shape != q.shape or out.stride(-1) != 1 or \
            (out.ndim == 3 and not out.is_contiguous()):
        raise ValueError("out must be of q's shape, of dtype, on its device, with unit column stride "
                         "(a stack contiguous)")
    if q.ndim == 3 and not (q.data.is_contiguous() and q.scales.is_contiguous()):
        for i in range(q.shape[0]):
            dequantize_mx4(q[i], dtype, out[i], stream)
        return out
    R = q.shape[0] * q.shape[1] if q.ndim == 3 else q.shape[0]
    with _device(q.device):
        rc = lib.gemm_mx4_dequantize(q.data.data_ptr(), q.data.stride(-2), q.scales.data_ptr(),
                                     q.scales.stride(-2), R, q.K, out.data_ptr(), FORMATS[dtype],
                                     out.stride(-2), _stream(stream, q.device))
    if rc != GEMM_OK:
        raise _error(rc)
    return out


def gemm_mx4_workspace_bytes(M, N, K):
    """Bytes of workspace gemm_mx4 of an MX4 a [M, K] and b [N, K] needs."""
    return int(lib.gemm_mx4_workspace_bytes(M, N, K))


def gemm_mx4(a, b, out=None, dtype=None, workspace=None, stream=None):
    """C [M, N] = a . b^T with fp32 accumulation, b an MX4 [N, K] (weights as
    rows).

    a an MX4 [M, K]: C in dtype (float16, the default, or bfloat16), on the
    scaled 4-bit matrix instructions.
    a float16 or bfloat16 [M, K] with unit stride along K: C in a's dtype, the
    weights exact; made for few rows (beyond some 64, quantise a first).

    workspace: gemm_mx4_workspace_bytes(M, N, K) bytes, 256-byte aligned, not
    shared with a call that may overlap; allocated here when not given."""
    if not isinstance(b, MX4) or b.ndim != 2 or a.ndim != 2:
        raise ValueError("expected a matrix a and an MX4 matrix b [N, K]")
    if not b.data.is_cuda or a.device != b.device:
        raise ValueError("inputs must share one GPU device")
    (M, K), (N, Kb) = a.shape, b.shape
    if K != Kb or min(M, N, K) <= 0:
        raise ValueError("incompatible or empty shape")
    if isinstance(a, MX4):
        dtype = dtype or torch.float16
        if dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("dtype must be float16 or bfloat16")
    else:
        if a.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("a must be an MX4, float16 or bfloat16 matrix")
        if dtype not in (None, a.dtype):
            raise TypeError("the output of a 16-bit a has its dtype")
        dtype = a.dtype
        if (a.stride(1) != 1 and K > 1) or a.stride(0) <= 0:
            raise ValueError("a must have unit stride along K and a positive row stride")
    if out is None:
        out = torch.empty((M, N), dtype=dtype, device=b.device)
    elif out.dtype != dtype or out.device != b.device or out.shape != (M, N) or out.stride(1) != 1 or \
            out.stride(0) < N:
        raise ValueError("out must be a row-major [M, N] tensor of the output dtype on the inputs' device")
    with _device(b.device):
        if isinstance(a, MX4):
            need = lib.gemm_mx4_workspace_bytes(M, N, K)
            if need and workspace is None:
                with torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext():
                    workspace = torch.empty(need, dtype=torch.uint8, device=b.device)
            ws, nws = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) \
                if workspace is not None else (0, 0)
            rc = lib.gemm_mx4(a.data.data_ptr(), a.data.stride(0), a.scales.data_ptr(), a.scales.stride(0),
                              b.data.data_ptr(), b.data.stride(0), b.scales.data_ptr(), b.scales.stride(0),
                              out.data_ptr(), FORMATS[dtype], out.stride(0), M, N, K,
                              _stream(stream, b.device), ws, nws)
        else:
            rc = lib.gemm_mx4_a16(a.data_ptr(), FORMATS[dtype], a.stride(0), b.data.data_ptr(),
                                  b.data.stride(0), b.scales.data_ptr(), b.scales.stride(0),
                                  out.data_ptr(), out.stride(0), M, N, K, _stream(stream, b.device))
    if rc != GEMM_OK:
        raise _error(rc)
    return out
