"""Root-mean-square norm with the residual's addition and its result in 8 bits
(the input of gemm_f8_scaled), and the norm's gradients.  Argument marshalling
for include/rms_norm_f8.h; the computation runs in the HIP library.

    rms_norm_f8(x, weight, eps, residual)        -> data [R, K], scales, h [R, K]
    rms_norm_backward(dy, h, weight, eps, dh)    -> dx [R, K], dweight [K]
    rms_norm_backward_workspace_bytes(R, K)

A stream by argument: as the package says.
"""
import torch

from ._lib import NormArgs, NormBackwardArgs, lib, packer
from .f8_scaled import BLOCK, FORMATS8, _check_f8_out, _new_f8
from .mx4 import FORMATS, _call, _check_stream, _given, _keep, _new, _new2, _workspace

MAX_K = 65536
F32 = FORMATS[torch.float32]

_c_norm, _c_bytes = lib.gemm_rms_norm_f8, lib.gemm_rms_norm_backward_workspace_bytes
_norm_args, _backward_args = packer(NormArgs), packer(NormBackwardArgs)


def _c_backward(args, workspace, nbytes, stream):
    # the stream comes before the workspace
    return lib.gemm_rms_norm_backward(args, stream, workspace, nbytes)


def _check_more(t, x, shape, K):
    """Row stride of further rows like x."""
    if t.dtype != x.dtype or t.device != x.device or t.shape != shape:
        raise ValueError("all rows must have one shape, dtype and device")
    ld, one = t.stride()
    if (one != 1 and K > 1) or ld <= 0:
        raise ValueError("rows must have unit stride along K and a positive row stride")
    return ld


def _check_rows(x, weight, eps):
    """(shape, R, K, row stride, format) of rows x."""
    fmt, device, shape = FORMATS.get(x.dtype), x.device, x.shape
    if fmt is None or fmt == F32 or (weight.dtype != x.dtype and weight.dtype != torch.float32):
        raise TypeError("rows must be float16 or bfloat16, weight of their dtype or float32")
    if len(shape) != 2 or device.type != "cuda" or weight.device != device:
        raise ValueError("expected an [R, K] matrix and a weight on one GPU device")
    R, K = shape
    if R <= 0 or K <= 0 or K > MAX_K:
        raise ValueError(f"empty shape, or rows of more than {MAX_K} elements")
    if weight.shape != (K,) or (K > 1 and weight.stride(0) != 1):
        raise ValueError("weight must be a contiguous [K] vector")
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    ld, one = x.stride()
    if (one != 1 and K > 1) or ld <= 0:
        raise ValueError("rows must have unit stride along K and a positive row stride")
    return shape, R, K, ld, fmt


def _rows_out(out, x, R, K, stream):
    """(tensor, row stride) of an output like x."""
    if out is None:
        return _new2(R, K, x.dtype, x.device, stream), K
    if out.dtype != x.dtype or out.device != x.device or out.shape != (R, K) or (out.stride(1) != 1 and K > 1) or \
            (out.stride(0) < K and R > 1):
        raise ValueError("out must be a row-major [R, K] tensor of the rows' dtype on their device")
    return out, out.stride(0) if R > 1 else K


def rms_norm_f8(x, weight, eps=1e-6, residual=None, dtype=torch.float8_e4m3fn, out=None, h=None, stream=None):
    """(data, scales, h): h = x + residual rounded to x's dtype (x itself without
    a residual), and h * weight / sqrt(mean(h^2) + eps) along K quantised to dtype
    (float8_e4m3fn or float8_e5m2) by row blocks, as quantize_f8 does it.

    x, residual [R, K] float16 or bfloat16, unit stride along K, K at most 65536;
    weight [K] of their dtype or float32.  All is float32: a row whose squares sum
    past 3.4e38 becomes zeros, one whose squares are all 0 has NaN scales if eps is 0.
    out: a pair (data, scales); h: where the sum goes, which may be x or residual
    themselves."""
    shape, R, K, ldx, fmt = _check_rows(x, weight, eps)
    fmt8, device = FORMATS8.get(dtype), x.device
    if fmt8 is None:
        raise TypeError("dtype must be float8_e4m3fn or float8_e5m2")
    if stream is not None:
        _check_stream(stream, device)
    if residual is None:
        if h is not None:
            raise ValueError("h is the sum with a residual")
        hp, ldh, rp, ldr = 0, 0, 0, 0
    else:
        ldr = _check_more(residual, x, shape, K)
        h, ldh = _rows_out(h, x, R, K, stream)
        hp, rp = h.data_ptr(), residual.data_ptr()
    if out is None:
        blocks = -(-K // BLOCK)
        data = _new_f8(R, K, dtype, device, stream)
        scales = _new2(R, blocks, torch.float32, device, stream)
        pitch, ss_r, ss_k = -(-K // 16) * 16, blocks, 1
    else:
        data, scales = out
        _check_f8_out(data, scales, dtype, device, R, K, 1)
        pitch, (ss_r, ss_k) = data.stride(0) if R > 1 else K, scales.stride()
    _call(device, stream, _c_norm,
          _norm_args(x.data_ptr(), ldx, rp, ldr, weight.data_ptr(), hp, ldh, data.data_ptr(), pitch, scales.data_ptr(),
                     ss_r, ss_k, R, K, eps, fmt, FORMATS[weight.dtype], fmt8))
    if stream is not None:
        _keep(stream, x, residual, weight, h, data, scales)
    return data, scales, x if residual is None else h


def rms_norm_backward_workspace_bytes(R, K):
    """Bytes of workspace rms_norm_backward of these sizes needs."""
    return int(_c_bytes(R, K))


def rms_norm_backward(dy, h, weight, eps=1e-6, dh=None, out=None, workspace=None, stream=None):
    """(dx, dweight): the gradients of y = h * weight / sqrt(mean(h^2) + eps),
    given y's (dy [R, K]) and, where h goes on as the residual stream, h's own
    (dh).  dx, which is x's and the residual's gradient alike, has h's dtype,
    dweight weight's; the rounding of y to 8 bits is passed straight through.
    Sums are float32, in a fixed order; where a row's squares sum past 3.4e38, dx is dh
    or NaN.

    dy, h, dh [R, K] float16 or bfloat16, unit stride along K, K at most 65536.
    out: where dx goes, which may be dy or dh themselves.
    workspace: rms_norm_backward_workspace_bytes(R, K) bytes, 256-byte aligned, not
    shared with a call that may overlap; allocated here when not given."""
    shape, R, K, ldh, fmt = _check_rows(h, weight, eps)
    device, ldy, dhp, lddh = h.device, _check_more(dy, h, shape, K), 0, 0
    if dh is not None:
        dhp, lddh = dh.data_ptr(), _check_more(dh, h, shape, K)
    if stream is not None:
        _check_stream(stream, device)
    dx, lddx = _rows_out(out, h, R, K, stream)
    dw = _new(K, weight.dtype, device, stream)
    if workspace is None:
        workspace = _workspace(_c_bytes(R, K), device, stream)
    _call(device, stream, _c_backward,
          _backward_args(dy.data_ptr(), ldy, h.data_ptr(), ldh, weight.data_ptr(), dhp, lddh, dx.data_ptr(), lddx,
                         dw.data_ptr(), R, K, eps, fmt, FORMATS[weight.dtype]), *_given(workspace, device))
    if stream is not None:
        _keep(stream, dy, h, weight, dh, dx, dw, workspace)
    return dx, dw
