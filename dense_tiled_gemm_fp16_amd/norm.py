"""Root-mean-square norm with the residual's addition and its result in 8 bits
(the input of gemm_f8_scaled), and the norm's gradients.  Argument marshalling
for include/rms_norm_f8.h; the computation runs in the HIP library.

    rms_norm_f8(x, weight, eps, residual)        -> data [R, K], scales, h [R, K]
    rms_norm_backward(dy, h, weight, eps, dh)    -> dx [R, K], dweight [K]
    rms_norm_backward_workspace_bytes(R, K)

A stream by argument: as the package says.
"""
import torch

from ._lib import lib
from .f8_scaled import BLOCK, FORMATS8, _check_f8_out, _new_f8
from .mx4 import FORMATS, _call, _check_stream, _given, _keep, _new, _workspace

MAX_K = 65536

_c_norm, _c_bytes = lib.gemm_rms_norm_f8, lib.gemm_rms_norm_backward_workspace_bytes


def _c_backward(*args):
    # the stream comes before the workspace
    return lib.gemm_rms_norm_backward(*args[:-3], args[-1], args[-3], args[-2])


def _check_rows(x, weight, eps, *others):
    fmt = FORMATS.get(x.dtype)
    if fmt is None or fmt == FORMATS[torch.float32] or weight.dtype not in (x.dtype, torch.float32):
        raise TypeError("rows must be float16 or bfloat16, weight of their dtype or float32")
    if x.ndim != 2 or not x.is_cuda or weight.device != x.device:
        raise ValueError("expected an [R, K] matrix and a weight on one GPU device")
    R, K = x.shape
    if R <= 0 or K <= 0 or K > MAX_K:
        raise ValueError(f"empty shape, or rows of more than {MAX_K} elements")
    if weight.shape != (K,) or (weight.stride(0) != 1 and K > 1):
        raise ValueError("weight must be a contiguous [K] vector")
    if not eps >= 0:
        raise ValueError("eps must not be negative")
    for t in others:
        if t is not None and (t.dtype != x.dtype or t.device != x.device or t.shape != x.shape):
            raise ValueError("all rows must have one shape, dtype and device")
    for t in (x, *others):
        if t is not None and ((t.stride(1) != 1 and K > 1) or t.stride(0) <= 0):
            raise ValueError("rows must have unit stride along K and a positive row stride")
    return R, K, fmt


def _rows_out(out, x, R, K, stream):
    """(tensor, row stride) of an output like x."""
    if out is None:
        return _new((R, K), x.dtype, x.device, stream), K
    if out.dtype != x.dtype or out.device != x.device or out.shape != (R, K) or (out.stride(1) != 1 and K > 1) or \
            (out.stride(0) < K and R > 1):
        raise ValueError("out must be a row-major [R, K] tensor of the rows' dtype on their device")
    return out, out.stride(0) if R > 1 else K


def rms_norm_f8(x, weight, eps=1e-6, residual=None, dtype=torch.float8_e4m3fn, out=None, h=None, stream=None):
    """(data, scales, h): h = x + residual rounded to x's dtype (x itself without
    a residual), and h * weight / sqrt(mean(h^2) + eps) along K quantised to dtype
    (float8_e4m3fn or float8_e5m2) by row blocks, as quantize_f8 does it.

    x, residual [R, K] float16 or bfloat16, unit stride along K, K at most 65536;
    weight [K] of their dtype or float32.  Sums are float32.
    out: a pair (data, scales); h: where the sum goes, which may be x or residual
    themselves."""
    R, K, fmt = _check_rows(x, weight, eps, residual)
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
        h, ldh = _rows_out(h, x, R, K, stream)
        hp, rp, ldr = h.data_ptr(), residual.data_ptr(), residual.stride(0)
    if out is None:
        data = _new_f8(R, K, dtype, device, stream)
        scales = _new((R, -(-K // BLOCK)), torch.float32, device, stream)
    else:
        data, scales = out
        _check_f8_out(data, scales, dtype, device, R, K, 1)
    _call(device, stream, _c_norm, x.data_ptr(), x.stride(0), rp, ldr, fmt, weight.data_ptr(), FORMATS[weight.dtype],
          eps, hp, ldh, data.data_ptr(), fmt8, data.stride(0) if R > 1 else K, scales.data_ptr(), *scales.stride(),
          R, K)
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
    Sums are float32, in a fixed order.

    dy, h, dh [R, K] float16 or bfloat16, unit stride along K, K at most 65536.
    out: where dx goes, which may be dy or dh themselves.
    workspace: rms_norm_backward_workspace_bytes(R, K) bytes, 256-byte aligned, not
    shared with a call that may overlap; allocated here when not given."""
    R, K, fmt = _check_rows(h, weight, eps, dy, dh)
    device = h.device
    if stream is not None:
        _check_stream(stream, device)
    dx, lddx = _rows_out(out, h, R, K, stream)
    dw = _new((K,), weight.dtype, device, stream)
    if workspace is None:
        workspace = _workspace(_c_bytes(R, K), device, stream)
    _call(device, stream, _c_backward, dy.data_ptr(), dy.stride(0), h.data_ptr(), h.stride(0), fmt, weight.data_ptr(),
          FORMATS[weight.dtype], eps, dh.data_ptr() if dh is not None else 0, dh.stride(0) if dh is not None else 0,
          dx.data_ptr(), lddx, dw.data_ptr(), R, K, *_given(workspace, device))
    if stream is not None:
        _keep(stream, dy, h, weight, dh, dx, dw, workspace)
    return dx, dw
