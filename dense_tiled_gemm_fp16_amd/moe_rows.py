"""Tokens sorted by expert and back: what stands before and behind gemm_grouped
in a mixture-of-experts layer, with the gradients.  Argument marshalling for
include/gemm_moe_rows.h; the computation runs in the HIP library.

    moe_sort(experts, E)                          -> MoeOrder(offsets, rows, slots)
    moe_gather(x, order)                          -> [T * top_k, H], sorted by expert
    moe_combine(y, order, weights)                -> [T, H]
    moe_combine_backward(dout, y, order, weights) -> dy, dweights
    moe_sort_workspace_bytes(T, top_k, E)

A layer of more tokens than gemm_moe takes:

    order = moe_sort(experts, E)                          # experts [T, top_k]
    a = moe_gather(x, order)
    y = gemm_grouped(act(gemm_grouped(a, w_up, order.offsets)), w_down, order.offsets)
    out = moe_combine(y, order, weights)

and its backward pass: moe_combine_backward gives the gradients of y and of the
weights, moe_combine(da, order) that of x.

A stream by argument: as the package says.
"""
from typing import NamedTuple

import torch

from ._lib import CombineArgs, CombineBackwardArgs, GatherArgs, SortArgs, lib, packer
from .mx4 import FORMATS, _call, _check_stream, _given, _keep, _new, _new2, _workspace

MAX_EXPERTS, MAX_TOKENS, MAX_PAIRS = 1024, 1 << 23, 1 << 31

_c_bytes = lib.gemm_moe_sort_workspace_bytes


_c_gather, _c_combine, _c_back = lib.gemm_moe_gather, lib.gemm_moe_combine, lib.gemm_moe_combine_backward
_sort_args, _gather_args, _combine_args, _back_args = map(packer, (SortArgs, GatherArgs, CombineArgs,
                                                                   CombineBackwardArgs))


def _c_sort(args, workspace, nbytes, stream):
    # the stream comes before the workspace
    return lib.gemm_moe_sort(args, stream, workspace, nbytes)


class MoeOrder(NamedTuple):
    """Pairs (token t, choice j), numbered t * top_k + j, sorted by expert and
    within an expert by number.

    offsets  int64 [E + 1]: expert e has the slots offsets[e] .. offsets[e+1]-1
    rows     int64 [T * top_k]: number of the pair in a slot; -1 from offsets[E] on
    slots    int64 [T, top_k]: slot of a pair, -1 without one

    One that moe_sort did not make has to keep to this: of pairs that share a slot, or
    whose slot is offsets[E] or above, moe_gather and moe_combine_backward leave any, or
    parts of each."""
    offsets: torch.Tensor
    rows: torch.Tensor
    slots: torch.Tensor


def moe_sort_workspace_bytes(T, top_k, E):
    """Bytes of workspace moe_sort of these sizes needs."""
    return int(_c_bytes(T, top_k, E))


def moe_sort(experts, E, workspace=None, stream=None):
    """The MoeOrder of experts [T, top_k] (int32 or int64, unit stride along
    top_k), E at most 1024.  A pair whose expert is outside 0 .. E - 1, such as a
    padded token's -1, has no slot; an expert may be chosen twice by one token.

    workspace: moe_sort_workspace_bytes(T, top_k, E) bytes, 256-byte aligned, not
    shared with a call that may overlap; allocated here when not given."""
    if experts.dtype not in (torch.int32, torch.int64):
        raise TypeError("experts must be int32 or int64")
    device = experts.device
    if experts.ndim != 2 or not experts.is_cuda:
        raise ValueError("expected experts [T, top_k] on a GPU")
    T, k = experts.shape
    if T <= 0 or k <= 0 or T >= MAX_TOKENS or T * k >= MAX_PAIRS or not 1 <= E <= MAX_EXPERTS:
        raise ValueError(f"empty or oversized shape, or E outside 1 .. {MAX_EXPERTS}")
    ld, one = experts.stride()
    if (one != 1 and k > 1) or ld <= 0:
        raise ValueError("experts must have unit stride along top_k and a positive row stride")
    if stream is not None:
        _check_stream(stream, device)
    offsets = _new(E + 1, torch.int64, device, stream)
    rows = _new(T * k, torch.int64, device, stream)
    slots = _new2(T, k, torch.int64, device, stream)
    if workspace is None:
        need = _c_bytes(T, k, E)
        if need:
            workspace = _workspace(need, device, stream)
    ws, nws = _given(workspace, device) if workspace is not None else (0, 0)
    _call(device, stream, _c_sort, _sort_args(experts.data_ptr(), ld if T > 1 else k, T, offsets.data_ptr(),
                                              rows.data_ptr(), slots.data_ptr(), experts.element_size(), k, E), ws, nws)
    if stream is not None:
        _keep(stream, experts, offsets, rows, slots, workspace)
    return MoeOrder(offsets, rows, slots)


def _check_order(order, device):
    """(offsets, slots, T, top_k, E) of an order on `device`."""
    offsets, _, slots = order
    if offsets.dtype != torch.int64 or slots.dtype != torch.int64:
        raise TypeError("an order's tables are int64")
    if offsets.device != device or slots.device != device:
        raise ValueError("inputs must share one GPU device")
    shape = slots.shape
    if offsets.ndim != 1 or len(shape) != 2 or not slots.is_contiguous() or not offsets.is_contiguous():
        raise ValueError("an order's offsets must be [E + 1] and its slots [T, top_k], both contiguous")
    (T, k), E = shape, offsets.shape[0] - 1
    if T <= 0 or k <= 0 or E <= 0 or T >= MAX_TOKENS or T * k >= MAX_PAIRS:
        raise ValueError("empty or oversized shape")
    return offsets, slots, T, k, E


def _check_matrix(t, rows, name):
    """(H, row stride) of a [rows, H] matrix with unit stride along H."""
    shape = t.shape
    if len(shape) != 2 or t.device.type != "cuda" or shape[0] != rows or shape[1] <= 0:
        raise ValueError(f"{name} must be a [{rows}, H] matrix on a GPU")
    ld, one = t.stride()
    if (one != 1 and shape[1] > 1) or ld <= 0:
        raise ValueError(f"{name} must have unit stride along H and a positive row stride")
    return shape[1], ld


def _check_weights(weights, y, T, k):
    """(format, row stride) of weights [T, top_k]."""
    if weights.dtype != torch.float32 and weights.dtype != y.dtype:
        raise TypeError("weights must be float32 or of the rows' dtype")
    if weights.device != y.device or weights.shape != (T, k):
        raise ValueError("weights must be [T, top_k] on the rows' device")
    ld, one = weights.stride()
    if (one != 1 and k > 1) or ld <= 0:
        raise ValueError("weights must have unit stride along top_k and a positive row stride")
    return FORMATS[weights.dtype], ld


def _out(out, rows, H, like, stream):
    """(tensor, row stride) of an output of like's dtype."""
    if out is None:
        return _new2(rows, H, like.dtype, like.device, stream), H
    if out.dtype != like.dtype or out.device != like.device or out.shape != (rows, H) or \
            (out.stride(1) != 1 and H > 1) or (out.stride(0) < H and rows > 1):
        raise ValueError(f"out must be a row-major [{rows}, {H}] tensor of the rows' dtype on their device")
    return out, out.stride(0) if rows > 1 else H


def moe_gather(x, order, out=None, stream=None):
    """[T * top_k, H] of x [T, H]'s rows sorted by expert: row order.slots[t, j]
    is x[t]; rows from order.offsets[E] on are zeros.  Any dtype of 1, 2 or 4
    bytes, so 8-bit rows too (which gemm_grouped takes without scales), or scales."""
    device, size = x.device, x.element_size()
    offsets, slots, T, k, E = _check_order(order, device)
    H, ld = _check_matrix(x, T, "x")
    if size not in (1, 2, 4):
        raise TypeError("elements must have 1, 2 or 4 bytes")
    if stream is not None:
        _check_stream(stream, device)
    out, ldo = _out(out, T * k, H, x, stream)
    _call(device, stream, _c_gather, _gather_args(x.data_ptr(), ld, offsets.data_ptr(), slots.data_ptr(),
                                                  out.data_ptr(), ldo, T, H, size, E, k))
    if stream is not None:
        _keep(stream, x, offsets, slots, out)
    return out


def moe_combine(y, order, weights=None, out=None, stream=None):
    """[T, H]: for each token the sum over its choices j of weights[t, j] *
    y[order.slots[t, j]], in float32 and in the order of j; choices without a slot
    count nothing.  y [T * top_k, H] float16, bfloat16 or float32; weights [T,
    top_k] of its dtype or float32, or None for ones (moe_gather's gradient)."""
    device, fmt = y.device, FORMATS.get(y.dtype)
    _, slots, T, k, _ = _check_order(order, device)
    H, ld = _check_matrix(y, T * k, "y")
    if fmt is None:
        raise TypeError("y must be float16, bfloat16 or float32")
    if stream is not None:
        _check_stream(stream, device)
    wp, wf, ldw = 0, fmt, 0
    if weights is not None:
        wf, ldw = _check_weights(weights, y, T, k)
        wp = weights.data_ptr()
    out, ldo = _out(out, T, H, y, stream)
    _call(device, stream, _c_combine, _combine_args(y.data_ptr(), ld, slots.data_ptr(), wp, ldw, out.data_ptr(), ldo, T,
                                                    H, fmt, wf, k))
    if stream is not None:
        _keep(stream, y, slots, weights, out)
    return out


def moe_combine_backward(dout, y, order, weights, out=None, stream=None):
    """(dy, dweights) of moe_combine, given its result's gradient dout [T, H]:
    dy[order.slots[t, j]] = weights[t, j] * dout[t], zeros from order.offsets[E]
    on, and dweights[t, j] = sum of dout[t] * y[order.slots[t, j]] in float32, zero
    without a slot.  dout and y of one dtype (float16, bfloat16 or float32)."""
    device, fmt = y.device, FORMATS.get(y.dtype)
    offsets, slots, T, k, E = _check_order(order, device)
    H, ld = _check_matrix(y, T * k, "y")
    if fmt is None or dout.dtype != y.dtype:
        raise TypeError("dout and y must both be float16, bfloat16 or float32")
    Hd, ldd = _check_matrix(dout, T, "dout")
    if dout.device != device or Hd != H:
        raise ValueError("dout must be [T, H] on y's device")
    wf, ldw = _check_weights(weights, y, T, k)
    if stream is not None:
        _check_stream(stream, device)
    out, ldo = _out(out, T * k, H, y, stream)
    dw = _new2(T, k, weights.dtype, device, stream)
    _call(device, stream, _c_back, _back_args(dout.data_ptr(), ldd, y.data_ptr(), ld, offsets.data_ptr(),
                                              slots.data_ptr(), weights.data_ptr(), ldw, out.data_ptr(), ldo,
                                              dw.data_ptr(), k, T, H, fmt, wf, E, k))
    if stream is not None:
        _keep(stream, dout, y, offsets, slots, weights, out, dw)
    return out, dw
