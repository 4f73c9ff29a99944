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

from ._lib import lib
from .mx4 import FORMATS, _call, _check_stream, _given, _keep, _new, _workspace

MAX_EXPERTS, MAX_TOKENS, MAX_PAIRS = 1024, 1 << 23, 1 << 31

_c_bytes = lib.gemm_moe_sort_workspace_bytes


def _c_sort(*args):
    # the stream comes before the workspace
    return lib.gemm_moe_sort(*args[:-3], args[-1], args[-3], args[-2])


class MoeOrder(NamedTuple):
    """Pairs (token t, choice j), numbered t * top_k + j, sorted by expert and
    within an expert by number.

    offsets  int64 [E + 1]: expert e has the slots offsets[e] .. offsets[e+1]-1
    rows     int64 [T * top_k]: number of the pair in a slot; -1 from offsets[E] on
    slots    int64 [T, top_k]: slot of a pair, -1 without one"""
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
    if (experts.stride(1) != 1 and k > 1) or experts.stride(0) <= 0:
        raise ValueError("experts must have unit stride along top_k and a positive row stride")
    if stream is not None:
        _check_stream(stream, device)
    # one allocation for the three tables
    table = _new((2 * T * k + E + 1,), torch.int64, device, stream)
    order = MoeOrder(table[2 * T * k:], table[:T * k], table[T * k:2 * T * k].view(T, k))
    if workspace is None:
        need = _c_bytes(T, k, E)
        if need:
            workspace = _workspace(need, device, stream)
    ws, nws = _given(workspace, device) if workspace is not None else (0, 0)
    p = table.data_ptr()
    _call(device, stream, _c_sort, experts.data_ptr(), experts.element_size(), experts.stride(0) if T > 1 else k, T, k,
          E, p + 16 * T * k, p, p + 8 * T * k, ws, nws)
    if stream is not None:
        _keep(stream, experts, table, workspace)
    return order


def _check_order(order, device):
    """(T, top_k, E) of an order on `device`."""
    offsets, _, slots = order
    if offsets.dtype != torch.int64 or slots.dtype != torch.int64:
        raise TypeError("an order's tables are int64")
    if offsets.device != device or slots.device != device:
        raise ValueError("inputs must share one GPU device")
    if offsets.ndim != 1 or offsets.shape[0] < 2 or slots.ndim != 2 or not slots.is_contiguous() or \
            offsets.stride(0) != 1:
        raise ValueError("an order's offsets must be [E + 1] and its slots [T, top_k], both contiguous")
    T, k = slots.shape
    if T <= 0 or k <= 0 or T >= MAX_TOKENS or T * k >= MAX_PAIRS:
        raise ValueError("empty or oversized shape")
    return T, k, offsets.shape[0] - 1


def _check_matrix(t, rows, name):
    """H of a [rows, H] matrix with unit stride along H."""
    if t.ndim != 2 or not t.is_cuda or t.shape[0] != rows or t.shape[1] <= 0:
        raise ValueError(f"{name} must be a [{rows}, H] matrix on a GPU")
    if (t.stride(1) != 1 and t.shape[1] > 1) or t.stride(0) <= 0:
        raise ValueError(f"{name} must have unit stride along H and a positive row stride")
    return t.shape[1]


def _check_weights(weights, y, T, k):
    if weights.dtype not in (y.dtype, torch.float32):
        raise TypeError("weights must be float32 or of the rows' dtype")
    if weights.device != y.device or weights.shape != (T, k) or (weights.stride(1) != 1 and k > 1) or \
            weights.stride(0) <= 0:
        raise ValueError("weights must be [T, top_k] with unit stride along top_k on the rows' device")


def _out(out, shape, like, stream):
    """(tensor, row stride) of an output of like's dtype."""
    if out is None:
        return _new(shape, like.dtype, like.device, stream), shape[1]
    if out.dtype != like.dtype or out.device != like.device or out.shape != shape or \
            (out.stride(1) != 1 and shape[1] > 1) or (out.stride(0) < shape[1] and shape[0] > 1):
        raise ValueError(f"out must be a row-major {list(shape)} tensor of the rows' dtype on their device")
    return out, out.stride(0) if shape[0] > 1 else shape[1]


def moe_gather(x, order, out=None, stream=None):
    """[T * top_k, H] of x [T, H]'s rows sorted by expert: row order.slots[t, j]
    is x[t]; rows from order.offsets[E] on are zeros.  Any dtype of 1, 2 or 4
    bytes, so 8-bit rows and their scales too."""
    T, k, E = _check_order(order, x.device)
    H, size = _check_matrix(x, T, "x"), x.element_size()
    if size not in (1, 2, 4):
        raise TypeError("elements must have 1, 2 or 4 bytes")
    if stream is not None:
        _check_stream(stream, x.device)
    out, ldo = _out(out, (T * k, H), x, stream)
    _call(x.device, stream, lib.gemm_moe_gather, x.data_ptr(), x.stride(0), size, order.offsets.data_ptr(),
          order.slots.data_ptr(), E, out.data_ptr(), ldo, T, k, H)
    if stream is not None:
        _keep(stream, x, order.offsets, order.slots, out)
    return out


def moe_combine(y, order, weights=None, out=None, stream=None):
    """[T, H]: for each token the sum over its choices j of weights[t, j] *
    y[order.slots[t, j]], in float32 and in the order of j; choices without a slot
    count nothing.  y [T * top_k, H] float16, bfloat16 or float32; weights [T,
    top_k] of its dtype or float32, or None for ones (moe_gather's gradient)."""
    T, k, _ = _check_order(order, y.device)
    H, fmt = _check_matrix(y, T * k, "y"), FORMATS.get(y.dtype)
    if fmt is None:
        raise TypeError("y must be float16, bfloat16 or float32")
    if stream is not None:
        _check_stream(stream, y.device)
    wp, wf, ldw = 0, fmt, 0
    if weights is not None:
        _check_weights(weights, y, T, k)
        wp, wf, ldw = weights.data_ptr(), FORMATS[weights.dtype], weights.stride(0)
    out, ldo = _out(out, (T, H), y, stream)
    _call(y.device, stream, lib.gemm_moe_combine, y.data_ptr(), y.stride(0), fmt, order.slots.data_ptr(), wp, wf, ldw,
          out.data_ptr(), ldo, T, k, H)
    if stream is not None:
        _keep(stream, y, order.slots, weights, out)
    return out


def moe_combine_backward(dout, y, order, weights, out=None, stream=None):
    """(dy, dweights) of moe_combine, given its result's gradient dout [T, H]:
    dy[order.slots[t, j]] = weights[t, j] * dout[t], zeros from order.offsets[E]
    on, and dweights[t, j] = sum of dout[t] * y[order.slots[t, j]] in float32, zero
    without a slot.  dout and y of one dtype (float16, bfloat16 or float32)."""
    T, k, E = _check_order(order, y.device)
    H, fmt = _check_matrix(y, T * k, "y"), FORMATS.get(y.dtype)
    if fmt is None or dout.dtype != y.dtype:
        raise TypeError("dout and y must both be float16, bfloat16 or float32")
    if dout.device != y.device or _check_matrix(dout, T, "dout") != H:
        raise ValueError("dout must be [T, H] on y's device")
    _check_weights(weights, y, T, k)
    if stream is not None:
        _check_stream(stream, y.device)
    out, ldo = _out(out, (T * k, H), y, stream)
    dw = _new((T, k), weights.dtype, y.device, stream)
    _call(y.device, stream, lib.gemm_moe_combine_backward, dout.data_ptr(), dout.stride(0), y.data_ptr(), y.stride(0),
          fmt, order.offsets.data_ptr(), order.slots.data_ptr(), E, weights.data_ptr(), FORMATS[weights.dtype],
          weights.stride(0), out.data_ptr(), ldo, dw.data_ptr(), k, T, k, H)
    if stream is not None:
        _keep(stream, dout, y, order.offsets, order.slots, weights, out, dw)
    return out, dw
