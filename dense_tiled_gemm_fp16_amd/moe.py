"""A mixture-of-experts layer for a few tokens (a decode step): routing, the
experts' products and the weighted sum in two kernels.  Argument marshalling
for include/gemm_moe.h; the computation runs in the HIP library.

    gemm_moe(x, logits, w_gate_up, w_down, top_k)        -> y [T, H]
    gemm_moe_workspace_bytes(T, E, top_k, H, I)
"""
import ctypes

import torch

from ._lib import MoeArgs, lib
from .mx4 import FORMATS, MX4, _call, _check_stream, _given, _keep, _new, _workspace

MAX_TOKENS, MAX_EXPERTS, MAX_TOP_K = 64, 512, 16


def _c_layer(args, workspace, nbytes, stream):
    # the stream comes before the workspace
    return lib.gemm_moe(args, stream, workspace, nbytes)


def gemm_moe_workspace_bytes(T, E, top_k, H, I):
    """Bytes of workspace gemm_moe needs for these sizes."""
    return int(lib.gemm_moe_workspace_bytes(T, E, top_k, H, I))


def _weights(w, name):
    """(pointer, expert stride, row stride, scales pointer and strides)."""
    if isinstance(w, MX4):
        data, ldd, scales, lds = w._rows()
        per_d, per_s = w._stack_strides()
        return data, per_d, ldd, scales, per_s, lds
    if w.stride(2) != 1 and w.shape[2] > 1:
        raise ValueError(f"{name} must have unit stride along its last axis")
    return w.data_ptr(), w.stride(0), w.stride(1), 0, 0, 0


def gemm_moe(x, logits, w_gate_up, w_down, top_k, renormalize=True, out=None, workspace=None, stream=None):
    """y [T, H] = sum over each token's top_k experts e of p_e w_down[e] (silu(g) * u),
    with (g, u) the two halves of w_gate_up[e] x.

    x [T, H] float16 or bfloat16 (T at most 64: for more tokens sort the rows
    by expert and use gemm_grouped), logits [T, E] float32 or 16-bit, w_gate_up
    [E, 2I, H] (gate rows first) and w_down [E, H, I], both of x's dtype or
    both MX4.  All with unit stride along the last axis.

    The top_k largest logits choose (equal ones: the lower index; -inf: never;
    E at most 512, top_k at most 16).  p is the softmax of the chosen logits, or
    with renormalize=False that of all.  A token of -inf logits alone, such as
    a padded row of a batch, gets zeros.

    Sums are fp32, and silu(g) * u keeps 16 significant bits at any magnitude.

    workspace: gemm_moe_workspace_bytes(T, E, top_k, H, I) bytes, 256-byte
    aligned, not shared with a call that may overlap; allocated here when not
    given."""
    quantised = isinstance(w_gate_up, MX4)
    if quantised != isinstance(w_down, MX4):
        raise TypeError("w_gate_up and w_down must both be MX4 or both tensors")
    if x.ndim != 2 or logits.ndim != 2 or w_gate_up.ndim != 3 or w_down.ndim != 3:
        raise ValueError("expected x [T, H], logits [T, E], w_gate_up [E, 2I, H], w_down [E, H, I]")
    if x.dtype not in (torch.float16, torch.bfloat16) or logits.dtype not in FORMATS:
        raise TypeError("x must be float16 or bfloat16, logits float32, float16 or bfloat16")
    if not quantised and (w_gate_up.dtype != x.dtype or w_down.dtype != x.dtype):
        raise TypeError("16-bit weights must have x's dtype")
    if not x.is_cuda or len({x.device, logits.device, w_gate_up.device, w_down.device}) != 1:
        raise ValueError("inputs must share one GPU device")
    if stream is not None:
        _check_stream(stream, x.device)
    T, H = x.shape
    E, H2, I = w_down.shape
    if logits.shape != (T, E) or w_gate_up.shape != (E, 2 * I, H) or H2 != H or min(T, H, E, I) <= 0:
        raise ValueError("incompatible or empty shape")
    if T > MAX_TOKENS or E > MAX_EXPERTS or not 1 <= top_k <= min(E, MAX_TOP_K):
        raise ValueError(f"at most {MAX_TOKENS} tokens and {MAX_EXPERTS} experts, top_k in 1 .. "
                         f"min(E, {MAX_TOP_K})")
    if (x.stride(1) != 1 and H > 1) or (logits.stride(1) != 1 and E > 1):
        raise ValueError("x and logits must have unit stride along the last axis")
    if out is None:
        out = _new((T, H), x.dtype, x.device, stream)
    elif out.dtype != x.dtype or out.device != x.device or out.shape != (T, H) or \
            (out.stride(1) != 1 and H > 1) or (out.stride(0) < H and T > 1):
        raise ValueError("out must be a row-major [T, H] tensor of x's dtype on its device")
    p1, e1, n1, s1, se1, sn1 = _weights(w_gate_up, "w_gate_up")
    p2, e2, n2, s2, se2, sn2 = _weights(w_down, "w_down")
    args = MoeArgs(x.data_ptr(), x.stride(0), logits.data_ptr(), logits.stride(0), p1, e1, n1, s1, se1, sn1,
                   p2, e2, n2, s2, se2, sn2, out.data_ptr(), out.stride(0) if T > 1 else H, T, E, H, I, top_k,
                   FORMATS[x.dtype], FORMATS[logits.dtype], int(quantised), int(bool(renormalize)))
    if workspace is None:
        workspace = _workspace(lib.gemm_moe_workspace_bytes(T, E, top_k, H, I), x.device, stream)
    _call(x.device, stream, _c_layer, ctypes.byref(args), *_given(workspace, x.device))
    if stream is not None:
        _keep(stream, x, logits, w_gate_up, w_down, out, workspace)
    return out
