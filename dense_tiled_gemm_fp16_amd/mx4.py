"""Microscaled 4-bit floating point (OCP MX FP4): quantisation and products
with 4-bit weights.  Argument marshalling for include/gemm_mx4.h; the
computation runs in the HIP library.

    MX4(data, scales, K)          -> a matrix (or a stack of them) in 4 bits
    quantize_mx4(x)               -> MX4 of x [R, K] or [G, R, K], along the last axis
    dequantize_mx4(q, dtype)      -> its values
    gemm_mx4(a, b)                -> C [M, N] = a . b^T, b MX4 [N, K], a MX4 [M, K]
                                     or float16 / bfloat16 [M, K]
    gemm_mx4_workspace_bytes(M, N, K)

A stream by argument: as the package says.
"""
import torch

from ._lib import lib

# Element formats of the C calls (enum gemm_mx4_format).
FORMATS = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
BLOCK = 32

# Looked up once: a decode call's time is the host's.
_c_quantize, _c_dequantize = lib.gemm_mx4_quantize, lib.gemm_mx4_dequantize
_c_workspace, _c_product16 = lib.gemm_mx4_workspace_bytes, lib.gemm_mx4_a16


def _c_product(*args):
    # the stream comes before the workspace
    return lib.gemm_mx4(*args[:-3], args[-1], args[-3], args[-2])


def _error(rc):
    from . import GemmError
    return GemmError(rc)


# The current stream as an integer, and the current device, without the checks
# and objects of torch.cuda around them: a small call is bound by its Python.
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _check_stream(stream, device):
    if stream.device != device:
        raise ValueError("stream must be one of the inputs' device")


def _call(device, stream, fn, *args):
    """fn(*args, stream) with `device` current."""
    index = device.index
    s = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == _current_device():
        rc = fn(*args, s)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, s)
    if rc:
        raise _error(rc)


def _new(shape, dtype, device, stream):
    """A result on the current stream, written on `stream`: allocated in the
    latter's order, kept until both are done with it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


_empty = torch.empty


def _new2(rows, cols, dtype, device, stream):
    """_new of a matrix (its sizes by position: 0.4 us less than as a tuple)."""
    if stream is None:
        return _empty(rows, cols, dtype=dtype, device=device)
    return _new((rows, cols), dtype, device, stream)


def _workspace(nbytes, device, stream):
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _keep(stream, *used):
    """Tensors and MX4s that a call on a stream by argument uses: the caller may
    drop them right after the call, and then their memory is not handed out
    again before the stream is done with them."""
    for u in used:
        for t in u._tensors() if isinstance(u, MX4) else (u,):
            if t is not None:
                t.record_stream(stream)


def _given(workspace, device):
    """(pointer, bytes) of a caller's workspace."""
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


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

    __slots__ = ("_data", "_scales", "_buffer", "_ldd", "_lds", "K", "shape", "device")

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
        self._data, self._scales, self._buffer = data, scales, None
        self._ldd, self._lds = data.stride(-2), scales.stride(-2)
        self.K, self.shape, self.device = K, (*data.shape[:-1], K), data.device

    @classmethod
    def _empty(cls, shape, device, stream):
        """Contiguous and uninitialised, data and scales in one allocation
        (the tensors are made when they are asked for)."""
        q = cls.__new__(cls)
        rows = 1
        for n in shape[:-1]:
            rows *= n
        K = shape[-1]
        q._data = q._scales = None
        q._buffer = _new((17 * rows * -(-K // BLOCK),), torch.uint8, device, stream)
        q.K, q.shape, q.device = K, tuple(shape), device
        q._lds = -(-K // BLOCK)
        q._ldd = 16 * q._lds
        return q

    def _split(self):
        blocks = -(-self.K // BLOCK)
        n = self._buffer.numel() // 17 * 16
        self._data = self._buffer[:n].view(*self.shape[:-1], 16 * blocks)
        self._scales = self._buffer[n:].view(*self.shape[:-1], blocks)

    @property
    def data(self):
        if self._data is None:
            self._split()
        return self._data

    @property
    def scales(self):
        if self._scales is None:
            self._split()
        return self._scales

    @property
    def ndim(self):
        return len(self.shape)

    @property
    def is_cuda(self):
        return self.device.type == "cuda"

    def is_contiguous(self):
        return self._buffer is not None or (self._data.is_contiguous() and self._scales.is_contiguous())

    def _rows(self):
        """(data pointer, row stride, scales pointer, row stride)."""
        if self._buffer is not None:
            p = self._buffer.data_ptr()
            return p, self._ldd, p + self._buffer.numel() // 17 * 16, self._lds
        return self._data.data_ptr(), self._ldd, self._scales.data_ptr(), self._lds

    def _tensors(self):
        return (self._buffer,) if self._buffer is not None else (self._data, self._scales)

    def _stack_strides(self):
        """Strides from matrix to matrix of a stack's data and scales."""
        if self._buffer is not None:
            rows, blocks = self.shape[-2], -(-self.K // BLOCK)
            return 16 * rows * blocks, rows * blocks
        return self._data.stride(0), self._scales.stride(0)

    def __getitem__(self, rows):
        return MX4(self.data[rows], self.scales[rows], self.K)

    def __repr__(self):
        return f"MX4(shape={self.shape}, device={self.device})"


def quantize_mx4(x, out=None, stream=None):
    """x [R, K] or [G, R, K] (float16, bfloat16 or float32, any positive
    strides) in MX4, quantised along K.

    A block's scale is 2^(floor(log2 m) - 2), m its largest magnitude (at least
    2^-127); elements round to nearest, ties to the even code, and saturate at
    6 scales.  A block with an infinity or a NaN becomes NaN.  The elements
    past K of the last block are zero.  out: an MX4 of x's shape with
    contiguous data and scales."""
    fmt, shape, strides, device = FORMATS.get(x.dtype), x.shape, x.stride(), x.device
    if fmt is None:
        raise TypeError("expected float16, bfloat16 or float32")
    if len(shape) not in (2, 3) or not x.is_cuda:
        raise ValueError("expected an [R, K] matrix or a [G, R, K] stack on a GPU")
    if min(shape) <= 0:
        raise ValueError("empty shape")
    if min(strides) <= 0:
        raise ValueError("strides must be positive")
    if stream is not None:
        _check_stream(stream, device)
    if out is None:
        out = MX4._empty(shape, device, stream)
    elif out.shape != tuple(shape) or out.device != device or not out.is_contiguous():
        raise ValueError("out must be an MX4 of x's shape on its device, contiguous")
    G, sg = (shape[0], strides[0]) if len(shape) == 3 else (1, 1)
    data, _, scales, _ = out._rows()
    _call(device, stream, _c_quantize, x.data_ptr(), fmt, sg, strides[-2], strides[-1], G, shape[-2], shape[-1],
          data, scales)
    if stream is not None:
        _keep(stream, x, out)
    return out


def dequantize_mx4(q, dtype=torch.bfloat16, out=None, stream=None):
    """The values of an MX4 matrix or stack, each rounded once to dtype
    (float16, bfloat16 or float32).  out: of q's shape, contiguous, or for a
    matrix row-major with any row stride."""
    fmt, shape, device = FORMATS.get(dtype), q.shape, q.device
    if fmt is None:
        raise TypeError("dtype must be float16, bfloat16 or float32")
    if not q.is_cuda or min(shape) <= 0:
        raise ValueError("expected a non-empty MX4 on a GPU")
    if stream is not None:
        _check_stream(stream, device)
    if out is None:
        out = _new(shape, dtype, device, stream)
    elif out.dtype != dtype or out.device != device or out.shape != shape or \
            (out.stride(-1) != 1 and shape[-1] > 1) or (len(shape) == 3 and not out.is_contiguous()):
        raise ValueError("out must be of q's shape, of dtype, on its device, with unit column stride "
                         "(a stack contiguous)")
    R, K = shape[0], shape[-1]
    data, ldd, scales, lds = q._rows()
    ldy = out.stride(-2) if R > 1 else K      # a single row has no next one
    if len(shape) == 3:
        if not q.is_contiguous():
            for i in range(R):
                dequantize_mx4(q[i], dtype, out[i], stream)
            return out
        # one matrix of all rows (a stack of single rows may have any row stride)
        R, lds, ldy = R * shape[1], -(-K // BLOCK), K
        ldd = 16 * lds
    _call(device, stream, _c_dequantize, data, ldd, scales, lds, R, K, out.data_ptr(), fmt, ldy)
    if stream is not None:
        _keep(stream, q, out)
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
    weights exact (below 2^128, as all of a quantised tensor are); made for few
    rows (beyond some 64, quantise a first).

    workspace: gemm_mx4_workspace_bytes(M, N, K) bytes, 256-byte aligned, not
    shared with a call that may overlap; allocated here when not given."""
    if type(b) is not MX4 or len(b.shape) != 2 or len(a.shape) != 2:
        raise ValueError("expected a matrix a and an MX4 matrix b [N, K]")
    device = b.device
    if device.type != "cuda" or a.device != device:
        raise ValueError("inputs must share one GPU device")
    if stream is not None:
        _check_stream(stream, device)
    (M, K), (N, Kb) = a.shape, b.shape
    if K != Kb or M <= 0 or N <= 0 or K <= 0:
        raise ValueError("incompatible or empty shape")
    quantised = type(a) is MX4
    if quantised:
        dtype = dtype or torch.float16
        if dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("dtype must be float16 or bfloat16")
    else:
        given, dtype = dtype, a.dtype
        if FORMATS.get(dtype, 2) == 2:
            raise TypeError("a must be an MX4, float16 or bfloat16 matrix")
        if given is not None and given != dtype:
            raise TypeError("the output of a 16-bit a has its dtype")
        lda, one = a.stride()
        if (one != 1 and K > 1) or lda <= 0:
            raise ValueError("a must have unit stride along K and a positive row stride")
    ldc = N
    if out is None:
        out = _new((M, N), dtype, device, stream)
    elif out.dtype != dtype or out.device != device or out.shape != (M, N) or \
            (out.stride(1) != 1 and N > 1) or (out.stride(0) < N and M > 1):
        raise ValueError("out must be a row-major [M, N] tensor of the output dtype on the inputs' device")
    elif M > 1:
        ldc = out.stride(0)
    fmt = FORMATS[dtype]
    bp, ldb, sp, lds = b._rows()
    if quantised:
        if workspace is None:
            need = _c_workspace(M, N, K)
            if need:
                workspace = _workspace(need, device, stream)
        ws, nws = _given(workspace, device) if workspace is not None else (0, 0)
        ap, lda, asp, ldas = a._rows()
        _call(device, stream, _c_product, ap, lda, asp, ldas, bp, ldb, sp, lds, out.data_ptr(), fmt, ldc, M, N, K,
              ws, nws)
    else:
        _call(device, stream, _c_product16, a.data_ptr(), fmt, lda, bp, ldb, sp, lds, out.data_ptr(), ldc, M, N, K)
    if stream is not None:
        _keep(stream, a, b, out, workspace)
    return out
