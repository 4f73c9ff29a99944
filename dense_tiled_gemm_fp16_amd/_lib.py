"""ctypes view of libgemmf16.so (the C-ABI in include/gemm_f16.h and
the headers beside it).

Argument marshalling only: every step of the computation runs in the HIP
library.  There is no fallback: if the library cannot be loaded, importing
this module raises."""
import ctypes
import os
import struct

from . import build as _build

i32, i64, vp, sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
f32 = ctypes.c_float

GEMM_OK = 0
STATUS = {0: "GEMM_OK", -1: "GEMM_ERR_NULL", -2: "GEMM_ERR_SHAPE", -3: "GEMM_ERR_STRIDE",
          -4: "GEMM_ERR_LDC", -5: "GEMM_ERR_ALIAS", -6: "GEMM_ERR_WORKSPACE",
          -7: "GEMM_ERR_OPTS", -8: "GEMM_ERR_HIP", -9: "GEMM_ERR_LAYOUT", -10: "GEMM_ERR_SCRATCH"}
SCRATCH_BYTES = 32 << 20   # GEMM_F16_SCRATCH_BYTES
VARIANT_AUTO, VARIANT_MAIN, VARIANT_SKINNY, VARIANT_SPLITK, VARIANT_TILE64X32, VARIANT_STREAMK = \
    0, 1, 2, 3, 4, 5
VARIANTS = {"auto": 0, "main": 1, "skinny": 2, "splitk": 3, "tile64x32": 4, "streamk": 5}
PATHS = {0: "gather", 1: "kvec", 2: "rvec", 3: "packed"}

EXPORTS = ["gemm_f16", "gemm_f16_ex", "gemm_f16_plan", "gemm_f16_plan_cus", "gemm_f16_workspace_bytes",
           "gemm_bf16", "gemm_bf16_ex", "gemm_bf16_plan", "gemm_bf16_workspace_bytes",
           "gemm_f8", "gemm_f8_ex", "gemm_f8_plan", "gemm_f8_plan_cus", "gemm_f8_workspace_bytes",
           "gemm_f16_packed_b_bytes", "gemm_f16_pack_b", "gemm_f16_packed",
           "gemm_f16_grouped", "gemm_bf16_grouped", "gemm_f8_grouped", "gemm_f16_grouped_workspace_bytes",
           "gemm_f16_noalloc", "gemm_f16_status_string", "gemm_f16_version"]

# Entry points of include/gemm_mx4.h.
EXPORTS_MX4 = ["gemm_mx4_quantize", "gemm_mx4_dequantize", "gemm_mx4", "gemm_mx4_workspace_bytes",
               "gemm_mx4_a16"]
# Entry points of include/gemm_moe.h.
EXPORTS_MOE = ["gemm_moe", "gemm_moe_workspace_bytes"]
# Entry points of include/gemm_f8_scaled.h.
EXPORTS_F8S = ["gemm_f8s_quantize", "gemm_f8s"]
# Entry points of include/rms_norm_f8.h.
EXPORTS_NORM = ["gemm_rms_norm_f8", "gemm_rms_norm_backward", "gemm_rms_norm_backward_workspace_bytes"]
# Entry points of include/gemm_moe_rows.h.
EXPORTS_MOE_ROWS = ["gemm_moe_sort", "gemm_moe_sort_workspace_bytes", "gemm_moe_gather", "gemm_moe_combine",
                    "gemm_moe_combine_backward"]


class Opts(ctypes.Structure):
    _fields_ = [("variant", i32), ("split_k", i32), ("panel", i32), ("tile", i32)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("variant", i32), ("tile_m", i32), ("tile_n", i32), ("tile_k", i32),
                ("split_k", i32), ("panel", i32), ("a_path", i32), ("b_path", i32),
                ("tile_id", i32), ("grid", i64), ("grid2", i64),
                ("workspace_bytes", ctypes.c_uint64), ("sk_tiles", i64)]

    def as_dict(self):
        return {f: getattr(self, f) for f, _ in self._fields_}


class MoeArgs(ctypes.Structure):   # gemm_moe_args
    _fields_ = [("X", vp), ("ldx", i64), ("logits", vp), ("ldl", i64),
                ("W1", vp), ("w1_e", i64), ("w1_n", i64), ("S1", vp), ("s1_e", i64), ("s1_n", i64),
                ("W2", vp), ("w2_e", i64), ("w2_n", i64), ("S2", vp), ("s2_e", i64), ("s2_n", i64),
                ("Y", vp), ("ldy", i64), ("T", i64), ("E", i64), ("H", i64), ("I", i64), ("top_k", i32),
                ("fmt", i32), ("fmt_logits", i32), ("mx4", i32), ("renormalize", i32)]


class F8sArgs(ctypes.Structure):   # gemm_f8s_args
    _fields_ = [("A", vp), ("lda", i64), ("SA", vp), ("lsa_m", i64), ("lsa_k", i64),
                ("B", vp), ("ldb", i64), ("SB", vp), ("lsb_n", i64), ("lsb_k", i64),
                ("C", vp), ("ldc", i64), ("M", i64), ("N", i64), ("K", i64),
                ("fmt_a", i32), ("fmt_b", i32), ("b_block_rows", i32), ("fmt_c", i32), ("variant", i32)]


class F8sQuantizeArgs(ctypes.Structure):   # gemm_f8s_quantize_args
    _fields_ = [("X", vp), ("ldx_r", i64), ("ldx_k", i64), ("R", i64), ("K", i64), ("data", vp), ("ldd", i64),
                ("scales", vp), ("lds_r", i64), ("lds_k", i64), ("fmt", i32), ("fmt8", i32), ("block_rows", i32)]


class NormArgs(ctypes.Structure):   # gemm_rms_norm_f8_args
    _fields_ = [("X", vp), ("ldx", i64), ("residual", vp), ("ldr", i64), ("W", vp), ("H", vp), ("ldh", i64),
                ("data", vp), ("ldd", i64), ("scales", vp), ("lds_r", i64), ("lds_k", i64), ("R", i64), ("K", i64),
                ("eps", f32), ("fmt", i32), ("fmt_w", i32), ("fmt8", i32)]


class NormBackwardArgs(ctypes.Structure):   # gemm_rms_norm_backward_args
    _fields_ = [("DY", vp), ("ldy", i64), ("H", vp), ("ldh", i64), ("W", vp), ("DH", vp), ("lddh", i64), ("DX", vp),
                ("lddx", i64), ("DW", vp), ("R", i64), ("K", i64), ("eps", f32), ("fmt", i32), ("fmt_w", i32)]


class SortArgs(ctypes.Structure):   # gemm_moe_sort_args
    _fields_ = [("experts", vp), ("ld", i64), ("T", i64), ("offsets", vp), ("rows", vp), ("slots", vp),
                ("id_bytes", i32), ("top_k", i32), ("E", i32)]


class GatherArgs(ctypes.Structure):   # gemm_moe_gather_args
    _fields_ = [("X", vp), ("ldx", i64), ("offsets", vp), ("slots", vp), ("Y", vp), ("ldy", i64), ("T", i64),
                ("H", i64), ("elem_bytes", i32), ("E", i32), ("top_k", i32)]


class CombineArgs(ctypes.Structure):   # gemm_moe_combine_args
    _fields_ = [("X", vp), ("ldx", i64), ("slots", vp), ("weights", vp), ("ldw", i64), ("Y", vp), ("ldy", i64),
                ("T", i64), ("H", i64), ("fmt", i32), ("fmt_w", i32), ("top_k", i32)]


class CombineBackwardArgs(ctypes.Structure):   # gemm_moe_combine_backward_args
    _fields_ = [("DY", vp), ("lddy", i64), ("X", vp), ("ldx", i64), ("offsets", vp), ("slots", vp), ("weights", vp),
                ("ldw", i64), ("DX", vp), ("lddx", i64), ("DW", vp), ("lddw", i64), ("T", i64), ("H", i64),
                ("fmt", i32), ("fmt_w", i32), ("E", i32), ("top_k", i32)]


def packer(cls):
    """cls's fields in order -> its bytes, which a c_void_p argument takes: a third
    of the time of making the Structure (padded to its end)."""
    code = {vp: "q", i64: "q", i32: "i", f32: "f"}
    return struct.Struct("@" + "".join(code[t] for _, t in cls._fields_) + "0q").pack


def _load():
    if not os.path.exists(_build.LIB):
        _build.build()
    lib = ctypes.CDLL(_build.LIB)
    args12 = [vp, i64, i64, vp, i64, i64, vp, i64, i64, i64, i64, vp]
    lib.gemm_f16.argtypes = args12
    lib.gemm_f16.restype = ctypes.c_int
    lib.gemm_f16_noalloc.argtypes = args12
    lib.gemm_f16_noalloc.restype = ctypes.c_int
    lib.gemm_f16_ex.argtypes = args12 + [vp, sz, ctypes.POINTER(Opts)]
    lib.gemm_f16_ex.restype = ctypes.c_int
    lib.gemm_f16_plan.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, i64, i64, i64,
                                  ctypes.POINTER(Opts), ctypes.POINTER(PlanInfo)]
    lib.gemm_f16_plan.restype = ctypes.c_int
    lib.gemm_f16_plan_cus.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, i64, i64, i64, i32,
                                      ctypes.POINTER(Opts), ctypes.POINTER(PlanInfo)]
    lib.gemm_f16_plan_cus.restype = ctypes.c_int
    lib.gemm_f16_workspace_bytes.argtypes = [i64, i64, i64, ctypes.POINTER(Opts)]
    lib.gemm_f16_workspace_bytes.restype = sz
    for pre in ("gemm_bf16",):
        getattr(lib, pre).argtypes = args12
        getattr(lib, pre).restype = ctypes.c_int
        getattr(lib, pre + "_ex").argtypes = lib.gemm_f16_ex.argtypes
        getattr(lib, pre + "_ex").restype = ctypes.c_int
        getattr(lib, pre + "_plan").argtypes = lib.gemm_f16_plan.argtypes
        getattr(lib, pre + "_plan").restype = ctypes.c_int
        getattr(lib, pre + "_workspace_bytes").argtypes = lib.gemm_f16_workspace_bytes.argtypes
        getattr(lib, pre + "_workspace_bytes").restype = sz
    args14 = [vp, i64, i64, vp, i64, i64, vp, i64, i64, i64, i64, i32, i32, vp]
    lib.gemm_f8.argtypes = args14
    lib.gemm_f8.restype = ctypes.c_int
    lib.gemm_f8_ex.argtypes = args14 + [vp, sz, ctypes.POINTER(Opts)]
    lib.gemm_f8_ex.restype = ctypes.c_int
    lib.gemm_f8_plan.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, i64, i64, i64, i32, i32,
                                 ctypes.POINTER(Opts), ctypes.POINTER(PlanInfo)]
    lib.gemm_f8_plan.restype = ctypes.c_int
    lib.gemm_f8_plan_cus.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, i64, i64, i64, i32, i32, i32,
                                     ctypes.POINTER(Opts), ctypes.POINTER(PlanInfo)]
    lib.gemm_f8_plan_cus.restype = ctypes.c_int
    lib.gemm_f8_workspace_bytes.argtypes = [i64, i64, i64, ctypes.POINTER(Opts)]
    lib.gemm_f8_workspace_bytes.restype = sz
    lib.gemm_f16_packed_b_bytes.argtypes = [i64, i64]
    lib.gemm_f16_packed_b_bytes.restype = sz
    lib.gemm_f16_pack_b.argtypes = [vp, i64, i64, i64, i64, vp, vp]
    lib.gemm_f16_pack_b.restype = ctypes.c_int
    lib.gemm_f16_packed.argtypes = [vp, i64, i64, vp, vp, i64, i64, i64, i64, vp]
    lib.gemm_f16_packed.restype = ctypes.c_int
    lib.gemm_f16_grouped.argtypes = [vp, i64, i64, vp, i64, i64, i64, vp, i64, vp, i32,
                                     i64, i64, i64, vp, vp, sz]
    lib.gemm_f16_grouped.restype = ctypes.c_int
    lib.gemm_bf16_grouped.argtypes = lib.gemm_f16_grouped.argtypes
    lib.gemm_bf16_grouped.restype = ctypes.c_int
    lib.gemm_f8_grouped.argtypes = [vp, i64, i64, vp, i64, i64, i64, vp, i64, vp, i32, i64, i64, i64,
                                    i32, i32, vp, vp, sz]
    lib.gemm_f8_grouped.restype = ctypes.c_int
    lib.gemm_f16_grouped_workspace_bytes.argtypes = [i32]
    lib.gemm_f16_grouped_workspace_bytes.restype = sz
    lib.gemm_mx4_quantize.argtypes = [vp, i32, i64, i64, i64, i64, i64, i64, vp, vp, vp]
    lib.gemm_mx4_quantize.restype = ctypes.c_int
    lib.gemm_mx4_dequantize.argtypes = [vp, i64, vp, i64, i64, i64, vp, i32, i64, vp]
    lib.gemm_mx4_dequantize.restype = ctypes.c_int
    lib.gemm_mx4.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, vp, i32, i64, i64, i64, i64, vp, vp, sz]
    lib.gemm_mx4.restype = ctypes.c_int
    lib.gemm_mx4_workspace_bytes.argtypes = [i64, i64, i64]
    lib.gemm_mx4_workspace_bytes.restype = sz
    lib.gemm_mx4_a16.argtypes = [vp, i32, i64, vp, i64, vp, i64, vp, i64, i64, i64, i64, vp]
    lib.gemm_mx4_a16.restype = ctypes.c_int
    lib.gemm_moe.argtypes = [ctypes.POINTER(MoeArgs), vp, vp, sz]
    lib.gemm_moe.restype = ctypes.c_int
    lib.gemm_moe_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
    lib.gemm_moe_workspace_bytes.restype = sz
    for name in ("gemm_f8s_quantize", "gemm_f8s", "gemm_rms_norm_f8", "gemm_moe_gather", "gemm_moe_combine",
                 "gemm_moe_combine_backward"):
        getattr(lib, name).argtypes = [vp, vp]
        getattr(lib, name).restype = ctypes.c_int
    for name in ("gemm_rms_norm_backward", "gemm_moe_sort"):
        getattr(lib, name).argtypes = [vp, vp, vp, sz]
        getattr(lib, name).restype = ctypes.c_int
    lib.gemm_rms_norm_backward_workspace_bytes.argtypes = [i64, i64]
    lib.gemm_rms_norm_backward_workspace_bytes.restype = sz
    lib.gemm_moe_sort_workspace_bytes.argtypes = [i64, i32, i32]
    lib.gemm_moe_sort_workspace_bytes.restype = sz
    lib.gemm_f16_status_string.argtypes = [ctypes.c_int]
    lib.gemm_f16_status_string.restype = ctypes.c_char_p
    lib.gemm_f16_version.argtypes = []
    lib.gemm_f16_version.restype = ctypes.c_int
    return lib


lib = _load()
LIB_PATH = _build.LIB


def status_string(rc):
    return lib.gemm_f16_status_string(rc).decode()


def make_opts(variant=0, split_k=0, panel=0, tile=0):
    if isinstance(variant, str):
        variant = VARIANTS[variant]
    return Opts(variant, split_k, panel, tile)
