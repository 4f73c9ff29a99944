"""The entry points of the 8-bit products scaled by blocks, of the norm and of
the rows sorted by expert on the CPU: the headers declare what the binding
lists, and every argument outside the contract is refused before any device is
touched."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
from dense_tiled_gemm_fp16_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = [0x7F0000000000 + (i << 36) for i in range(10)]      # never dereferenced


def declared(header):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(gemm_\w+)\s*\(", text, re.M)))


@pytest.mark.parametrize("header,names", [("gemm_f8_scaled.h", _lib.EXPORTS_F8S), ("rms_norm_f8.h", _lib.EXPORTS_NORM),
                                          ("gemm_moe_rows.h", _lib.EXPORTS_MOE_ROWS)])
def test_header_declares_the_binding_list(header, names):
    assert declared(header) == sorted(names)
    out = subprocess.run(["nm", "-D", "--defined-only", g.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    assert set(names) <= set(re.findall(r"\sT\s(\w+)$", out, re.M))


def test_headers_compile_as_c(tmp_path):
    src = tmp_path / "all.c"
    src.write_text('#include "rms_norm_f8.h"\n#include "gemm_moe_rows.h"\nint main(void) { return 0; }\n')
    subprocess.run(["gcc", "-Wall", "-Werror", "-std=c99", "-fsyntax-only", "-I", os.path.join(ROOT, "include"),
                    str(src)], check=True)


def quantize(X=P[0], fmt=1, sr=300, sk=1, R=4, K=300, rows=1, data=P[1], fmt8=0, ldd=304, scales=P[2], ss_r=3, ss_k=1):
    return g.lib.gemm_f8s_quantize(ctypes.byref(_lib.F8sQuantizeArgs(X, sr, sk, R, K, data, ldd, scales, ss_r, ss_k, fmt,
                                                                    fmt8, rows)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=0), -1), (dict(data=0), -1), (dict(scales=0), -1),
    (dict(R=0), -2), (dict(K=0), -2), (dict(K=2 ** 40, ldd=2 ** 40), -2), (dict(sr=2 ** 62), -2),
    (dict(ldd=2 ** 62), -2), (dict(ss_r=2 ** 61), -2),
    (dict(fmt=3), -7), (dict(fmt=-1), -7), (dict(fmt8=2), -7), (dict(fmt8=-1), -7), (dict(rows=64), -7),
    (dict(sr=0), -3), (dict(sk=0), -3), (dict(ss_r=0), -3), (dict(ss_k=-1), -3), (dict(ldd=299), -4),
    (dict(ss_r=1), -4), (dict(ss_r=2, ss_k=1), -4), (dict(ss_r=1, ss_k=3), -4),
    (dict(scales=P[2] + 2), -9), (dict(data=P[0] + 64), -5), (dict(scales=P[0] + 64), -5), (dict(scales=P[1] + 16), -5),
])
def test_quantize_refusals(kw, code):
    assert quantize(**kw) == code


def product(**kw):
    d = dict(A=P[0], lda=304, SA=P[1], lsa_m=3, lsa_k=1, B=P[2], ldb=304, SB=P[3], lsb_n=3, lsb_k=1, C=P[4], ldc=200,
             M=100, N=200, K=300, fmt_a=0, fmt_b=1, b_block_rows=128, fmt_c=1, variant=0)
    d.update(kw)
    return g.lib.gemm_f8s(ctypes.byref(_lib.F8sArgs(**d)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(A=0), -1), (dict(SA=0), -1), (dict(B=0), -1), (dict(SB=0), -1), (dict(C=0), -1),
    (dict(M=0), -2), (dict(N=-1), -2), (dict(K=0), -2), (dict(K=2 ** 40, lda=2 ** 40, ldb=2 ** 40), -2),
    (dict(lda=2 ** 62), -2), (dict(ldc=2 ** 62), -2), (dict(lsa_m=2 ** 61), -2), (dict(lsb_k=2 ** 62), -2),
    (dict(fmt_a=2), -7), (dict(fmt_b=-1), -7), (dict(b_block_rows=2), -7), (dict(fmt_c=3), -7),
    (dict(variant=-1), -7), (dict(variant=10), -7), (dict(variant=9, b_block_rows=1, lsb_n=3), -7),
    (dict(variant=9, fmt_c=2, ldc=200), -7),
    (dict(lda=0), -3), (dict(lda=288), -3), (dict(ldb=288), -3), (dict(lsa_m=0), -3), (dict(lsa_k=0), -3),
    (dict(lsb_n=-3), -3), (dict(lsb_k=0), -3), (dict(ldc=199), -4),
    (dict(lda=300), -9), (dict(lda=2 ** 23 + 16), -9), (dict(ldb=2 ** 24), -9), (dict(lsa_m=2 ** 22), -9),
    (dict(lsb_n=2 ** 22), -9), (dict(ldb=312), -9), (dict(A=P[0] + 8), -9), (dict(B=P[2] + 4), -9), (dict(SA=P[1] + 2), -9),
    (dict(C=P[4] + 1), -9), (dict(C=P[0]), -5), (dict(C=P[1]), -5), (dict(C=P[2]), -5), (dict(C=P[3]), -5),
])
def test_product_refusals(kw, code):
    assert product(**kw) == code


@pytest.mark.parametrize("name", ["gemm_f8s", "gemm_f8s_quantize", "gemm_rms_norm_f8", "gemm_moe_gather",
                                  "gemm_moe_combine", "gemm_moe_combine_backward"])
def test_no_arguments_at_all(name):
    assert getattr(g.lib, name)(None, None) == -1


@pytest.mark.parametrize("name", ["gemm_rms_norm_backward", "gemm_moe_sort"])
def test_no_arguments_at_all_with_workspace(name):
    assert getattr(g.lib, name)(None, None, 0, 0) == -1


@pytest.mark.parametrize("cls", [_lib.F8sArgs, _lib.F8sQuantizeArgs, _lib.NormArgs, _lib.NormBackwardArgs, _lib.SortArgs,
                                 _lib.GatherArgs, _lib.CombineArgs, _lib.CombineBackwardArgs])
def test_packed_arguments_are_the_structure(cls):
    values = [float(i) if t is ctypes.c_float else i + 1 for i, (_, t) in enumerate(cls._fields_)]
    packed = _lib.packer(cls)(*values)
    assert packed == bytes(cls(*values))


def test_structures_have_the_headers_sizes(tmp_path):
    names = {"gemm_f8s_args": _lib.F8sArgs, "gemm_f8s_quantize_args": _lib.F8sQuantizeArgs,
             "gemm_rms_norm_f8_args": _lib.NormArgs, "gemm_rms_norm_backward_args": _lib.NormBackwardArgs,
             "gemm_moe_sort_args": _lib.SortArgs, "gemm_moe_gather_args": _lib.GatherArgs,
             "gemm_moe_combine_args": _lib.CombineArgs, "gemm_moe_combine_backward_args": _lib.CombineBackwardArgs}
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "rms_norm_f8.h"', '#include "gemm_moe_rows.h"',
             "int main(void) {"]
    for name, cls in names.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "sizes.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "sizes")], check=True)
    out = subprocess.run([str(tmp_path / "sizes")], capture_output=True, text=True, check=True).stdout.split()
    want = []
    for cls in names.values():
        want += [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]
    assert [int(v) for v in out] == want


def norm(X=P[0], ldx=300, res=P[1], ldr=300, fmt=1, W=P[2], fmt_w=2, eps=1e-6, H=P[3], ldh=300, data=P[4], fmt8=0,
         ldd=304, scales=P[5], ss_r=3, ss_k=1, R=4, K=300):
    return g.lib.gemm_rms_norm_f8(ctypes.byref(_lib.NormArgs(X, ldx, res, ldr, W, H, ldh, data, ldd, scales, ss_r, ss_k,
                                                             R, K, eps, fmt, fmt_w, fmt8)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=0), -1), (dict(W=0), -1), (dict(data=0), -1), (dict(scales=0), -1), (dict(H=0), -1),
    (dict(R=0), -2), (dict(K=0), -2), (dict(K=65537, ldd=70000, ldh=70000), -2), (dict(ldx=2 ** 62), -2),
    (dict(fmt=2), -7), (dict(fmt=-1), -7), (dict(fmt_w=0), -7), (dict(fmt8=2), -7), (dict(eps=-1.0), -7),
    (dict(eps=float("nan")), -7), (dict(ldx=0), -3), (dict(ldr=0), -3), (dict(ss_r=0), -3), (dict(ss_k=0), -3),
    (dict(ldd=299), -4), (dict(ldh=299), -4), (dict(ss_r=2), -4), (dict(ss_r=1, ss_k=3), -4), (dict(scales=P[5] + 1), -9),
    (dict(data=P[0]), -5), (dict(data=P[1]), -5), (dict(data=P[2]), -5), (dict(data=P[3]), -5), (dict(scales=P[0]), -5),
    (dict(scales=P[4]), -5), (dict(H=P[0] + 2), -5), (dict(H=P[0], ldh=302), -5), (dict(H=P[1] + 600), -5),
    (dict(H=P[2]), -5),
])
def test_norm_refusals(kw, code):
    assert norm(**kw) == code


def norm_back(DY=P[0], ldy=300, H=P[1], ldh=300, fmt=1, W=P[2], fmt_w=1, eps=1e-6, DH=P[3], lddh=300, DX=P[4], lddx=300,
              DW=P[5], R=4, K=300, ws=0, nws=0):
    return g.lib.gemm_rms_norm_backward(ctypes.byref(_lib.NormBackwardArgs(DY, ldy, H, ldh, W, DH, lddh, DX, lddx, DW, R,
                                                                           K, eps, fmt, fmt_w)), None, ws, nws)


@pytest.mark.parametrize("kw,code", [
    (dict(DY=0), -1), (dict(H=0), -1), (dict(W=0), -1), (dict(DX=0), -1), (dict(DW=0), -1),
    (dict(R=0), -2), (dict(K=0), -2), (dict(K=70000, lddx=70000), -2), (dict(ldy=2 ** 62), -2),
    (dict(fmt=2), -7), (dict(fmt_w=0), -7), (dict(eps=-1.0), -7),
    (dict(ldy=0), -3), (dict(ldh=0), -3), (dict(lddh=-1), -3), (dict(lddx=299), -4),
    (dict(DX=P[0] + 4), -5), (dict(DX=P[0], lddx=304), -5), (dict(DX=P[1]), -5), (dict(DX=P[2]), -5), (dict(DX=P[5]), -5),
    (dict(DW=P[0]), -5), (dict(DW=P[1]), -5), (dict(DW=P[2]), -5), (dict(DW=P[3]), -5),
    (dict(ws=P[6], nws=100), -6), (dict(ws=P[6] + 4, nws=1 << 20), -6), (dict(ws=P[0], nws=1 << 20), -5),
    (dict(ws=P[4], nws=1 << 20), -5),
])
def test_norm_backward_refusals(kw, code):
    assert norm_back(**kw) == code


def sort(ids=P[0], size=8, ld=2, T=4, k=2, E=4, off=P[1], rows=P[2], slots=P[3], ws=0, nws=0):
    return g.lib.gemm_moe_sort(ctypes.byref(_lib.SortArgs(ids, ld, T, off, rows, slots, size, k, E)), None, ws, nws)


@pytest.mark.parametrize("kw,code", [
    (dict(ids=0), -1), (dict(off=0), -1), (dict(rows=0), -1), (dict(slots=0), -1),
    (dict(T=0), -2), (dict(k=0), -2), (dict(E=0), -2), (dict(E=1025), -2), (dict(T=2 ** 23), -2),
    (dict(T=2 ** 22, k=512), -2), (dict(size=2), -7), (dict(ld=0), -3), (dict(ld=2 ** 60), -2),
    (dict(ids=P[0] + 4), -9), (dict(off=P[1] + 4), -9), (dict(rows=P[2] + 4), -9), (dict(slots=P[3] + 1), -9),
    (dict(off=P[0]), -5), (dict(rows=P[0]), -5), (dict(slots=P[2] + 8), -5), (dict(rows=P[1] + 8), -5),
    (dict(T=100000, ws=P[4], nws=64), -6), (dict(T=100000, ws=P[4] + 8, nws=1 << 24), -6),
    (dict(T=100000, ws=P[2], nws=1 << 24), -5),
])
def test_sort_refusals(kw, code):
    assert sort(**kw) == code


def gather(X=P[0], ldx=8, size=2, off=P[1], slots=P[2], E=4, Y=P[3], ldy=8, T=4, k=2, H=8):
    return g.lib.gemm_moe_gather(ctypes.byref(_lib.GatherArgs(X, ldx, off, slots, Y, ldy, T, H, size, E, k)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=0), -1), (dict(off=0), -1), (dict(slots=0), -1), (dict(Y=0), -1), (dict(T=0), -2), (dict(k=0), -2),
    (dict(E=0), -2), (dict(H=0), -2), (dict(H=2 ** 25, ldy=2 ** 25), -2), (dict(size=8), -7), (dict(ldx=0), -3),
    (dict(ldy=7), -4), (dict(Y=P[0]), -5), (dict(Y=P[1]), -5), (dict(Y=P[2]), -5),
])
def test_gather_refusals(kw, code):
    assert gather(**kw) == code


def combine(X=P[0], ldx=8, fmt=1, slots=P[1], w=P[2], fmt_w=2, ldw=2, Y=P[3], ldy=8, T=4, k=2, H=8):
    return g.lib.gemm_moe_combine(ctypes.byref(_lib.CombineArgs(X, ldx, slots, w, ldw, Y, ldy, T, H, fmt, fmt_w, k)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=0), -1), (dict(slots=0), -1), (dict(Y=0), -1), (dict(T=0), -2), (dict(k=-1), -2), (dict(H=0), -2),
    (dict(fmt=3), -7), (dict(fmt_w=0), -7), (dict(ldx=0), -3), (dict(ldw=0), -3), (dict(ldy=7), -4),
    (dict(Y=P[0]), -5), (dict(Y=P[1]), -5), (dict(Y=P[2]), -5),
])
def test_combine_refusals(kw, code):
    assert combine(**kw) == code


def combine_back(DY=P[0], lddy=8, X=P[1], ldx=8, fmt=1, off=P[2], slots=P[3], E=4, w=P[4], fmt_w=2, ldw=2, DX=P[5],
                 lddx=8, DW=P[6], lddw=2, T=4, k=2, H=8):
    return g.lib.gemm_moe_combine_backward(ctypes.byref(_lib.CombineBackwardArgs(
        DY, lddy, X, ldx, off, slots, w, ldw, DX, lddx, DW, lddw, T, H, fmt, fmt_w, E, k)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(DY=0), -1), (dict(X=0), -1), (dict(off=0), -1), (dict(slots=0), -1), (dict(w=0), -1), (dict(DX=0), -1),
    (dict(DW=0), -1), (dict(T=0), -2), (dict(E=0), -2), (dict(H=0), -2), (dict(fmt=4), -7), (dict(fmt_w=0), -7),
    (dict(lddy=0), -3), (dict(ldx=0), -3), (dict(ldw=0), -3), (dict(lddx=7), -4), (dict(lddw=1), -4),
    (dict(DX=P[0]), -5), (dict(DX=P[1]), -5), (dict(DX=P[3]), -5), (dict(DW=P[4]), -5), (dict(DW=P[5]), -5),
])
def test_combine_backward_refusals(kw, code):
    assert combine_back(**kw) == code


def test_python_refusals_need_no_gpu():
    x = torch.zeros(4, 300, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 304, dtype=torch.float8_e4m3fn)[:, :300], torch.zeros(4, 3)
    for bad in (lambda: g.quantize_f8(x), lambda: g.gemm_f8_scaled(q, s, q, s), lambda: g.rms_norm_f8(x, x[0]),
                lambda: g.rms_norm_backward(x, x, x[0]), lambda: g.moe_sort(torch.zeros(4, 2, dtype=torch.int64), 4)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: g.quantize_f8(x.double()), lambda: g.quantize_f8(x, dtype=torch.float16),
                lambda: g.gemm_f8_scaled(x, s, q, s), lambda: g.gemm_f8_scaled(q, s.double(), q, s),
                lambda: g.rms_norm_f8(x.float(), x[0]), lambda: g.moe_sort(torch.zeros(4, 2), 4)):
        with pytest.raises(TypeError):
            bad()


def test_workspaces_of_empty_shapes():
    assert g.rms_norm_backward_workspace_bytes(0, 4) == 0 == g.rms_norm_backward_workspace_bytes(4, 70000)
    assert g.moe_sort_workspace_bytes(0, 2, 4) == 0 == g.moe_sort_workspace_bytes(64, 2, 4)
    assert g.moe_sort_workspace_bytes(100000, 2, 4) > 0
