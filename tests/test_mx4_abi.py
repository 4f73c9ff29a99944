"""The MX4 entry points on the CPU: the header declares what the binding
lists, and every argument outside the contract is refused before any device
is touched."""
import os
import re
import subprocess

import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
from dense_tiled_gemm_fp16_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PX, PD, PS, PB, PT, PC = (0x7F0000000000 + (i << 36) for i in range(6))   # never dereferenced


def declared(header):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\**\s+\**(gemm_\w+)\s*\(", text, re.M)))


def test_header_declares_the_binding_list():
    assert declared("gemm_mx4.h") == sorted(_lib.EXPORTS_MX4)
    out = subprocess.run(["nm", "-D", "--defined-only", g.LIB_PATH], capture_output=True, text=True,
                         check=True).stdout
    exported = set(re.findall(r"\sT\s(\w+)$", out, re.M))
    assert set(_lib.EXPORTS_MX4) <= exported


def quantize(X=PX, fmt=0, sg=1, sr=70, sk=1, G=1, R=4, K=70, data=PD, scales=PS):
    return g.lib.gemm_mx4_quantize(X, fmt, sg, sr, sk, G, R, K, data, scales, None)


@pytest.mark.parametrize("kw,code", [
    (dict(X=0), -1), (dict(data=0), -1), (dict(scales=0), -1),
    (dict(G=0), -2), (dict(R=0), -2), (dict(K=0), -2), (dict(K=-1), -2), (dict(K=2 ** 40), -2),
    (dict(sr=2 ** 62), -2), (dict(G=2, sg=2 ** 62), -2), (dict(G=2 ** 40, R=2 ** 40), -2),
    (dict(fmt=3), -7), (dict(fmt=-1), -7),
    (dict(sr=0), -3), (dict(sk=0), -3), (dict(sg=-1), -3),
    (dict(data=PX + 64), -5), (dict(scales=PX + 64), -5), (dict(scales=PD + 16), -5),
    (dict(data=PD + 8), -9),
])
def test_quantize_refusals(kw, code):
    assert quantize(**kw) == code


def dequantize(data=PD, ldd=48, scales=PS, lds=3, R=4, K=70, Y=PX, fmt=1, ldy=70):
    return g.lib.gemm_mx4_dequantize(data, ldd, scales, lds, R, K, Y, fmt, ldy, None)


@pytest.mark.parametrize("kw,code", [
    (dict(data=0), -1), (dict(scales=0), -1), (dict(Y=0), -1), (dict(R=0), -2), (dict(K=0), -2),
    (dict(fmt=5), -7), (dict(ldy=69), -4), (dict(ldd=32), -3), (dict(lds=2), -3), (dict(ldd=0), -3),
    (dict(ldd=2 ** 62), -2), (dict(ldy=2 ** 61), -2), (dict(ldd=56), -9), (dict(data=PD + 4), -9),
    (dict(Y=PD), -5), (dict(Y=PS - 8), -5),
])
def test_dequantize_refusals(kw, code):
    assert dequantize(**kw) == code


def product(A=PX, lda=48, SA=PT, ldsa=3, B=PB, ldb=48, SB=PS, ldsb=3, C=PC, fmt=0, ldc=9, M=5, N=9, K=70,
            ws=0, nws=0):
    return g.lib.gemm_mx4(A, lda, SA, ldsa, B, ldb, SB, ldsb, C, fmt, ldc, M, N, K, None, ws, nws)


@pytest.mark.parametrize("kw,code", [
    (dict(A=0), -1), (dict(SA=0), -1), (dict(B=0), -1), (dict(SB=0), -1), (dict(C=0), -1),
    (dict(M=0), -2), (dict(N=0), -2), (dict(K=0), -2), (dict(fmt=2), -7), (dict(ldc=8), -4),
    (dict(ldb=2 ** 27), -9), (dict(ldsa=2 ** 27), -9), (dict(M=65, lda=2 ** 27), -9),
    (dict(lda=32), -3), (dict(ldsb=2), -3), (dict(lda=50), -9), (dict(B=PB + 1), -9),
    (dict(C=PX), -5), (dict(C=PT), -5), (dict(C=PB + 16), -5), (dict(C=PS), -5), (dict(ldc=2 ** 62), -2),
    (dict(M=65535 * 64 + 1), -2), (dict(N=2 ** 27 + 1, ldc=2 ** 27 + 1), -2),
])
def test_product_refusals(kw, code):
    assert product(**kw) == code


def product16(A=PX, fmt=0, lda=70, B=PB, ldb=48, SB=PS, ldsb=3, C=PC, ldc=9, M=5, N=9, K=70):
    return g.lib.gemm_mx4_a16(A, fmt, lda, B, ldb, SB, ldsb, C, ldc, M, N, K, None)


@pytest.mark.parametrize("kw,code", [
    (dict(A=0), -1), (dict(B=0), -1), (dict(SB=0), -1), (dict(C=0), -1), (dict(M=0), -2), (dict(N=-1), -2),
    (dict(K=0), -2), (dict(fmt=2), -7), (dict(lda=0), -3), (dict(ldc=8), -4), (dict(ldb=32), -3),
    (dict(lda=2 ** 26), -9), (dict(ldsb=2 ** 27), -9),
    (dict(B=PB + 8), -9), (dict(C=PX + 2), -5), (dict(C=PS), -5), (dict(lda=2 ** 62), -2),
    (dict(M=65535 * 32 + 1), -2), (dict(N=2 ** 27 + 1, ldc=2 ** 27 + 1), -2),
])
def test_product16_refusals(kw, code):
    assert product16(**kw) == code


def test_python_refusals():
    x = torch.zeros(4, 70, dtype=torch.float16)
    with pytest.raises(ValueError):
        g.quantize_mx4(x)                       # not on a GPU
    with pytest.raises(TypeError):
        g.quantize_mx4(x.to(torch.int32))
    data, scales = torch.zeros(4, 48, dtype=torch.uint8), torch.zeros(4, 3, dtype=torch.uint8)
    q = g.MX4(data, scales, 70)
    assert q.shape == (4, 70) and q[1:3].shape == (2, 70)
    for bad in ((data, scales, 97), (data[:, :32], scales, 70), (data, scales[:3], 70),
                (data.t(), scales.t(), 70), (data, scales, 0)):
        with pytest.raises(ValueError):
            g.MX4(*bad)
    with pytest.raises(TypeError):
        g.MX4(data.to(torch.int8), scales, 70)
    with pytest.raises(ValueError):
        g.dequantize_mx4(q)
    with pytest.raises(TypeError):
        g.dequantize_mx4(q, torch.int32)
    with pytest.raises(ValueError):
        g.gemm_mx4(x, q)
    with pytest.raises(ValueError):
        g.gemm_mx4(x, x)
