"""Outputs that end inside a chunk of eight columns while the rows of C stay
16-byte aligned (N no multiple of 8, ldc one): every column up to N has to be
written, and none behind it.  The 256 x 256 tiles store C through LDS in such
chunks, whatever the operands' format."""
import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
import mx4_ref
import oracle
import synth
from gpu_util import DEV, ORACLE_THREADS, Out, assert_bits_equal, place, say, to_dev
from test_f8 import f8_rows, inputs, reference

pytestmark = pytest.mark.gpu

# (M, N, ldc): last columns 1, 2, 4, 7 and 3 of a chunk, in the tile's first and second half of a wave's
# columns, rows padded to 8 columns and further
EDGES = [(300, 257, 264), (257, 514, 520), (513, 300, 304), (300, 519, 520), (64, 387, 400), (260, 3, 8)]


def written(buf, out, ldc, N):
    """The result of an aligned, padded output; checks what lies behind N."""
    torch.cuda.synchronize()
    assert out.data_ptr() % 16 == 0 and ldc % 8 == 0 and N % 8 != 0
    assert (buf[:, N:] == 5.0).all(), "write behind the last column"
    return out


@pytest.mark.parametrize("M,N,ldc", EDGES)
@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("K", [64, 104])
def test_main_tile(M, N, ldc, fmt, K):
    A = synth.matrix(M, K, 9100 + M, 0, "int", fmt=fmt)
    B = synth.matrix(K, N, 9100 + N, 1, "int", fmt=fmt)
    ref = oracle.gemm(A, (K, 1), B, (N, 1), M, N, K, nthreads=ORACLE_THREADS, dtype=fmt)
    a, b, out = to_dev(A), place(B, "col"), Out(M, N, ldc=ldc)
    assert out.view.data_ptr() % 16 == 0
    if fmt == "bf16":
        a, b = a.view(torch.bfloat16), b.view(torch.bfloat16)
        out.view = out.view.view(torch.bfloat16)
    say(f"store edge {fmt} {M}x{N}x{K} ldc={ldc}")
    assert g.plan(a, b, out=out.view, variant="main", tile=14)["tile_id"] == 14
    g.gemm(a, b, out=out.view, variant="main", tile=14)
    torch.cuda.synchronize()
    assert_bits_equal(out.result(), ref, f"{fmt} {M}x{N}x{K} ldc={ldc}")


@pytest.mark.parametrize("M,N,ldc", EDGES)
def test_f8_tile(M, N, ldc):
    K = 192
    A, Bt = inputs(M, N, K, 9200 + M + N, "int", "e4m3", "e4m3")
    a, b, out = f8_rows(A, "e4m3"), f8_rows(Bt, "e4m3").t(), Out(M, N, ldc=ldc)
    say(f"store edge f8 {M}x{N}x{K} ldc={ldc}")
    assert g.plan(a, b, out=out.view, variant="main", tile=15)["tile_id"] == 15
    g.gemm(a, b, out=out.view, variant="main", tile=15)
    torch.cuda.synchronize()
    assert_bits_equal(out.result(), reference(A, Bt, "e4m3", "e4m3"), f"f8 {M}x{N}x{K} ldc={ldc}")


@pytest.mark.parametrize("M,N,ldc", EDGES)
def test_packed(M, N, ldc):
    K = 96
    A = synth.matrix(M, K, 9300 + M, 0, "int")
    B = synth.matrix(K, N, 9300 + N, 1, "int")
    ref = oracle.gemm(A, (K, 1), B, (N, 1), M, N, K, nthreads=ORACLE_THREADS)
    out = Out(M, N, ldc=ldc)
    say(f"store edge packed {M}x{N}x{K} ldc={ldc}")
    g.gemm_packed(to_dev(A), g.pack_b(to_dev(B)), out=out.view)
    torch.cuda.synchronize()
    assert_bits_equal(out.result(), ref, f"packed {M}x{N}x{K} ldc={ldc}")


@pytest.mark.parametrize("M,N,ldc,K", [(1801, 1543, 1544, 96), (1600, 1937, 1944, 200), (1801, 1540, 1544, 33),
                                       (12500, 130, 136, 96)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_mx4_tile(M, N, ldc, K, dtype):
    """Scales of 1: sums are exact, one rounding remains."""
    rng = np.random.default_rng(M + N)
    a, b = mx4_ref.random_codes(rng, M, K, 127, 127), mx4_ref.random_codes(rng, N, K, 127, 127)
    qa, qb = (g.MX4(torch.from_numpy(d).to(DEV), torch.from_numpy(s).to(DEV), K) for d, s in (a, b))
    assert g.gemm_mx4_workspace_bytes(M, N, K) > 0              # the tile path
    buf = torch.full((M, ldc), 5.0, dtype=dtype, device=DEV)
    out = buf[:, :N]
    out.fill_(float("nan"))
    say(f"store edge mx4 {M}x{N}x{K} ldc={ldc} {dtype}")
    g.gemm_mx4(qa, qb, out=out, dtype=dtype)
    want = torch.from_numpy(mx4_ref.values(*a, K) @ mx4_ref.values(*b, K).T).to(dtype)
    got = written(buf, out, ldc, N).cpu()
    assert torch.equal(got, want), f"{(~(got == want)).sum()} outputs differ"
    # C two bytes off a 16-byte boundary, the same sums
    off = torch.empty(M * ldc + 1, dtype=dtype, device=DEV)[1:].view(M, ldc)[:, :N]
    assert torch.equal(g.gemm_mx4(qa, qb, out=off, dtype=dtype).cpu(), want)
