"""The C entry points without a workspace: the library allocates one in the
stream's order, so calls may follow each other without a wait."""
import ctypes

import numpy as np
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
import mx4_ref as ref
from dense_tiled_gemm_fp16_amd import _lib
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def test_mx4_tile():
    M, N, K = 1700, 1800, 200
    rng = np.random.default_rng(1)
    a, b = (g.MX4(torch.from_numpy(d).to(DEV), torch.from_numpy(s).to(DEV), K)
            for d, s in (ref.random_codes(rng, M, K), ref.random_codes(rng, N, K)))
    want = g.gemm_mx4(a, b, dtype=torch.bfloat16)
    outs = [torch.zeros_like(want) for _ in range(3)]
    say("mx4 without a workspace")
    stream = torch.cuda.current_stream().cuda_stream
    for out in outs:
        assert g.lib.gemm_mx4(a.data.data_ptr(), a.data.stride(0), a.scales.data_ptr(), a.scales.stride(0),
                              b.data.data_ptr(), b.data.stride(0), b.scales.data_ptr(), b.scales.stride(0),
                              out.data_ptr(), 1, N, M, N, K, stream, None, 0) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)


@pytest.mark.parametrize("T,E,k,H,I", [(3, 6, 2, 200, 64), (48, 64, 8, 2000, 300)])
def test_experts(T, E, k, H, I):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)

    def rand(*shape):
        return (torch.randn(*shape, generator=gen, device=DEV) * shape[-1] ** -0.5).to(torch.bfloat16)

    x, logits, up, down = rand(T, H), rand(T, E), rand(E, 2 * I, H), rand(E, H, I)
    want = g.gemm_moe(x, logits, up, down, k)
    outs = [torch.zeros_like(want) for _ in range(3)]
    say(f"experts without a workspace {T} {E}")
    stream = torch.cuda.current_stream().cuda_stream
    for out in outs:
        args = _lib.MoeArgs(X=x.data_ptr(), ldx=H, logits=logits.data_ptr(), ldl=E, W1=up.data_ptr(), w1_e=2 * I * H,
                            w1_n=H, W2=down.data_ptr(), w2_e=H * I, w2_n=I, Y=out.data_ptr(), ldy=H, T=T, E=E, H=H,
                            I=I, top_k=k, fmt=1, fmt_logits=1, mx4=0, renormalize=1)
        assert g.lib.gemm_moe(ctypes.byref(args), stream, None, 0) == 0
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for out in outs)
