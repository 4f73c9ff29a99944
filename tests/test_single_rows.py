"""Outputs of a single row: the stride of an axis of one is free, so a column
turned round is one."""
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def column(n, dtype):
    """[1, n] with strides (1, 1), inside a buffer whose ends stay 3."""
    buf = torch.full((n + 8, 1), 3.0, dtype=dtype, device=DEV)
    return buf, buf[4:n + 4].t()


def check(buf, out, want):
    n = out.shape[1]
    assert torch.equal(out, want) and (buf[:4] == 3).all() and (buf[n + 4:] == 3).all()


@pytest.mark.parametrize("K", [1, 40, 300])
def test_dequantize(K):
    q = g.quantize_mx4(torch.randn(1, K, device=DEV))
    for dtype in (torch.float16, torch.float32):
        buf, out = column(K, dtype)
        say(f"single row dequantize {K}")
        check(buf, g.dequantize_mx4(q, dtype, out=out), g.dequantize_mx4(q, dtype))
        stack = g.MX4(q.data.expand(2, 1, -1), q.scales.expand(2, 1, -1), K)
        both = torch.empty(2, K + 3, dtype=dtype, device=DEV)[:, :K].as_strided((2, 1, K), (K, 1, 1))
        assert both.is_contiguous()
        assert torch.equal(g.dequantize_mx4(stack, dtype, out=both)[1], g.dequantize_mx4(q, dtype))


@pytest.mark.parametrize("N", [1, 33, 300])
def test_products(N):
    x = torch.randn(1, 64, device=DEV, dtype=torch.bfloat16)
    w = g.quantize_mx4(torch.randn(N, 64, device=DEV))
    say(f"single row products {N}")
    for a in (x, g.quantize_mx4(x)):
        buf, out = column(N, torch.bfloat16)
        check(buf, g.gemm_mx4(a, w, out=out, dtype=torch.bfloat16), g.gemm_mx4(a, w, dtype=torch.bfloat16))


def test_experts():
    x, logits = torch.randn(1, 96, device=DEV).half(), torch.randn(1, 4, device=DEV)
    up, down = torch.randn(4, 64, 96, device=DEV).half() * 0.1, torch.randn(4, 96, 32, device=DEV).half() * 0.1
    buf, out = column(96, torch.float16)
    say("single row experts")
    check(buf, g.gemm_moe(x, logits, up, down, 2, out=out), g.gemm_moe(x, logits, up, down, 2))
