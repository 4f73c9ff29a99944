"""The codes and scales that the norm makes of its result y are those that
quantisation makes of y in float32: where y is exact, bit for bit."""
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
from f8_ref import E4M3, E5M2, f64, quotients, round8
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.mark.parametrize("R,K", [(5, 100), (300, 128), (3, 515), (40, 1024), (7, 7168), (2, 16384), (2, 16392), (2, 40001)])
@pytest.mark.parametrize("dtype,wt,res,f8", [(BF16, F32, True, E4M3), (F16, F16, False, E4M3), (BF16, BF16, False, E5M2),
                                             (F16, F32, True, E5M2)])
def test_codes_are_those_of_the_quantiser(R, K, dtype, wt, res, f8):
    """Rows of 1 and -1 without eps: their mean square is 1 exactly, so y is the
    weight with its row's signs.  The weight's values have 8 bits, which leaves many
    quotients midway between two 8-bit ones."""
    say(f"norm codes {R}x{K} {dtype} {wt} {res} {f8}")
    gen = torch.Generator(device="cpu")
    gen.manual_seed(R + K)
    sign = (torch.randint(0, 2, (R, K), generator=gen) * 2 - 1).float()
    w = (torch.randn(K, generator=gen) * 2).to(BF16).to(wt)
    y = sign * w.float()
    x = (sign / 2 if res else sign).to(dtype).to(DEV)
    data, scales, h = g.rms_norm_f8(x, w.to(DEV), 0.0, residual=x.clone() if res else None, dtype=f8)
    assert torch.equal(h.float().cpu(), sign)
    want, ws = g.quantize_f8(y.to(DEV), dtype=f8)
    assert torch.equal(scales, ws)
    assert torch.equal(data.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))
    q, _ = quotients(f64(y), 1, f8)
    assert (f64(data) == round8(q, f8)).all()
