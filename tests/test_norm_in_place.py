"""Gradients of the norm in place where a row ends inside a lane's eight elements and
lies in several waves: the last lane loads elements of its neighbour's, of another
wave too, before any of them is overwritten."""
import pytest
import torch

import dense_tiled_gemm_fp16_amd as g
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def randn(*shape, dtype, seed):
    gen = torch.Generator(device="cpu")
    gen.manual_seed(seed)
    return torch.randn(*shape, generator=gen).to(dtype).to(DEV)


# Rows of one to eight waves, and K's end just behind a wave's (1025, 1537, 4097, 8193) or
# anywhere else; enough rows that workgroups take several.
@pytest.mark.parametrize("R,K", [(1300, 509), (2100, 1021), (2100, 1025), (2100, 1031), (1500, 1537), (1500, 2049), (1200, 2053),
                                 (1100, 3483), (1100, 4097), (1100, 4103), (1100, 7167), (600, 8191), (600, 8193), (600, 12289),
                                 (600, 16383)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_gradients_where_dy_or_dh_was(R, K, dtype):
    say(f"norm backward in place {R}x{K} {dtype}")
    dy, h, dh = (randn(R, K, dtype=dtype, seed=s) for s in (1, 2, 3))
    w = randn(K, dtype=F32, seed=4)
    for d in (dh, None):
        dx, dw = g.rms_norm_backward(dy, h, w, dh=d)
        for turn in range(3):
            for i in range(2 if d is not None else 1):
                a, b = dy.clone(), None if d is None else d.clone()
                into = (a, b)[i]
                gx, gw = g.rms_norm_backward(a, h, w, dh=b, out=into)
                assert gx is into and torch.equal(gx, dx) and torch.equal(gw, dw)
