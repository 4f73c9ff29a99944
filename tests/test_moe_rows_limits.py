"""Sizes that the row moves refuse before anything is enqueued (CPU)."""
import ctypes

import pytest

import dense_tiled_gemm_fp16_amd as g
from dense_tiled_gemm_fp16_amd import _lib

SHAPE = -2
AT = [1 << 46, 1 << 50, 1 << 54, 1 << 58, 1 << 59]      # far from each other, read by nothing


def gather(T, H, k, size=2):
    return g.lib.gemm_moe_gather(ctypes.byref(_lib.GatherArgs(AT[0], H, AT[1], AT[2], AT[3], H, T, H, size, 8, k)), None)


def combine(T, H, k, fmt=1):
    return g.lib.gemm_moe_combine(ctypes.byref(_lib.CombineArgs(AT[0], H, AT[1], AT[2], k, AT[3], H, T, H, fmt, 2, k)), None)


def backward(T, H, k, fmt=1):
    return g.lib.gemm_moe_combine_backward(ctypes.byref(_lib.CombineBackwardArgs(
        AT[0], H, AT[1], H, 1 << 40, 1 << 42, AT[2], k, AT[3], H, AT[4], k, T, H, fmt, 2, 8, k)), None)


@pytest.mark.parametrize("call", [gather, combine, backward])
@pytest.mark.parametrize("T,H,k", [(1 << 23, 1, 1), (1 << 22, 1, 512), (1, (1 << 24) + 1, 1), (0, 8, 1), (8, 0, 1), (8, 8, 0)])
def test_tokens_pairs_and_row_lengths(call, T, H, k):
    assert call(T, H, k) == SHAPE


def test_parts_of_rows():
    """2048 bytes of a row in gather, 1024 elements in combine: 2^25 of them are one
    too many."""
    assert gather(1 << 22, 8 * 1024, 1) == SHAPE and gather(1 << 22, 8 * 512, 1, 4) == SHAPE
    assert combine(1 << 22, 8 * 1024, 1) == SHAPE and combine(1 << 22, 7 * 1024 + 1, 1, 2) == SHAPE
