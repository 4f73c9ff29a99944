"""The built code of the quantiser, norm and row kernels, on the CPU: none keeps
registers in memory, and the sort's kernels use no packed float32 arithmetic and
no atomics on floating-point values."""
import re

import pytest

from test_isa import kernels  # noqa: F401  (a fixture)

TEMPLATES = ("f8_rows_kernel", "f8_tiles_kernel", "rms_norm_f8_kernel", "rms_norm_back_kernel", "rms_norm_back_wide_kernel",
             "rms_norm_dw_kernel", "moe_gather_kernel", "moe_combine_kernel", "moe_combine_back_kernel")
SORT = ("moe_count_kernel", "moe_place_kernel")


def found(kernels, prefix):  # noqa: F811
    pattern = re.compile(r"^(void )?gemmf16::" + prefix + r"[<(]")
    out = {k: v for k, v in kernels.items() if pattern.match(k)}
    assert out, prefix
    return out


@pytest.mark.parametrize("prefix", TEMPLATES + SORT)
def test_no_registers_in_memory(kernels, prefix):  # noqa: F811
    for name, ops in found(kernels, prefix).items():
        assert not [op for op in ops if op.startswith("scratch_")], name


@pytest.mark.parametrize("prefix", SORT)
def test_sort_without_packed_float32_or_float_atomics(kernels, prefix):  # noqa: F811
    for name, ops in found(kernels, prefix).items():
        bad = [op for op in ops if re.match(r"v_pk_(add|mul|fma)_f32", op) or re.search(r"atomic.*_(f32|f64|f16|bf16)", op)]
        assert not bad, (name, bad)
