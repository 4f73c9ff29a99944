"""The instructions of the block-scaled FP8, norm and row kernels as built, on
the CPU: products on the matrix core in the form their results need, no registers
spilled to memory in a product, no packed float32 arithmetic and no atomics on
floating-point values anywhere."""
import re

from test_isa import _of, _targs, kernels  # noqa: F401  (a fixture)

F8 = ("v_mfma_f32_16x16x128_f8f6f4", "v_mfma_scale_f32_16x16x128_f8f6f4")
F16 = "v_mfma_f32_16x16x32_f16"
NEW = ("f8s_tile_kernel", "f8s_strip_kernel", "f8s_big_kernel", "f8_rows_kernel", "f8_tiles_kernel", "rms_norm_f8_kernel",
       "rms_norm_back_kernel", "rms_norm_back_wide_kernel", "rms_norm_dw_kernel", "moe_gather_kernel", "moe_combine_kernel",
       "moe_combine_back_kernel")


def test_products_keep_their_mfma(kernels):  # noqa: F811
    for prefix, count in (("f8s_tile_kernel", 2 * 4 * 4), ("f8s_strip_kernel", 6 * 4 * 4)):
        found = _of(kernels, prefix)
        assert len(found) == count              # shapes x format pairs x (row blocks, float32 results)
        for name, ops in found.items():
            wide = _targs(name)[-1] == "true"
            f8 = sum(ops[op] for op in F8)
            assert (ops[F16] >= 8 and f8 == 0) if wide else (f8 >= 2 and ops[F16] == 0), (name, f8, ops[F16])
    found = _of(kernels, "f8s_big_kernel")
    assert len(found) == 8                      # format pairs x output formats
    for name, ops in found.items():
        assert sum(ops[op] for op in F8) >= 64, name


def test_products_do_not_spill(kernels):  # noqa: F811
    for prefix in ("f8s_tile_kernel", "f8s_strip_kernel", "f8s_big_kernel"):
        for name, ops in _of(kernels, prefix).items():
            assert not [op for op in ops if op.startswith("scratch_")], name


def test_no_packed_float32_and_no_float_atomics(kernels):  # noqa: F811
    for prefix in NEW:
        for name, ops in _of(kernels, prefix).items():
            bad = [op for op in ops if re.match(r"v_pk_(add|mul|fma)_f32", op) or re.search(r"atomic.*_(f32|f64|f16|bf16)", op)]
            assert not bad, (name, bad)
