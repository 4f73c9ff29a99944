"""The built code of the quantiser, norm and row kernels, on the CPU: none keeps
registers in memory, the sort's kernels use no packed float32 arithmetic and no
atomics on floating-point values, and the kernels of the norm's gradients take no
more registers than the number of their workgroups counts on."""
import os
import re
import subprocess

import pytest

import dense_tiled_gemm_fp16_amd as g
from test_isa import LIB, LLVM, MAGIC, TARGET, _tools, kernels  # noqa: F401  (a fixture)

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


def test_registers_of_the_norms_gradients(tmp_path):
    """Four waves a SIMD (of 512 registers a lane) up to two octets a lane and in the
    wide kernel, two with four octets."""
    if not _tools() or not os.path.exists(os.path.join(LLVM, "llvm-readelf")):
        pytest.skip("objcopy / c++filt / ROCm llvm tools not available")
    fat = tmp_path / "fatbin"
    subprocess.run(["objcopy", "-O", "binary", "--only-section=.hip_fatbin", LIB, str(fat)], check=True, capture_output=True)
    data = fat.read_bytes()
    starts = [m.start() for m in re.finditer(re.escape(MAGIC), data)] + [len(data)]
    counts = {}
    for a, b in zip(starts, starts[1:]):
        if b"rms_norm_back" not in data[a:b]:
            continue
        part, co = tmp_path / "part", tmp_path / "co"
        part.write_bytes(data[a:b])
        subprocess.run([os.path.join(LLVM, "clang-offload-bundler"), "--unbundle", "--type=o", f"--input={part}",
                        f"--targets={TARGET}", f"--output={co}"], check=True, capture_output=True)
        notes = subprocess.run([os.path.join(LLVM, "llvm-readelf"), "--notes", str(co)], check=True, capture_output=True,
                               text=True).stdout
        for name, vgprs in re.findall(r"\.name: +(_Z\S+)(?:(?!\.name:).)*?\.vgpr_count: +(\d+)", notes, re.S):
            if "rms_norm_back" in name:
                counts[name] = int(vgprs)
    wide = {n: v for n, v in counts.items() if "rms_norm_back_wide_kernel" in n}
    rows = {n: v for n, v in counts.items() if "rms_norm_back_kernel" in n}
    assert len(wide) == 8 and len(rows) == 2 * 3 * 16
    assert max(wide.values()) <= 128
    for name, vgprs in rows.items():
        octets = int(re.search(r"rms_norm_back_kernelILi\dELi(\d)E", name).group(1))
        assert vgprs <= (128 if octets <= 2 else 256), (name, vgprs)


@pytest.mark.parametrize("K,workgroups", [(7168, 512), (8200, 256), (16384, 256), (16392, 256), (65536, 256)])
def test_workgroups_of_the_norms_gradients(K, workgroups):
    """A row of sums for each workgroup; of rows that fill a compute unit's registers,
    one workgroup a unit."""
    assert g.rms_norm_backward_workspace_bytes(100000, K) == workgroups * K * 4
