"""Matrix results in accumulation registers of the library as built are read
late enough: the scan of test_isa_hazards, which follows results in v[..],
with results in a[..] followed too and matrix instructions that take a result
as a factor counted as readers.  Only kernels of which some result was
followed count as scanned."""
import os
import re
import shutil

import pytest

from test_isa_hazards import LIB, LLVM, code_objects, parse

READERS = ("v_", "global_", "ds_", "buffer_", "flat_", "scratch_")


def registers(operand):
    """(file, index) of every register that an operand names."""
    m = re.match(r"^-?\|?([va])(\d+)\|?$", operand)
    if m:
        return {(m[1], int(m[2]))}
    m = re.match(r"^([va])\[(\d+):(\d+)\]$", operand)
    return {(m[1], i) for i in range(int(m[2]), int(m[3]) + 1)} if m else set()


def early_reads(code):
    """(matrix instructions followed, early readers)."""
    base = code[0][2]
    at = {c[2] - base: i for i, c in enumerate(code)}
    followed, bad = 0, []
    for i, (op, args, _, _) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        result = registers(args[0])
        followed += bool(result)
        need = (8 if "32x32" in op else 4) + 4
        todo, seen = [(i + 1, 0, frozenset(result))], set()
        while todo:
            j, waited, live = todo.pop()
            while j < len(code) and waited < need and live and (j, waited, live) not in seen:
                seen.add((j, waited, live))
                o, a, _, target = code[j]
                reads = a[1:3] if o.startswith("v_mfma") else a if o.startswith(READERS) else []
                if any(registers(x) & live for x in reads):
                    bad.append(f"{op} {args[0]} .. {waited} states .. {o} {', '.join(a)}")
                    break
                if o.startswith("v_mfma"):
                    live = live - registers(a[0])
                waited += int(a[0]) + 1 if o == "s_nop" else 1
                if o == "s_branch" or o.startswith("s_cbranch"):
                    if target is not None and int(target, 16) in at:
                        todo.append((at[int(target, 16)], waited, live))
                    if o == "s_branch":
                        break
                if o == "s_endpgm":
                    break
                j += 1
    return followed, bad


def planted(result, reader, between="s_cbranch_vccnz 1 // 000000000008: 0 <k+0x10>"):
    (_, code), = parse("\n".join([
        "0000000000000000 <k>:", f"\tv_mfma_f32_16x16x32_f16 {result}, v[4:7], v[8:11], {result} // 000000000000: 0",
        f"\t{between}", "\ts_nop 15 // 00000000000C: 0", f"\t{reader} // 000000000010: 0",
        "\ts_endpgm // 000000000014: 0"]))
    return early_reads(code)


@pytest.mark.parametrize("result,reader", [
    ("a[0:3]", "v_accvgpr_read_b32 v12, a2"), ("a[0:3]", "global_store_dwordx4 v[20:21], a[0:3], off"),
    ("v[0:3]", "v_mov_b64_e32 v[12:13], v[2:3]"), ("a[0:3]", "v_accvgpr_write_b32 a1, v9"),
    ("v[0:3]", "v_mfma_f32_16x16x32_f16 v[16:19], v[0:3], v[8:11], 0"),
    ("a[0:3]", "v_mfma_f32_16x16x32_f16 a[16:19], v[8:11], a[0:3], a[16:19]")])
def test_scan_finds_planted_early_reads(result, reader):
    followed, bad = planted(result, reader)
    assert followed >= 1 and len(bad) == 1
    # on every path behind the wait states; the same numbers in the other file
    assert planted(result, reader, "s_nop 0 // 000000000008: 0")[1] == []
    other = {"a": "v", "v": "a"}[result[0]] + result[1:]
    assert planted(other, reader)[1] == []
    # a sum that goes on in the same registers is no early read
    assert planted(result, f"v_mfma_f32_16x16x32_f16 {result}, v[4:7], v[8:11], {result}")[1] == []


def test_matrix_results_in_either_file_are_read_late_enough():
    if not os.path.exists(LIB):
        pytest.fail("libgemmf16.so is not built")
    if not (shutil.which("objcopy") and os.path.exists(os.path.join(LLVM, "llvm-objdump"))):
        pytest.skip("objcopy / ROCm llvm tools not available")
    kernels, bad = 0, {}
    for text in code_objects(LIB):
        for name, code in parse(text):
            matrix = sum(c[0].startswith("v_mfma") for c in code)
            followed, found = early_reads(code)
            assert followed == matrix, f"{name}: {matrix - followed} results not followed"
            kernels += followed > 0
            if found:
                bad[name] = found[:3]
    assert kernels > 300, kernels
    assert not bad, bad
