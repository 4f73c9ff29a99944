"""Matrix results in the library as built are read late enough.

On CDNA a matrix instruction's result registers need a number of wait states
before another vector instruction may read or overwrite them, and it is the
compiler that has to put them there.  hipcc 7.2 leaves them out where the
reader is the first instruction of another basic block (a register move behind
a conditional branch), and the move then copies stale sums, now and then.  So
the gfx950 code of this library is scanned: from every
matrix instruction along every path, no vector or memory instruction may touch
its result within the wait states that LLVM's own tables ask for (passes + 4,
with 8 passes for a 32 x 32 and 4 for a 16 x 16 instruction, the least any of
the formats used here takes)."""
import os
import re
import shutil
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "dense_tiled_gemm_fp16_amd", "libgemmf16.so")
LLVM = "/opt/rocm/llvm/bin"
TARGET = "hipv4-amdgcn-amd-amdhsa--gfx950"


def code_objects(lib):
    with tempfile.TemporaryDirectory() as tmp:
        fat = os.path.join(tmp, "fatbin")
        subprocess.run(["objcopy", "-O", "binary", "--only-section=.hip_fatbin", lib, fat], check=True,
                       capture_output=True)
        data = open(fat, "rb").read()
        starts = [m.start() for m in re.finditer(re.escape(b"__CLANG_OFFLOAD_BUNDLE__"), data)] + [len(data)]
        for n, (a, b) in enumerate(zip(starts, starts[1:])):
            part, co = os.path.join(tmp, f"b{n}"), os.path.join(tmp, f"co{n}")
            open(part, "wb").write(data[a:b])
            subprocess.run([os.path.join(LLVM, "clang-offload-bundler"), "--unbundle", "--type=o",
                            f"--input={part}", f"--targets={TARGET}", f"--output={co}"], check=True,
                           capture_output=True)
            yield subprocess.run([os.path.join(LLVM, "llvm-objdump"), "-d", co], check=True,
                                 capture_output=True, text=True).stdout


def registers(operand):
    m = re.match(r"^-?\|?v(\d+)\|?$", operand)
    if m:
        return {int(m[1])}
    m = re.match(r"^v\[(\d+):(\d+)\]$", operand)
    return set(range(int(m[1]), int(m[2]) + 1)) if m else set()


def parse(text):
    """(kernel, [(mnemonic, operands, address, branch offset)])."""
    name, code = None, []
    for line in text.splitlines():
        m = re.match(r"^[0-9a-f]+ <(.*)>:$", line)
        if m:
            if code:
                yield name, code
            name, code = m[1], []
            continue
        m = re.match(r"^\s+([a-z_][a-z0-9_]*)\s*(.*?)\s*// ([0-9A-F]+):.*?(?:<.*\+0x([0-9a-f]+)>)?$", line)
        if m and name:
            operands = [t.split()[0] for t in m[2].split(",") if t.split()]
            code.append((m[1], operands, int(m[3], 16), m[4]))
    if code:
        yield name, code


def early_reads(code):
    base = code[0][2]
    at = {c[2] - base: i for i, c in enumerate(code)}
    bad = []
    for i, (op, args, _, _) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        need = (8 if "32x32" in op else 4) + 4
        todo, seen = [(i + 1, 0, registers(args[0]))], set()
        while todo:
            j, waited, live = todo.pop()
            while j < len(code) and waited < need and live and (j, waited) not in seen:
                seen.add((j, waited))
                o, a, _, target = code[j]
                if o.startswith("v_mfma"):
                    live = live - registers(a[0])
                elif o.startswith(("v_", "global_", "ds_", "buffer_", "flat_", "scratch_")):
                    if any(registers(x) & live for x in a):
                        bad.append(f"{op} {args[0]} .. {waited} states .. {o} {', '.join(a)}")
                        break
                waited += int(a[0]) + 1 if o == "s_nop" else 1
                if o == "s_branch" or o.startswith("s_cbranch"):
                    if target is not None and int(target, 16) in at:
                        todo.append((at[int(target, 16)], waited, live))
                    if o == "s_branch":
                        break
                if o == "s_endpgm":
                    break
                j += 1
    return bad


def test_scan_finds_a_planted_early_read():
    text = "\n".join(["0000000000000000 <k>:", "\tv_mfma_f32_16x16x32_f16 v[0:3], v[4:7], v[8:11], v[0:3] // 000000000000: 0",
                      "\ts_cbranch_vccnz 1 // 000000000008: 0 <k+0x10>", "\ts_nop 15 // 00000000000C: 0",
                      "\tv_mov_b64_e32 v[12:13], v[2:3] // 000000000010: 0", "\ts_endpgm // 000000000014: 0"])
    (_, code), = parse(text)
    assert len(early_reads(code)) == 1
    (_, code), = parse(text.replace("s_cbranch_vccnz 1 // 000000000008: 0 <k+0x10>", "s_nop 0 // 000000000008: 0"))
    assert early_reads(code) == []


def test_matrix_results_are_read_late_enough():
    if not os.path.exists(LIB):
        pytest.fail("libgemmf16.so is not built")
    if not (shutil.which("objcopy") and os.path.exists(os.path.join(LLVM, "llvm-objdump"))):
        pytest.skip("objcopy / ROCm llvm tools not available")
    kernels, bad = 0, {}
    for text in code_objects(LIB):
        for name, code in parse(text):
            kernels += any(c[0].startswith("v_mfma") for c in code)
            found = early_reads(code)
            if found:
                bad[name] = found[:3]
    assert kernels > 100, kernels
    assert not bad, bad
