"""No matrix instruction of the built library writes over part of its own
addend. D = A B + C takes D and C in the same registers or in disjoint ones; a D
that begins inside C overwrites elements of C before they are read.

The compiler does not see to that for the scaled instruction. The first form of
the MXFP4 Linears held two sets of accumulators, moved from one to the other by
products with D beside C, and 28 of these overlapped by 2 to 14 registers: those
elements of a row block lost products. The accumulators of the present kernels
stay where they are (D = C) or start from C = 0, and this reads the library's
own code for an instruction of which neither is true."""
import os
import re
import shutil
import subprocess

import pytest

import expert_grouped_gemm_amd as moe
from test_kernel_resources import _code_objects

OBJDUMP = next((p for p in (os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-objdump"),
                            shutil.which("llvm-objdump")) if p and os.path.exists(p)), None)
REGS = r"([va])\[(\d+):(\d+)\]"
MFMA = re.compile(rf"\bv_s?mfma\S*\s+{REGS},[^,]+,[^,]+,\s*(?:{REGS}|\S+)")


def _writes_over_its_addend(line):
    """Of one instruction's text: None if it is no matrix instruction, else whether D and C overlap in part."""
    m = MFMA.search(line)
    if m is None:
        return None
    file_d, d0, d1, file_c, c0, c1 = m.groups()
    if file_c is None or file_c != file_d or (d0, d1) == (c0, c1):
        return False
    return int(d0) <= int(c1) and int(c0) <= int(d1)


@pytest.mark.parametrize("line,bad", [
    ("v_mfma_scale_f32_32x32x64_f8f6f4 v[192:207], v[160:163], v[172:175], v[182:197], v180, v152 cbsz:4", True),
    ("v_mfma_f32_32x32x16_bf16 a[0:15], v[42:45], v[38:41], a[14:29]", True),
    ("v_mfma_f32_32x32x16_bf16 v[2:17], v[42:45], v[38:41], v[2:17]", False),
    ("v_mfma_f32_32x32x16_bf16 v[2:17], v[2:5], v[38:41], v[18:33]", False),
    ("v_mfma_f32_32x32x16_bf16 v[2:17], v[42:45], v[38:41], 0", False),
    ("v_mov_b32_e32 v2, v3", None),
])
def test_the_reading_of_an_instruction(line, bad):
    assert _writes_over_its_addend(line) is bad


def test_no_product_writes_over_its_addend(tmp_path):
    if OBJDUMP is None:
        pytest.skip("llvm-objdump not found")
    if not os.path.exists(moe.LIB_PATH):
        from expert_grouped_gemm_amd import build
        build.build()
    seen, bad = 0, []
    for i, obj in enumerate(_code_objects(moe.LIB_PATH)):
        f = tmp_path / f"{i}.elf"
        f.write_bytes(obj)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(f)], capture_output=True, text=True,
                              check=True).stdout
        for line in text.splitlines():
            if "mfma" in line:
                over = _writes_over_its_addend(line)
                seen += over is not None
                if over:
                    bad.append(line.split("//")[0].strip())
    assert seen > 1000        # the reading found the products
    assert not bad, bad[:5]
