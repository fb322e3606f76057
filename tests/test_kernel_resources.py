"""Registers spilled by the matrix-core kernels, as the compiler recorded them
in the built library's code objects.

A spill inside a K loop costs a round trip to memory at every stage, so one in a
product that has none is an error here (the first form of the MXFP4 Linears
spilled 4055 registers and took five times as long). The weight gradients of
long experts keep 16 spilled registers (output row numbers, not accumulators)."""
import os
import re
import shutil
import struct
import subprocess

import pytest

import expert_grouped_gemm_amd as moe

READELF = next((p for p in (os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin", "llvm-readelf"),
                            shutil.which("llvm-readelf")) if p and os.path.exists(p)), None)
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _code_objects(path):
    """The gfx950 code objects of a library: a bundle is the magic, a count and, per entry, its offset (from the
    magic), its size and its target's name."""
    data = open(path, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        (count,), pos = struct.unpack_from("<Q", data, at + len(MAGIC)), at + len(MAGIC) + 8
        for _ in range(count):
            off, size, n = struct.unpack_from("<QQQ", data, pos)
            target = data[pos + 24:pos + 24 + n]
            pos += 24 + n
            if target.endswith(b"gfx950"):
                yield data[at + off:at + off + size]
        at = data.find(MAGIC, at + len(MAGIC))


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    if READELF is None:
        pytest.skip("llvm-readelf not found")
    if not os.path.exists(moe.LIB_PATH):
        from expert_grouped_gemm_amd import build
        build.build()
    out, tmp = {}, tmp_path_factory.mktemp("co")
    for i, obj in enumerate(_code_objects(moe.LIB_PATH)):
        f = tmp / f"{i}.elf"
        f.write_bytes(obj)
        notes = subprocess.run([READELF, "--notes", str(f)], capture_output=True, text=True, check=True).stdout
        for k in notes.split("- .agpr_count:")[1:]:
            get = lambda field: re.search(rf"\.{field}:\s+(\S+)", k).group(1)  # noqa: E731
            out[get("name")] = {f: int(get(f)) for f in ("vgpr_spill_count", "private_segment_fixed_size")}
    return out


def _one(kernels, pattern):
    found = [v for n, v in kernels.items() if re.search(pattern, n)]
    assert len(found) == 1, (pattern, sorted(kernels))
    return found[0]


@pytest.mark.parametrize("kernel", [r"15moe_gemm_kernelILi3E", r"22expert_backward_kernelILi0E",
                                    r"22expert_backward_kernelILi1E", r"22expert_backward_kernelILi2E",
                                    r"28weight_backward_short_kernelILi3E", r"28weight_backward_short_kernelILi4E"])
def test_products_spill_nothing(kernels, kernel):
    assert _one(kernels, kernel) == dict(vgpr_spill_count=0, private_segment_fixed_size=0)


@pytest.mark.parametrize("kernel", [r"22expert_backward_kernelILi3E", r"22expert_backward_kernelILi4E"])
def test_weight_gradients_of_long_experts_spill_no_more_than_known(kernels, kernel):
    assert _one(kernels, kernel)["vgpr_spill_count"] <= 16
