"""The loads from memory to LDS that product.h writes as inline assembly, of which
the compiler knows only what it is told (CPU: read from what is built here).

- m0, which holds the LDS address, is named as overwritten.
- A vector instruction's write of a scalar register needs five wait states before a
  load reads it, and the compiler counts none for inline assembly.
"""
import os
import re
import subprocess

import pytest

from test_kernel_metadata import LIB, LLVM, code_objects

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# three instructions that read LDS through m0 = 0, a load between each two
USES_M0 = """
#include "product.h"
using namespace hr;
__global__ void between(int *out, const char *from) {
    __shared__ int lds[256];
    HR_LDS int *p = (HR_LDS int *)lds;
    int n = __builtin_amdgcn_ds_append(p);
    dma16(buffer_of(from), threadIdx.x * 16, 64);
    n += __builtin_amdgcn_ds_append(p);
    dma4(buffer_of(from), threadIdx.x * 4, 64);
    n += __builtin_amdgcn_ds_append(p);
    landed<0>();
    out[threadIdx.x] = n;
}
"""


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="no hipcc")
def test_m0_is_written_again_behind_a_load(tmp_path):
    source = tmp_path / "m0.hip"
    source.write_text(USES_M0)
    text = subprocess.run([HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang",
                           "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-I",
                           os.path.join(ROOT, "message_fp16_all_amd", "csrc"), "--offload-device-only", "-S", str(source),
                           "-o", "-"], check=True, capture_output=True, text=True).stdout
    lines = [" ".join(m.group(0).split()) for m in re.finditer(r"s_mov_b32 m0, \S+|ds_append|buffer_load.* lds", text)]
    assert lines.count("ds_append") == 3 and sum("lds" in v for v in lines) == 2, lines
    for i, v in enumerate(lines):
        if v == "ds_append":
            assert lines[i - 1] == "s_mov_b32 m0, 0", lines


def registers(operand):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    return {int(m.group(1))} if m else set()


@pytest.mark.skipif(not os.path.exists(LIB) or not os.path.exists(f"{LLVM}/llvm-objdump"),
                    reason="libhr.so not built or ROCm LLVM tools missing")
def test_no_load_reads_a_scalar_register_just_written(tmp_path):
    loads = 0
    for co in code_objects(tmp_path):
        text = subprocess.run([f"{LLVM}/llvm-objdump", "-d", "--no-show-raw-insn", "--no-leading-addr", str(co)], check=True,
                              capture_output=True, text=True).stdout
        lines = [v.split("//")[0].strip() for v in text.splitlines()]
        for i, line in enumerate(lines):
            if not (line.startswith("buffer_load_dword") and line.endswith(" lds")):
                continue
            loads += 1
            wanted = set().union(*(registers(v) for v in re.findall(r"s\[\d+:\d+\]", line)))
            assert len(wanted) == 4, line
            waits, j = 0, i - 1
            while waits < 5 and j >= 0 and lines[j] and not lines[j].endswith(":"):
                op, _, operands = lines[j].partition(" ")
                if op.startswith("v_"):
                    assert not registers(operands.split(",")[0].strip()) & wanted, lines[j:i + 1]
                waits += int(operands) + 1 if op == "s_nop" else 1
                j -= 1
    assert loads > 1000
