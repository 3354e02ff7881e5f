"""What the assembly of the expert layers' kernels shows about their loads (host-only check)."""

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KDIR = os.path.join(ROOT, "structured_sparse_gemm_w24_amd", "csrc", "kernels")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def _assembly(source, folder):
    if shutil.which(HIPCC) is None and not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    from structured_sparse_gemm_w24_amd.build import HIP_FLAGS
    flags = [f for f in HIP_FLAGS if f not in ("-fPIC", "-fvisibility=hidden")]
    out = os.path.join(folder, source + ".s")
    p = subprocess.run([HIPCC, *flags, "--cuda-device-only", "-S", os.path.join(KDIR, source), "-o", out],
                       capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    return open(out).read()


def _bodies(asm):
    """kernel name -> its instructions"""
    for name in re.findall(r"^\s*\.amdhsa_kernel (\S+)", asm, re.M):
        at = asm.index("\n" + name + ":")
        yield name, asm[at:asm.index(".Lfunc_end", at)]


def test_loads_that_may_pass_the_end_have_their_whole_offset_checked(tmp_path):
    """A buffer load's range check leaves its scalar offset out.  A weight read along its rows (the input
    gradient's second operand) is read past its last row's end where a tile is wider than the rows: those loads
    carry all of their offset in the vector register.  A's rows end inside the buffer, so its may do otherwise."""
    checked = 0
    for name, body in _bodies(_assembly("grouped.hip", tmp_path)):
        if "GroupRowsILb1E" not in name:
            continue
        loads = re.findall(r"buffer_load_dword\w* v\d+, (s\[\d+:\d+\]), (\w+) offen(?: offset:\d+)? lds", body)
        moved = {r for r, more in loads if more != "0"}
        first = loads[0][0]  # (a stage's loads begin with A's)
        assert moved <= {first} and {r for r, _ in loads} > {first}, name
        checked += bool(moved)
    assert checked == 2  # fp16 and bf16 of the tile that moves A's stage to the scalar offset
