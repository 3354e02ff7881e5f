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
        # (the largest dw tile never runs on split sums)
        assert "GroupWeightsILi4E" not in name or "3CfgILi4ELi2ELi2ELi4E" not in name, name
        if "GroupRowsILb1E" not in name:
            continue
        loads = re.findall(r"buffer_load_dword\w* v\d+, (s\[\d+:\d+\]), (\w+) offen(?: offset:\d+)? lds", body)
        moved = {r for r, more in loads if more != "0"}
        first = loads[0][0]  # (a stage's loads begin with A's)
        assert moved <= {first} and {r for r, _ in loads} > {first}, name
        checked += bool(moved)
    assert checked == 2  # fp16 and bf16 of the tile that moves A's stage to the scalar offset


def test_kernels_of_few_rows(tmp_path):
    """Every compiled kernel is one that a call reaches (packed operands are whole pieces, K is their padded one),
    none spills, none has packed fp32 arithmetic."""
    asm = _assembly("mxfp4_few.hip", tmp_path)
    names = [name for name, _ in _bodies(asm)]
    packed = [n for n in names if "few_rows_kernelIh" in n]
    assert len(packed) == 3 * 2 * 3  # output types, grouped or not, tiles
    assert len(names) - len(packed) == 2 * 2 * 3 * 2  # and whole rows or not
    for d in re.findall(r"^\s*\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", asm, re.M | re.S):
        value = lambda key: int(re.search(r"\.amdhsa_" + key + r"\s+(\d+)", d[1]).group(1))
        assert value("private_segment_fixed_size") == 0 and value("group_segment_fixed_size") <= 160 * 1024, d[0]
    assert not re.search(r"^\s*v_pk_(fma|mul|add)_f32", asm, re.M)
