"""Registers and spills of the 4-bit cache's kernels, checked at compile time on
the CPU (see tests/test_kernel_resources.py).

attn4_tc_kernel divides its registers between its warps with setmaxnreg: two
warpgroups of 176, one of 32 and two of 48 make 5 x 96, so a build that gave it
fewer than 96 at launch would wait for registers that never come.  Its spills are
of the roles with few registers, outside their inner loops.  attn4_rows_kernel
runs three warps to a scheduler (168 registers a thread) or two (255); its few
spilled words were measured against fewer warps (times beside the code).
"""
import os
import re
import shutil
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_kernel_resources import ENTRY, REGS, SPILL, _report

UNITS = ["attn4_tc.cu", "attn4_rows.cu", "kv4_rows.cu"]
SPILLS = {"attn4_tc_kernel": 700, "attn4_rows_kernelILi8E": 320, "attn4_rows_kernel": 128,
          "rope_append_kv4_kernel": 32}  # bytes of spill loads that a kernel may have


def _limit(name):
    m = re.search(r"attn4_rows_kernelILi(\d)ELi(\d)ELb([01])E", name)
    if m:
        nc, cpg, f32 = map(int, m.groups())
        return 168 if nc <= 4 and not (f32 and nc == 4 and cpg == 1) else 255
    if "rope_append_kv4_kernel" in name:
        return 64 if re.search(r"ILi[1-4]E", name) else 128
    return 64 if "kv4_read_kernel" in name else 96


def test_kv4_kernels_fit_their_register_budget(tmp_path):
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not found")
    with ThreadPoolExecutor(len(UNITS)) as ex:
        reports = list(ex.map(lambda u: _report(u, str(tmp_path)), UNITS))
    seen, problems = 0, []
    for text in reports:
        name = None
        for line in text.splitlines():
            m = ENTRY.search(line)
            if m:
                name = m.group(1)
            if name is None:
                continue
            m = SPILL.search(line)
            if m and int(m.group(2)) > next((v for k, v in SPILLS.items() if k in name), 0):
                problems.append(f"{name} spills ({line.strip()})")
            m = REGS.search(line)
            if m:
                seen += 1
                used = int(m.group(1))
                if used > _limit(name):
                    problems.append(f"{name} uses {used} registers, budget {_limit(name)}")
                if "attn4_tc_kernel" in name and used != 96:
                    problems.append(f"{name} is launched with {used} registers, its split needs 96")
                name = None
    assert seen >= 40, f"only {seen} kernels found in the reports"
    assert not problems, "\n".join(problems)
