"""Registers and spills of the paged-cache and batched-attention kernels, checked
at compile time on the CPU (see tests/test_kernel_resources.py).

attn_tc_kernel divides its registers between its warps with setmaxnreg: two
warpgroups of 208 and one of 88 make 3 x 168, so a build that gave it fewer
than 168 at launch would wait for registers that never come.  The others must
stay within what their CTAs per SM leave, without spills but for two kernels
whose launch bounds are worth a few spilled words (times beside the code), and
the narrowest form of attn_simt_kernel, which the compiler holds at 128
registers (bf16 head sizes up to 64 that the tensor cores do not take).
"""
import os
import re
import shutil
from concurrent.futures import ThreadPoolExecutor

import pytest

from test_kernel_resources import ENTRY, REGS, SPILL, _report

UNITS = ["attn_tc.cu", "attn_rows.cu", "attn_tile.cu", "attn_simt.cu", "rope_append.cu", "kv_plan.cu"]
# bytes of spill loads that a kernel may have
SPILLS = {"attn_tile_kernelILi1EE": 64, "attn_simt_kernelILb1ELi1ELi64EE": 64,
          "rope_append_kernelILi4E": 32, "rope_append_kernelILi8E": 128}
# registers a thread: 65536 by threads and CTAs per SM
LIMITS = {"attn_tc_kernel": 168, "rope_append_kernel": 48, "kv_plan_kernel": 64, "attn_join_kernel": 255,
          "attn_tile_kernelILi1EE": 128, "attn_tile_kernelILi2EE": 255, "attn_simt_kernel": 255}


def _limit(name):
    m = re.search(r"attn_rows_kernelILb[01]ELi(\d+)ELi(\d+)E", name)
    if m:  # two CTAs of 256 threads up to four pieces of results a lane, then one
        return 128 if int(m.group(1)) * int(m.group(2)) <= 4 else 255
    return next((v for k, v in LIMITS.items() if k in name), None)


def test_serving_kernels_fit_their_register_budget(tmp_path):
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
                used, limit = int(m.group(1)), _limit(name)
                if limit is None or used > limit:
                    problems.append(f"{name} uses {used} registers, budget {limit}")
                if "attn_tc_kernel" in name and used != 168:
                    problems.append(f"{name} is launched with {used} registers, its split needs 168")
                name = None
    assert seen >= 40, f"only {seen} kernels found in the reports"
    assert not problems, "\n".join(problems)
