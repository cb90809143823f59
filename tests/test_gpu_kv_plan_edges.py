"""kv_plan at its ends, against the plan in Python integers
(tests/paged_reference.py): steps in which nothing happens."""
import pytest
import torch

import group_quantized_moe_gb300 as q
from test_gpu_paged import check_plan, dev, i32  # noqa: F401 (dev: fixture)

pytestmark = pytest.mark.gpu


def test_step_without_requests_and_tokens(dev):
    check_plan([], [], 16, T=0, cols=2)
    check_plan([], [], 64, T=0, cols=0, n_free=0)


def test_step_without_requests_overwrites_its_outputs(dev):
    """cu_new[0] and blocks_used are written, whatever they held."""
    out = q.alloc_kv_plan(0, 0)
    out.cu_new.fill_(7)
    out.blocks_used.fill_(7)
    table = torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    p = q.kv_plan(i32([]), i32([]), table, i32([4, 5]), 16, 0, out=out)
    assert p.cu_new.tolist() == [0] and p.blocks_used.tolist() == [0]
    assert q.qmm_device_status(clear=True) == 0
