"""kv_plan at its ends, against the plan in Python integers
(tests/paged_reference.py): steps in which nothing happens, sums of lengths
beyond 32 bits."""
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


def test_sums_beyond_32_bits(dev):
    """Lengths whose sums pass 2^31: they stop there, the requests before and
    the tokens that fit are planned as ever, and the shortage is reported."""
    big = top = 2 ** 31 - 1
    for R0 in (0, 3, 40, 1100):  # the sums pass 2^31 in the first thread, a warp, a block's warps
        ctx, new = [5] * R0 + [big, 0, big - 2, 7, 1], [1] * R0 + [big, big, 5, big, 3]
        table = torch.full((len(ctx), 4), -1, dtype=torch.int32, device="cuda")
        table[:, 0] = torch.arange(len(ctx))
        free = torch.arange(2000, 2009, dtype=torch.int32, device="cuda")
        T = R0 + 6
        p = q.kv_plan(i32(ctx), i32(new), table, free, 16, T)
        assert q.qmm_device_status(clear=True) == q.QMM_DEV_KV_SHORT
        cu = [0]
        for n in new:
            cu.append(min(cu[-1] + n, top))
        assert p.cu_new.tolist() == cu
        assert p.kv_lens.tolist() == [min(c + n, top) for c, n in zip(ctx, new)]
        assert p.positions.tolist() == [5] * R0 + [top] * 6
        assert p.slots.tolist() == [16 * r + 5 for r in range(R0)] + [-1] * 6
        # four columns: all of request R0 + 1's, three of R0 + 3's and none of the others'
        assert p.blocks_used.tolist() == [4 + 3]
        assert table[R0].tolist() == [R0, -1, -1, -1]
        assert table[R0 + 1].tolist() == [2000, 2001, 2002, 2003]
        assert table[R0 + 3].tolist() == [R0 + 3, 2004, 2005, 2006]
