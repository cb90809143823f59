"""rope_append where its cache or its rows are at their ends."""
import pytest
import torch

import group_quantized_moe_gb300 as q
from test_gpu_paged import BF16, F32, dev, i32, rnd  # noqa: F401 (dev: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_cache_without_blocks(dev, dtype):
    """Every slot lies beyond a cache of no blocks: queries, keys and values as
    without a cache, nothing stored, and the flag that a larger cache's missing
    slot sets; padding and tokens without a slot set none."""
    nh, nkv, hd, S = 2, 1, 8, 16
    cos, sin = q.rope_table(10, hd, device=dev)
    cache = q.paged_kv(0, nkv, S, hd, dtype=dtype, device=dev)
    x = rnd(1, (3, (nh + 2 * nkv) * hd), F32).cuda()
    pos = i32([1, 2, -1])
    want = q.rope_append(x, nh, pos, None, cos, sin, None, keep_kv=True, n_kv=nkv, y_dtype=dtype)
    for slots, status in (([0, 5, 7], q.QMM_DEV_BAD_BLOCK), ([-1, 40, 0], q.QMM_DEV_BAD_BLOCK),
                          ([-1, -1, 3], 0)):
        got = q.rope_append(x, nh, pos, torch.tensor(slots, device=dev), cos, sin, cache, keep_kv=True)
        assert q.qmm_device_status(clear=True) == status, slots
        assert all(torch.equal(a, b) for a, b in zip(got, want))
