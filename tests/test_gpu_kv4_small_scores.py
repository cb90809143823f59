"""Attention over a 4-bit cache at the ends of the range: queries and a scale so
small that their product leaves fp32's, where all weights are equal and a row is the
mean of the values it sees; queries and keys far from one."""
import numpy as np
import pytest
import torch

import group_quantized_moe_gb300 as q
import kv4_reference as ref
from parity_checks import assert_within
from test_gpu_kv4 import filled, pack
from test_gpu_paged import BF16, F32, cu_of, dev, i32, num, rnd, round_bound  # noqa: F401 (dev: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("q_exp,scale", [(-110, 1e-30), (0, 1e-44), (-60, 1e-40), (40, 1e-38), (-120, 0.125)])
@pytest.mark.parametrize("lens", [[(100, 1), (37, 2)], [(300, 60), (77, 77)]])
def test_scores_near_zero(dev, lens, q_exp, scale, dtype):
    nh, nkv, hd, group, S = 4, 2, 64, 32, 16
    need = [-(-L // S) for L, _ in lens]
    data = filled(sum(need), nkv, hd, group, S, 3)
    table = np.full((len(lens), max(need)), -1, dtype=np.int32)
    for r, m in enumerate(need):
        table[r, :m] = np.arange(m) + sum(need[:r])
    T = sum(n for _, n in lens)
    qq = (rnd(2, (T, nh, hd), F32).double() * 2.0 ** q_exp).to(dtype).cuda()
    y = q.attn_paged(qq, q.PagedKV4(torch.from_numpy(data).cuda(), hd, group, S), torch.from_numpy(table).cuda(),
                     cu_of([n for _, n in lens]), i32(L for L, _ in lens), scale=scale)
    assert q.qmm_device_status(clear=True) == 0
    want, b = ref.paged(num(qq), data, group, S, table, lens, float(np.float32(scale)), dtype == F32)
    assert_within(num(y), want, round_bound(want, b, F32), f"{dtype} {q_exp} {scale}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("e", [80, -80])
@pytest.mark.parametrize("lens", [[(500, 1), (37, 2)], [(400, 90), (77, 77)]])
def test_queries_and_keys_far_from_one(dev, lens, e, dtype):
    """Keys of 2^e and queries of 2^-e: scores are what they are for ordinary ones."""
    nh, nkv, hd, group, S = 4, 2, 128, 64, 16
    rng = np.random.default_rng(4)
    need = [-(-L // S) for L, _ in lens]
    k, v = rng.standard_normal((2, sum(need), nkv, S, hd))
    data = pack(ref.quantise((k * 2.0 ** e).astype(np.float32), group), ref.quantise(v.astype(np.float32), group),
                hd, group, S)
    table = np.full((len(lens), max(need)), -1, dtype=np.int32)
    for r, m in enumerate(need):
        table[r, :m] = np.arange(m) + sum(need[:r])
    T = sum(n for _, n in lens)
    qq = (rnd(2, (T, nh, hd), F32, 2.0).double() * 2.0 ** -e).to(dtype).cuda()
    y = q.attn_paged(qq, q.PagedKV4(torch.from_numpy(data).cuda(), hd, group, S), torch.from_numpy(table).cuda(),
                     cu_of([n for _, n in lens]), i32(L for L, _ in lens))
    assert q.qmm_device_status(clear=True) == 0
    # the bound of ordinary keys and queries, of which these are powers of two
    near = pack(ref.quantise(k.astype(np.float32), group), ref.quantise(v.astype(np.float32), group), hd, group, S)
    want, b = ref.paged(num(qq) * 2.0 ** e, near, group, S, table, lens, hd ** -0.5, dtype == F32)
    assert_within(num(y), want, round_bound(want, b, F32), f"{dtype} 2^{e}")
