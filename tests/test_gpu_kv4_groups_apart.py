"""Attention over a 4-bit cache whose groups of values lie many powers of two apart:
every group is held to a bound of its own scales, as if the others were not there
(tests/kv4_reference.py derives it; its term for parts below fp16's normal range,
2^-29 of the largest weight times scale, goes by the group)."""
import numpy as np
import pytest
import torch

import group_quantized_moe_gb300 as q
import kv4_reference as ref
from parity_checks import assert_within
from test_gpu_kv4 import pack
from test_gpu_paged import BF16, F32, cu_of, dev, i32, num, rnd, round_bound  # noqa: F401 (dev: fixture)

pytestmark = pytest.mark.gpu


def run_apart(lens, nh, nkv, hd, group, dtype, exponents, seed=1, S=16, qs=2.0):
    """exponents: of rng and [blocks, nkv, S, G], the powers of two that the groups of
    values are multiplied by."""
    rng = np.random.default_rng(seed)
    need = [-(-L // S) for L, _ in lens]
    nb, G = sum(need), -(-hd // group)
    table, used = np.full((len(lens), max(need)), -1, dtype=np.int32), 0
    for r, m in enumerate(need):
        table[r, :m] = np.arange(used, used + m)
        used += m
    k, v = rng.standard_normal((2, nb, nkv, S, hd))
    v = v * np.repeat(2.0 ** exponents(rng, (nb, nkv, S, G)), group, -1)[..., :hd]
    data = pack(ref.quantise(k.astype(np.float32), group), ref.quantise(v.astype(np.float32), group), hd, group, S)
    T = sum(n for _, n in lens)
    qq = rnd(seed, (T, nh, hd), dtype, qs).cuda()
    y = q.attn_paged(qq, q.PagedKV4(torch.from_numpy(data).cuda(), hd, group, S), torch.from_numpy(table).cuda(),
                     cu_of([n for _, n in lens]), i32(L for L, _ in lens))
    assert q.qmm_device_status(clear=True) == 0
    kk, vv = ref.unpack(data, hd, group, S)
    t = 0
    for r, (L, n) in enumerate(lens):
        j = np.arange(L)
        keys, vals = ([x[table[r][j // S], :, j % S] for x in part] for part in (kk, vv))
        vis = j[None, :] <= (L - n + np.arange(n))[:, None]
        for g in range(G):
            only = [vals[0], vals[1], vals[2] * (np.arange(G) == g)]
            want, b = ref.attend(num(qq[t:t + n]), keys, only, group, vis, hd ** -0.5, dtype == F32)
            d = slice(g * group, min(hd, (g + 1) * group))
            assert_within(num(y[t:t + n])[..., d], want[..., d], round_bound(want[..., d], b[..., d], F32),
                          f"request {r}: group {g} of {hd}, {dtype}")
        t += n


HEADS = [(8, 2, 128, 64), (4, 4, 64, 32), (6, 1, 128, 32), (3, 3, 96, 64), (4, 2, 256, 64), (2, 1, 200, 32)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("apart", [16, 24, 32, 40])
@pytest.mark.parametrize("nh,nkv,hd,group", HEADS)
def test_groups_apart(dev, nh, nkv, hd, group, apart, dtype):
    """Every second group 2^-apart of the others, over one tile and many."""
    by = lambda rng, shape: np.broadcast_to(-apart * (np.arange(shape[-1]) % 2), shape).astype(float)
    run_apart([(900, 1), (20, 1), (300, 2)], nh, nkv, hd, group, dtype, by)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd,group", HEADS)
def test_groups_of_any_scale(dev, nh, nkv, hd, group, dtype):
    """Every group of every row another power of two, from 2^-30 to 2^30."""
    run_apart([(700, 1), (1500, 2)], nh, nkv, hd, group, dtype, lambda rng, shape: rng.integers(-30, 31, shape).astype(float))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_groups_that_grow_and_shrink(dev, dtype):
    """One group's scales grow with the keys while the other's shrink."""
    def by(rng, shape):
        up = np.linspace(-40, 40, shape[0] * shape[2]).reshape(shape[0], 1, shape[2], 1)
        return np.concatenate([up, -up], -1) + np.zeros(shape)

    for L in (31, 400, 3000):
        run_apart([(L, 1)], 4, 2, 128, 64, dtype, by)
