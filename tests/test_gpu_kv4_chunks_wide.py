"""The chunk kernel of the 4-bit cache (attn4_tc_kernel) over keys and values that
its straight conversions do not take: keys whose rows lie in other ranges than
fp16's, values with zero points beyond bf16's whole numbers, beside ordinary ones.
Against plain numpy in 64 bits.

Bound, with u = 2^-24 (the tensor cores cut a sum off where fp32 would round, 2 u a
term) and a score s = scale q.k:
  score    a key is rounded to fp16, half a step (2^-11), its row divided by a power
           of two where that keeps it in range: a row's bound (|zp| + 16) s goes to
           [2^13, 2^14), so that what is below fp16's normal numbers is off by 2^-25
           or 2^-38 of the bound.  Queries are bf16 elements times a power of two, the
           row's largest at least 2^14: exact but for 2^-25, 2^-39 of the largest.
           Sums 2 u (hd + 16), and 4 u of the score for its factors.
  weight   relative e = expm1(error of the score) + 2^-21 (the exponential's own)
  result   weights and values are rounded to bf16, 2^-8 each, sums 2 (L + 64) u
"""
import numpy as np
import pytest
import torch

import group_quantized_moe_gb300 as q
import kv4_reference as ref
from parity_checks import assert_within
from test_gpu_kv4 import pack
from test_gpu_paged import BF16, F32, cu_of, dev, i32, num, rnd, round_bound  # noqa: F401 (dev: fixture)

pytestmark = pytest.mark.gpu


def attend_tiles(qr, keys, vals, group, visible, scale):
    """qr [n, nh, hd]; keys, vals: codes [L, nkv, hd], zps, scales [L, nkv, G]
    -> y, bound [n, nh, hd].  Every row sees a key."""
    n, nh, hd = qr.shape
    L, nkv = keys[0].shape[:2]
    k, v = ref.values(keys, group), ref.values(vals, group)
    row = ((np.abs(keys[1]) + 16) * keys[2]).max(-1)  # [L, nkv]
    y, b = np.zeros((n, nh, hd)), np.zeros((n, nh, hd))
    for h in range(nh):
        g = h // (nh // nkv)
        qh = np.abs(qr[:, h])
        s = np.where(visible, scale * (qr[:, h] @ k[:, g].T), -np.inf)
        size = qh @ np.abs(k[:, g]).T
        es = scale * ((2.0 ** -11 + 2 * ref.U * (hd + 16)) * size
                      + 2.0 ** -38 * qh.sum(axis=1, keepdims=True) * row[None, :, g]
                      + 2.0 ** -39 * qh.max(axis=1, keepdims=True) * np.abs(k[:, g]).sum(-1)[None])
        es = es + 4 * ref.U * np.where(visible, np.abs(s), 0).max(axis=1, keepdims=True)
        p = np.where(visible, np.exp(s - s.max(axis=1, keepdims=True)), 0)
        p /= p.sum(axis=1, keepdims=True)
        e = np.expm1(es) + 2.0 ** -21
        e = e + (p * e).sum(axis=1, keepdims=True) + 2 * 2.0 ** -8 + 2.0 ** -16 + 2 * (L + 64) * ref.U
        y[:, h] = p @ v[:, g]
        b[:, h] = (p * e) @ np.abs(v[:, g])
    return y, b


def run_chunks(lens, nh, nkv, hd, group, S, keys, values, q_exp, seed=1, y_dtype=F32, repeats=1,
               positive=False):
    """keys, values: from a generator and a shape [blocks, nkv, S, hd], the rows as
    numbers; queries of about 2^q_exp, positive ones if asked."""
    rng = np.random.default_rng(seed)
    need = [-(-L // S) for L, _ in lens]
    nb = sum(need) + 2
    ids = rng.permutation(nb).astype(np.int32)
    table, used = np.full((len(lens), max(need)), -1, dtype=np.int32), 0
    for r, m in enumerate(need):
        table[r, :m] = ids[used:used + m]
        used += m
    shape = (nb, nkv, S, hd)
    parts = [ref.quantise(f(rng, shape).astype(np.float32), group) for f in (keys, values)]
    data = pack(*parts, hd, group, S)
    T, grp = sum(n for _, n in lens), nh // nkv
    assert T * grp > 32 * len(lens) and len(lens) < 6 or all(n * grp > 32 for _, n in lens)  # all of it in tiles
    qq = (rnd(seed, (T, nh, hd), BF16, 2.0).float() * 2.0 ** q_exp).bfloat16().cuda()
    qq = qq.abs() if positive else qq
    args = (qq, q.PagedKV4(torch.from_numpy(data).cuda(), hd, group, S), torch.from_numpy(table).cuda(),
            cu_of([n for _, n in lens]), i32(L for L, _ in lens))
    y = q.attn_paged(*args, y_dtype=y_dtype)
    for _ in range(repeats):
        assert torch.equal(q.attn_paged(*args, y_dtype=y_dtype), y)
    assert q.qmm_device_status(clear=True) == 0
    kk, vv = ref.unpack(data, hd, group, S)
    t = 0
    for r, (L, n) in enumerate(lens):
        j = np.arange(L)
        rows = [[x[table[r][j // S], :, j % S] for x in part] for part in (kk, vv)]
        want, b = attend_tiles(num(qq[t:t + n]), *rows, group, j[None, :] <= (L - n + np.arange(n))[:, None], hd ** -0.5)
        assert_within(num(y[t:t + n]), want, round_bound(want, b, y_dtype), f"request {r}: {n} tokens of {L}")
        t += n
    return parts


def normal(rng, shape):
    return rng.standard_normal(shape)


def scaled(exponents):
    """Rows of 2^e, e drawn from `exponents` for each."""
    return lambda rng, shape: rng.standard_normal(shape) * 2.0 ** rng.choice(exponents, shape[:3] + (1,))


# (exponents of the key rows, of the queries): scores of the largest rows are of order one
KEYS = {"40 down to -40": (np.arange(-40, 41, 8), -40), "tiny": (np.arange(-40, -34), 36), "huge": (np.arange(30, 38), -36),
        "some rows 2^20": (np.array([0, 0, 0, 0, 20]), -20), "some rows 2^-16": (np.array([0, 0, -16]), 0),
        "2^14 and 2^16": (np.array([14, 16]), -16)}
# one and two query tiles a unit, units cut between workers
LENS = {"single": [(1300, 20), (1000, 14), (260, 10), (1, 1)], "pairs": [(1500, 300), (700, 700)]}


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("keys", KEYS)
@pytest.mark.parametrize("nh,nkv,hd,group", [(8, 2, 128, 64), (16, 4, 64, 32)])
def test_key_rows_out_of_range(dev, nh, nkv, hd, group, keys, lens):
    exponents, q_exp = KEYS[keys]
    run_chunks(LENS[lens], nh, nkv, hd, group, 16, scaled(exponents), normal, q_exp, repeats=3)


@pytest.mark.parametrize("nh,nkv,hd,group,S", [(4, 1, 96, 32, 32), (8, 2, 72, 64, 64), (5, 1, 32, 32, 16), (12, 3, 128, 32, 128)])
def test_key_rows_out_of_range_other_heads(dev, nh, nkv, hd, group, S):
    run_chunks([(900, 200), (300, 64)], nh, nkv, hd, group, S, scaled(np.arange(-24, 25, 8)), normal, -24, y_dtype=BF16)


@pytest.mark.parametrize("n,L", [(10, 700), (70, 450)])
def test_key_rows_out_of_range_many_units(dev, n, L):
    """Several units to a worker, of one query tile and of two, each of more key
    tiles than there are stages: the same bits every time."""
    run_chunks([(L - r % 7, n) for r in range(110)], 8, 2, 128, 64, 16, scaled(np.arange(20, 26)), normal, -24, repeats=10)


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("nh,nkv,hd,group", [(8, 2, 128, 64), (16, 4, 64, 32), (4, 1, 96, 32)])
def test_value_zero_points_out_of_range(dev, nh, nkv, hd, group, lens):
    """Groups of values far from zero beside their range: zero points of both signs,
    from within bf16's whole numbers to the largest."""
    def values(rng, shape):
        g = -(-hd // group)
        mean = np.repeat(rng.choice([-1.0, 1.0], shape[:3] + (g,)) * np.exp(rng.standard_normal(shape[:3] + (g,))), group, -1)
        narrow = np.repeat(2.0 ** -rng.integers(0, 16, shape[:3] + (g,)).astype(float), group, -1)
        return (mean * (1 + narrow * rng.standard_normal(mean.shape)))[..., :hd]

    _, (_, zp, _) = run_chunks(LENS[lens], nh, nkv, hd, group, 32, normal, values, 0)
    for lo, hi in ((0, 100), (121, 1000), (2000, 2049)):
        assert (np.abs(zp) >= lo).sum() > 50 and ((np.abs(zp) >= lo) & (np.abs(zp) < hi)).any()
    assert (zp < -1000).any() and (zp > 1000).any()


def test_values_of_any_scale(dev):
    run_chunks(LENS["pairs"], 8, 2, 128, 64, 16, normal, scaled(np.arange(-40, 41, 8)), 0)


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("nh,nkv,hd,group", [(8, 2, 128, 64), (16, 4, 64, 32), (4, 1, 96, 32)])
def test_narrow_key_groups(dev, nh, nkv, hd, group, lens):
    """Groups of keys far from zero beside their range, whose scales are below fp16's
    normal numbers although their values are not.  Scales rounded to fp16 would be off
    by as much for every value of a row: values have the sign of that error."""
    row = {}

    def keys(rng, shape):
        g = shape[:3] + (-(-hd // group), 1)
        row["s"] = s = rng.choice(np.arange(129, 160, 2), shape[:3] + (1, 1)) * 2.0 ** -25
        z = rng.choice([-1, 1], g) * np.rint(0.0037 / s)
        codes = rng.integers(0, 16, g[:4] + (group,))
        codes[..., 0], codes[..., 1] = 0, 15
        return ((z + codes) * s).reshape(shape[:3] + (-1,))[..., :hd]

    def values(rng, shape):
        s = row["s"][..., 0]
        return np.where(s.astype(np.float16) > s, 1.0, -1.0) * (1 + 0.1 * rng.standard_normal(shape))

    (_, zp, s), _ = run_chunks(LENS[lens], nh, nkv, hd, group, 16, keys, values, 12, positive=True)
    assert (s < 2.0 ** -14).all() and ((np.abs(zp) + 16) * s >= 2.0 ** -9).all() and (np.abs(zp) <= 1000).all()


@pytest.mark.parametrize("exponents", [(0,), (0, -24), (20, 24)])
def test_key_groups_of_zeros(dev, exponents):
    """Zeros in some groups and some rows, beside keys in fp16's range and out of it."""
    def keys(rng, shape):
        k = scaled(exponents)(rng, shape)
        k[..., :64] *= rng.random(shape[:3] + (1,)) < 0.7
        k[..., 64:] *= rng.random(shape[:3] + (1,)) < 0.7
        return k

    (_, zp, s), _ = run_chunks(LENS["pairs"], 8, 2, 128, 64, 16, keys, normal, -max(exponents))
    assert ((s == 2.0 ** -100) & (zp == 0)).any() and (s == 2.0 ** -100).all(-1).any()


@pytest.mark.parametrize("exponents", [(0,), (0, 24)])
@pytest.mark.parametrize("n", [12, 200])
def test_nan_keys_beside_rows_out_of_range(dev, n, exponents):
    """A NaN in a group of a key reaches the queries that see it, and only them."""
    nh, nkv, hd, group, S, L = 8, 2, 128, 64, 16, 600
    rng = np.random.default_rng(6)
    nb = -(-L // S)
    k = scaled(exponents)(rng, (nb, nkv, S, hd)).astype(np.float32)
    v = rng.standard_normal((nb, nkv, S, hd)).astype(np.float32)
    qq = (rnd(3, (n, nh, hd), BF16).float() * 2.0 ** -max(exponents)).bfloat16().cuda()
    call = lambda k: q.attn_paged(qq, q.PagedKV4(torch.from_numpy(pack(
        ref.quantise(k, group), ref.quantise(v, group), hd, group, S)).cuda(), hd, group, S),
        torch.arange(nb, dtype=torch.int32, device="cuda")[None], i32([0, n]), i32([L]))
    clean = call(k)
    assert clean.isfinite().all()
    for j in (L - n // 2, L - 1):
        bad = k.copy()
        bad[j // S, :, j % S, 5] = np.nan
        y = call(bad)
        first = j - (L - n)
        assert torch.equal(y[:first], clean[:first]) and y[first:].isnan().all()


@pytest.mark.parametrize("n", [12, 200])
def test_largest_values_unseen(dev, n):
    """Values next to fp32's largest, which bf16 would round to infinity, reach no
    query that does not see them."""
    nh, nkv, hd, group, S, L = 8, 2, 128, 64, 16, 600
    rng = np.random.default_rng(6)
    nb = -(-L // S)
    k, v = rng.standard_normal((2, nb, nkv, S, hd)).astype(np.float32)
    qq = rnd(3, (n, nh, hd), BF16).cuda()
    call = lambda v: q.attn_paged(qq, q.PagedKV4(torch.from_numpy(pack(
        ref.quantise(k, group), ref.quantise(v, group), hd, group, S)).cuda(), hd, group, S),
        torch.arange(nb, dtype=torch.int32, device="cuda")[None], i32([0, n]), i32([L]))
    clean = call(v)
    for j in (L - n // 2, L - 1):
        large = v.copy()
        large[j // S, :, j % S] = np.where(np.arange(hd) % 2, np.float32(3.4e38), np.float32(0))
        first = j - (L - n)
        assert torch.equal(call(large)[:first], clean[:first])
