"""attn_paged and attn_prompt where a call's lengths, table or values are at
their ends, against plain 64-bit numpy (tests/paged_reference.py): every kernel
behind the two calls, whole units and divided ones."""
import numpy as np
import pytest
import torch

import group_quantized_moe_gb300 as q
import paged_reference as ref
from parity_checks import assert_within
from test_gpu_paged import BF16, F32, cu_of, dev, i32, num, rnd, round_bound  # noqa: F401 (dev: fixture)

pytestmark = pytest.mark.gpu


def tensor_core(dtype, hd):
    """The calls whose weights are rounded to bf16 where they meet the values."""
    return dtype == BF16 and hd <= 128 and hd % 8 == 0


# query heads, key/value heads, head size, tokens a request: few rows (attn_rows_kernel;
# attn_tc_kernel, one query tile), many (attn_tile_kernel; attn_tc_kernel, two), and
# the sizes that attn_simt_kernel takes
FORMS = [(4, 2, 64, 1), (8, 1, 128, 1), (8, 2, 64, 60), (2, 2, 80, 200), (8, 2, 256, 1), (16, 2, 256, 20),
         (4, 1, 512, 40), (3, 3, 20, 2), (6, 1, 36, 70)]


def make(seed, R, n, nh, nkv, hd, S, cols, dtype):
    """R requests of n tokens each over a table of `cols` columns; behind them
    the row holds more blocks of the cache, which no call may use."""
    nb = R * (cols + 4)
    k, v = (rnd(seed + i, (nb, nkv, S, hd), dtype).cuda() for i in (1, 2))
    wide = np.random.default_rng(seed).permutation(nb).astype(np.int32).reshape(R, cols + 4)
    x = rnd(seed, (R * n, nh, hd), dtype, 2.0).cuda()
    return x, k, v, wide, torch.from_numpy(wide).cuda()[:, :cols]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd,n", FORMS)
def test_more_cache_rows_than_the_table_holds(dev, nh, nkv, hd, n, dtype):
    """Query i sees the keys j <= L - n + i that the table holds, whatever L is
    beyond it, and the missing keys are reported."""
    for S, cols in ((16, 3), (32, 21), (16, 130)):
        cap = S * cols
        lens = [cap, cap + 1, max(cap - 1, 0), cap + n, cap + n // 2, cap + 7 * n + 900, 2 ** 31 - 1, 5]
        x, k, v, wide, table = make(hd + n, len(lens), n, nh, nkv, hd, S, cols, dtype)
        y = q.attn_paged(x, q.PagedKV(k, v), table, cu_of([n] * len(lens)), i32(lens))
        assert q.qmm_device_status(clear=True) == q.QMM_DEV_BAD_BLOCK
        # the reference takes the keys behind the table for ones in blocks outside the cache
        short = [min(L, cap + 2 * n) for L in lens]
        full = np.full((len(lens), -(-max(short) // S)), -1, dtype=np.int32)
        full[:, :cols] = wide[:, :cols]
        want, b = ref.paged(num(x), num(k), num(v), full, [(L, n) for L in short], hd ** -0.5,
                            tensor_core(dtype, hd))
        assert_within(num(y), want, round_bound(want, b, F32), f"S{S} cols{cols}")
        # lengths up to the table's end, and idle requests beyond it, report nothing
        q.attn_paged(x[:n], q.PagedKV(k, v), table[:2], cu_of([n, 0]), i32([cap, cap + 99]))
        assert q.qmm_device_status(clear=True) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd,n", FORMS)
def test_fewer_rows_than_the_tokens(dev, nh, nkv, hd, n, dtype):
    """cu_q beyond the rows of q: the rows there are see the same keys."""
    S, cols, more = 16, 40, 37
    L = 300 + n + more
    x, k, v, wide, table = make(hd, 2, n, nh, nkv, hd, S, cols, dtype)
    cache = q.PagedKV(k, v)
    y = q.attn_paged(x, cache, table, i32([0, n, 2 * n + more]), i32([n, L]))
    want, b = ref.paged(num(x), num(k), num(v), wide, [(n, n), (L - more, n)], hd ** -0.5,
                        tensor_core(dtype, hd))
    assert_within(num(y), want, round_bound(want, b, F32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd,n", FORMS)
def test_nan_queries_and_keys_reach_their_rows(dev, nh, nkv, hd, n, dtype):
    """A row whose scores hold a NaN is NaN, wherever the NaN lies (alone in its
    part of a divided unit, behind every key of the row's maximum) and however
    small that part's weight is; the other rows are as without it."""
    S = 16
    for L in (n, n + 8, n + 128, 4000 + n):  # parts of one key, and of many
        cols = -(-L // S)
        x, k, v, wide, table = make(hd + L, 2, n, nh, nkv, hd, S, cols, dtype)
        cache, cu, kvl = q.PagedKV(k, v), cu_of([n, n]), i32([L, L])
        clean = q.attn_paged(x, cache, table, cu, kvl)
        x2 = x.clone()
        x2[n - 1] = float("nan")
        y = q.attn_paged(x2, cache, table, cu, kvl)
        assert y[n - 1].isnan().all(), L
        y[n - 1] = clean[n - 1]
        assert torch.equal(y, clean), L
        for j in (L - 1, L - n, (L - n) // 2, 0):
            k2 = k.clone()
            k2[wide[0, j // S], :, j % S] = float("nan")
            y = q.attn_paged(x, q.PagedKV(k2, v), table, cu, kvl)
            first = max(0, j - (L - n))  # the first row that sees key j
            assert y[first:n].isnan().all(), (L, j)
            assert torch.equal(y[:first], clean[:first]) and torch.equal(y[n:], clean[n:]), (L, j)
        # a part of little weight: one key far above the others, the NaN far away
        k2, x2 = k.clone(), x.clone()
        k2[wide[0, (L - n) // 2 // S], :, (L - n) // 2 % S] = 100.0
        x2[:n] = x2[:n].abs() + 1.0
        k2[wide[0, (L - n) // S], :, (L - n) % S] = float("nan")
        y = q.attn_paged(x2, q.PagedKV(k2, v), table, cu, kvl)
        assert y[:n].isnan().all(), L


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd", [(4, 4, 64), (8, 1, 128), (32, 8, 64), (24, 24, 100), (4, 4, 256)])
def test_nan_queries_of_prompts_reach_their_rows(dev, nh, nkv, hd, dtype):
    for lens in ([9, 40], [300, 700], [1500]):
        T = sum(lens)
        x, k, v = (rnd(s, (T, h, hd), dtype).cuda() for s, h in ((1, nh), (2, nkv), (3, nkv)))
        clean = q.attn_prompt(x, k, v, cu_of(lens))
        for t in (0, lens[0] - 1, T - 1):
            x2 = x.clone()
            x2[t] = float("nan")
            y = q.attn_prompt(x2, k, v, cu_of(lens))
            assert y[t].isnan().all(), (lens, t)
            y[t] = clean[t]
            assert torch.equal(y, clean), (lens, t)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("hd", [64, 512])
def test_cache_of_one_head_laid_out_by_rows(dev, hd, dtype):
    """One key/value head: blocks made as [rows, 1, columns] and seen as [1, rows,
    columns]."""
    nh, S, nb, L = 4, 16, 9, 130
    k, v = (rnd(i, (nb, S, 1, hd), dtype).cuda().transpose(1, 2) for i in (1, 2))
    x = rnd(3, (3, nh, hd), dtype).cuda()
    table = torch.arange(nb, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    y = q.attn_paged(x, q.PagedKV(k, v), table, cu_of([3]), i32([L]))
    want, b = ref.paged(num(x), num(k), num(v), table.cpu().numpy(), [(L, 3)], hd ** -0.5,
                        tensor_core(dtype, hd))
    assert_within(num(y), want, round_bound(want, b, F32))


# bf16 on the CUDA cores: weights in fp32, so none of the allowance for weights
# rounded to bf16
CORES = [(2, 1, 4), (3, 3, 20), (16, 2, 60), (20, 1, 84), (24, 24, 100), (4, 2, 132), (2, 1, 256), (8, 4, 256),
         (2, 2, 260), (4, 1, 512), (64, 1, 512)]


@pytest.mark.parametrize("y_dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd", CORES)
def test_bf16_on_the_cuda_cores_keeps_its_weights_in_fp32(dev, monkeypatch, nh, nkv, hd, y_dtype):
    import test_gpu_paged as t
    monkeypatch.setattr(t, "tensor_core", lambda dtype: False)
    t.run_prompt([37, 1, 0, 150], nh, nkv, hd, BF16, y_dtype, pad=2)
    t.run_prompt([500], nh, nkv, hd, BF16, y_dtype, seed=3)
    t.run_paged(t.DECODE, nh, nkv, hd, 16, BF16, y_dtype)
    t.run_paged([(3000, 1)], nh, nkv, hd, 64, BF16, y_dtype)
    t.run_paged([(300, 40), (64, 64), (17, 5), (3, 9)], nh, nkv, hd, 32, BF16, y_dtype, bad=[(0, 2)])


@pytest.mark.parametrize("nh,nkv,hd", [(4, 2, 64), (16, 8, 128)])
def test_bf16_rows_of_8_bytes_take_the_cuda_cores(dev, nh, nkv, hd):
    """Rows a multiple of 8 bytes apart, not of 16: no tensor map, the same results."""
    n, L = 90, 200
    pad = lambda seed, h: rnd(seed, (n, h * hd + 4), BF16).cuda()[:, :h * hd].view(n, h, hd)
    x, k, v = pad(1, nh), pad(2, nkv), pad(3, nkv)
    y = q.attn_prompt(x, k, v, cu_of([50, 40]))
    want, b = ref.prompt(num(x), num(k), num(v), [50, 40], hd ** -0.5)
    assert_within(num(y), want, round_bound(want, b, F32))
    S, nb = 16, 13
    both = rnd(4, (nb, 2 * nkv * S * hd + 8), BF16).cuda()  # blocks of 16-byte distance, queries not
    kc, vc = (both[:, i * nkv * S * hd:(i + 1) * nkv * S * hd].view(nb, nkv, S, hd) for i in range(2))
    table = torch.arange(nb, dtype=torch.int32, device="cuda")[None]
    y = q.attn_paged(x, q.PagedKV(kc, vc), table, cu_of([n]), i32([L]))
    want, b = ref.paged(num(x), num(kc), num(vc), table.cpu().numpy(), [(L, n)], hd ** -0.5)
    assert_within(num(y), want, round_bound(want, b, F32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd,n", FORMS)
def test_nan_values_reach_every_row_that_sees_them(dev, nh, nkv, hd, n, dtype):
    """A NaN value makes the rows NaN that see its key, also where the key lies so
    far below the row's maximum that its weight, or its whole part's, is zero
    in fp32; rows that do not see it are as without it."""
    S = 16
    for L in (n + 8, n + 131, 4000 + n):
        cols = -(-L // S)
        x, k, v, wide, table = make(hd + L, 2, n, nh, nkv, hd, S, cols, dtype)
        x = x.abs() + 1.0
        top = 0  # every row sees key 0, far above the others
        k[wide[0, top // S], :, top % S] = 100.0
        cache, cu, kvl = q.PagedKV(k, v), cu_of([n, n]), i32([L, L])
        clean = q.attn_paged(x, cache, table, cu, kvl)
        assert torch.isfinite(clean).all()
        for j in (L - 1, L - n, (L - n) // 2, 1):
            v2 = v.clone()
            v2[wide[0, j // S], :, j % S] = float("nan")
            y = q.attn_paged(x, q.PagedKV(k, v2), table, cu, kvl)
            first = max(0, j - (L - n))
            assert y[first:n].isnan().all(), (L, j)
            assert torch.equal(y[:first], clean[:first]) and torch.equal(y[n:], clean[n:]), (L, j)
