"""The paged cache and the batched attention on the GPU, against plain 64-bit
numpy (tests/paged_reference.py, which derives the bounds): block tables and
slots exactly; rotated queries, cache rows and attention outputs within their
bounds; everything a call does not own left as it was."""
import numpy as np
import pytest
import torch

import group_quantized_moe_gb300 as q
import paged_reference as ref
from group_quantized_moe_gb300 import build_lib
from parity_checks import assert_within

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build_lib.build()
    q.lib()
    d = torch.device("cuda:0")
    torch.cuda.set_device(d)
    q.qmm_device_status(clear=True)
    yield d
    assert q.qmm_device_status(clear=True) == 0


def rnd(seed, shape, dtype, scale=1.0):
    """Values of the type itself, so that both sides start from the same numbers."""
    a = np.random.default_rng(seed).standard_normal(shape).astype(np.float32) * np.float32(scale)
    return torch.from_numpy(a).to(dtype)


def num(t):
    return t.cpu().double().numpy()


def i32(v):
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def cu_of(lens):
    return i32(np.concatenate([[0], np.cumsum(lens)]).astype(np.int64))


def round_bound(y, b, y_dtype):
    return b + (ref.HALF_BF16 if y_dtype == BF16 else ref.U) * (np.abs(y) + b)


def tensor_core(dtype):
    """bf16 calls may multiply the values by weights rounded to bf16."""
    return dtype == BF16


# ------------------------------------------------------------------- kv_plan

def check_plan(ctx, new, S, T=None, cols=None, n_free=None, seed=1, extra=0):
    rng = np.random.default_rng(seed)
    need = [-(-(max(c, 0) + max(n, 0)) // S) for c, n in zip(ctx, new)]
    have = [-(-max(c, 0) // S) for c in ctx]
    T = sum(max(n, 0) for n in new) if T is None else T
    cols = max(need + [1]) + 2 if cols is None else cols
    ids = rng.permutation(sum(need) + 5).astype(np.int32)
    table = np.full((len(ctx), cols), -7, dtype=np.int32)
    used = 0
    for r, h in enumerate(have):
        h = min(h, cols)
        table[r, :h] = ids[used:used + h]
        used += h
    free = ids[used:] if n_free is None else ids[used:used + n_free]
    want = ref.plan(ctx, new, table, free, S, T)
    wide = torch.full((len(ctx), cols + extra), -9, dtype=torch.int32, device="cuda")
    dt = wide[:, :cols]
    dt.copy_(torch.from_numpy(table))
    p = q.kv_plan(i32(ctx), i32(new), dt, torch.from_numpy(free.copy()).cuda(), S, T)
    np.testing.assert_array_equal(dt.cpu().numpy(), want[0])
    assert (wide[:, cols:] == -9).all()
    assert p.cu_new.tolist() == want[1] and p.kv_lens.tolist() == want[2]
    assert p.positions.tolist() == want[3]
    assert p.slots.tolist() == want[4]
    assert p.blocks_used.tolist() == [want[5]]
    assert q.qmm_device_status(clear=True) == (q.QMM_DEV_KV_SHORT if want[6] else 0)


@pytest.mark.parametrize("S", [16, 32, 64, 128, 256])
def test_plan_block_sizes(dev, S):
    check_plan([0, 0, S - 1, S, S + 1, 5 * S, 1], [1, 3 * S + 1, 1, 1, S, 0, S - 1], S)


@pytest.mark.parametrize("R", [1, 2, 31, 257, 1025, 3001])
def test_plan_many_requests(dev, R):
    rng = np.random.default_rng(R)
    ctx = rng.integers(0, 700, R) * (rng.random(R) < 0.8)
    new = rng.choice([0, 1, 1, 1, 2, 17, 90], R)
    check_plan([int(c) for c in ctx], [int(n) for n in new], 16, T=int(new.sum()) + 13,
               extra=7)


def test_plan_empty_and_negative(dev):
    check_plan([], [], 16, T=3, cols=2)
    check_plan([5, -3, 40], [0, 2, -1], 16)
    check_plan([7, 9], [0, 0], 32, T=0)


def test_plan_shortages(dev):
    check_plan([0, 0, 0], [40, 40, 40], 16, n_free=4)          # free list too short
    check_plan([0, 30], [70, 3], 16, cols=3)                   # table too narrow
    check_plan([100], [5], 16, cols=3)                         # ... for the context itself
    check_plan([0, 3], [40, 40], 16, T=50)                     # token buffers too short
    check_plan([4], [5], 16, cols=0, n_free=0)


# --------------------------------------------------------------- rope_append

@pytest.mark.parametrize("nh,nkv,hd,xd,yd,S,keep", [
    (4, 2, 64, F32, BF16, 16, True), (6, 1, 128, BF16, BF16, 64, False),
    (3, 3, 20, F32, F32, 32, True), (5, 5, 4, BF16, F32, 16, True), (8, 2, 512, F32, F32, 16, False),
    (2, 1, 260, BF16, BF16, 256, True), (28, 4, 80, F32, BF16, 128, True)])
def test_rope_append(dev, nh, nkv, hd, xd, yd, S, keep):
    rng = np.random.default_rng(hd)
    T, max_seq, nb = 37, 300, 9
    width = (nh + 2 * nkv) * hd
    big = rnd(hd + 1, (T, width + 8), xd).cuda()
    x = big[:, 8:]  # rows of a wider buffer, 8 elements in
    pos = rng.integers(0, max_seq, T).astype(np.int32)
    pos[5], slot = -1, rng.permutation(nb * S)[:T].astype(np.int64)
    slot[[3, 11]] = -1
    cos, sin = q.rope_table(max_seq, hd, device=dev)
    # keys and values interleaved in one allocation
    both = rnd(9, (nb, 2, nkv, S, hd), yd).cuda()
    before = both.clone()
    cache = q.PagedKV(both[:, 0], both[:, 1])
    gq, gk, gv = q.rope_append(x, nh, torch.from_numpy(pos).cuda(), torch.from_numpy(slot).cuda(),
                               cos, sin, cache, keep_kv=keep)
    y, b = ref.rope(num(x).reshape(T, -1, hd), pos, num(cos), num(sin), nh + nkv)
    bound = round_bound(y, b, yd) + 1e-30
    assert_within(num(gq), y[:, :nh], bound[:, :nh], "q")
    want, wb = num(before), np.zeros(both.shape) + 1e-30
    for t in range(T):
        if slot[t] >= 0 and pos[t] >= 0:
            blk, row = slot[t] // S, slot[t] % S
            for kv in range(2):
                h0 = nh + kv * nkv
                want[blk, kv, :, row] = y[t, h0:h0 + nkv]
                wb[blk, kv, :, row] = bound[t, h0:h0 + nkv]
    assert_within(num(both), want, wb, "cache")
    if keep:
        assert_within(num(gk), y[:, nh:nh + nkv], bound[:, nh:nh + nkv], "k")
        assert_within(num(gv), y[:, nh + nkv:], bound[:, nh + nkv:], "v")
    else:
        assert gk is None and gv is None


def test_rope_append_out_of_range(dev):
    nh, nkv, hd, S = 2, 1, 8, 16
    cos, sin = q.rope_table(10, hd, device=dev)
    cache = q.PagedKV(*(torch.zeros((2, nkv, S, hd), device=dev) for _ in range(2)))
    x = torch.ones((3, (nh + 2 * nkv) * hd), device=dev)
    gq, _, _ = q.rope_append(x, nh, i32([9, 10, 1]), torch.tensor([32, 0, 31], device=dev), cos, sin,
                             cache)
    assert q.qmm_device_status(clear=True) == q.QMM_DEV_BAD_POSITION | q.QMM_DEV_BAD_BLOCK
    assert (gq[1] == 0).all() and (gq[0] != 0).any()
    assert (cache.v[1, 0, 15] == 1).all() and cache.v.sum() == hd


def test_rope_append_without_a_cache(dev):
    cos, sin = q.rope_table(10, 16, device=dev)
    x = rnd(3, (4, 4 * 16), F32).cuda()
    gq, gk, gv = q.rope_append(x, 2, i32([0, 1, 2, 9]), None, cos, sin, None, keep_kv=True, n_kv=1)
    y, b = ref.rope(num(x).reshape(4, 4, 16), [0, 1, 2, 9], num(cos), num(sin), 3)
    got = torch.cat([gq, gk, gv], 1)
    assert_within(num(got), y, b + ref.U * np.abs(y) + 1e-30)


# --------------------------------------------------------------- attn_prompt

def run_prompt(lens, nh, nkv, hd, dtype, y_dtype=F32, pad=0, seed=1, strided=False, qs=2.0):
    T = sum(lens) + pad
    if strided:  # slices of one stacked projection, rows padded
        row = (nh + 2 * nkv) * hd
        buf = rnd(seed, (T, row + 16), dtype).cuda()
        buf[:, :nh * hd] *= qs
        qq = buf[:, :nh * hd].view(T, nh, hd)
        k = buf[:, nh * hd:(nh + nkv) * hd].view(T, nkv, hd)
        v = buf[:, (nh + nkv) * hd:row].view(T, nkv, hd)
    else:
        qq = rnd(seed, (T, nh, hd), dtype, qs).cuda()
        k, v = rnd(seed + 1, (T, nkv, hd), dtype).cuda(), rnd(seed + 2, (T, nkv, hd), dtype).cuda()
    y = torch.full((T, nh, hd), 7.0, dtype=y_dtype, device="cuda")
    q.attn_prompt(qq, k, v, cu_of(lens), y=y)
    want, b = ref.prompt(num(qq), num(k), num(v), lens, hd ** -0.5, tensor_core(dtype))
    assert_within(num(y), want, round_bound(want, b, y_dtype), f"{lens} {nh}/{nkv} d{hd} {dtype}")
    return y


SHAPES = [(4, 4, 64), (8, 2, 128), (6, 1, 128), (7, 1, 32), (16, 2, 64), (2, 2, 80), (12, 4, 96)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd", SHAPES)
def test_prompt_shapes(dev, nh, nkv, hd, dtype):
    run_prompt([1, 130, 0, 63, 17, 64, 65], nh, nkv, hd, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd", [(2, 1, 4), (3, 3, 20), (4, 2, 132), (2, 1, 256), (2, 2, 260),
                                       (4, 1, 512), (70, 1, 64), (160, 1, 16)])
def test_prompt_other_heads(dev, nh, nkv, hd, dtype):
    run_prompt([37, 1, 70], nh, nkv, hd, dtype)


@pytest.mark.parametrize("dtype,y_dtype", [(F32, BF16), (BF16, BF16), (BF16, F32)])
def test_prompt_strides_types_and_padding(dev, dtype, y_dtype):
    run_prompt([100, 3, 200], 8, 2, 64, dtype, y_dtype, pad=5, strided=True)
    run_prompt([0, 0], 4, 4, 64, dtype, y_dtype, pad=3)
    run_prompt([90, 41], 4, 4, 20, dtype, y_dtype, strided=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 255, 256, 257, 700])
def test_prompt_lengths(dev, n, dtype):
    run_prompt([n], 4, 1, 128, dtype, seed=n)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_long_and_many(dev, dtype):
    run_prompt([2500], 2, 1, 64, dtype)
    rng = np.random.default_rng(3)
    run_prompt([int(n) for n in rng.integers(0, 40, 150)], 4, 2, 64, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd", [(32, 8, 64), (32, 32, 128), (40, 4, 20), (24, 24, 100), (30, 5, 80),
                                       (16, 4, 132), (12, 12, 256), (8, 2, 260), (8, 1, 512)])
def test_prompt_many_rows(dev, nh, nkv, hd, dtype):
    """More query rows than the kernel for few rows takes, whole units and divided ones."""
    run_prompt([300, 1, 0, 77, 150, 64], nh, nkv, hd, dtype, pad=3, strided=hd % 8 == 0)
    run_prompt([700], nh, nkv, hd, dtype, qs=50.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd", [(8, 8, 20), (8, 8, 100), (4, 4, 256), (4, 4, 512)])
def test_prompt_many_short_ones(dev, nh, nkv, hd, dtype):
    """8 to 16 query rows a request and head."""
    rng = np.random.default_rng(4)
    run_prompt([int(n) for n in rng.integers(0, 24, 100)], nh, nkv, hd, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_sharp_scores(dev, dtype):
    """Scores of hundreds: the running maximum moves by far more than one weight's range."""
    run_prompt([400], 4, 2, 64, dtype, qs=100.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_prompt_unseen_values_do_not_matter(dev, dtype):
    """NaN and infinity in keys and values from row j on: rows before j as
    they are without them, rows from j on NaN (a NaN key or value reaches
    every later row)."""
    n, nh, nkv, hd = 300, 4, 2, 64
    qq, k, v = (rnd(s, (2 * n, h, hd), dtype).cuda() for s, h in ((1, nh), (2, nkv), (3, nkv)))
    clean = q.attn_prompt(qq, k, v, cu_of([n, n]))
    for j, what in ((0, "v"), (1, "v"), (150, "v"), (150, "k"), (290, "v"), (299, "v")):
        k2, v2 = k.clone(), v.clone()
        (v2 if what == "v" else k2)[j] = float("nan")
        y = q.attn_prompt(qq, k2, v2, cu_of([n, n]))
        assert torch.equal(y[:j], clean[:j]) and torch.equal(y[n:], clean[n:]), (j, what)
        assert y[j:n].isnan().all(), (j, what)
    v2 = v.clone()
    v2[200, :, 5] = float("inf")
    y = q.attn_prompt(qq, k, v2, cu_of([n, n]))
    assert torch.equal(y[:200], clean[:200])
    assert (y[200:n, :, 5] == float("inf")).all() and y[200:n, :, :5].isfinite().all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd", [(32, 8, 64), (8, 4, 256), (40, 8, 100)])
def test_prompt_unseen_values_do_not_matter_with_many_rows(dev, nh, nkv, hd, dtype):
    n = 300
    qq, k, v = (rnd(s, (2 * n, h, hd), dtype).cuda() for s, h in ((1, nh), (2, nkv), (3, nkv)))
    clean = q.attn_prompt(qq, k, v, cu_of([n, n]))
    for j, what in ((0, "v"), (150, "v"), (150, "k"), (299, "v")):
        k2, v2 = k.clone(), v.clone()
        (v2 if what == "v" else k2)[j] = float("nan")
        y = q.attn_prompt(qq, k2, v2, cu_of([n, n]))
        assert torch.equal(y[:j], clean[:j]) and torch.equal(y[n:], clean[n:]), (j, what)
        assert y[j:n].isnan().all(), (j, what)


def test_prompt_repeats_bit_for_bit_on_any_stream(dev):
    n, nh, nkv, hd = 700, 8, 2, 128
    for dtype in (F32, BF16):
        qq, k, v = (rnd(s, (n, h, hd), dtype).cuda() for s, h in ((1, nh), (2, nkv), (3, nkv)))
        cu = cu_of([300, 400])
        a = q.attn_prompt(qq, k, v, cu)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        b = q.attn_prompt(qq, k, v, cu, stream=s)
        s.synchronize()
        assert torch.equal(a, b)


# ---------------------------------------------------------------- attn_paged

def run_paged(lens, nh, nkv, hd, S, dtype, y_dtype=F32, seed=1, pad=0, bad=(), poison=True, qs=2.0,
              interleave=False):
    """lens: (cache rows, new tokens); bad: (request, column) entries outside the cache."""
    rng = np.random.default_rng(seed)
    need = [max(0, -(-L // S)) for L, _ in lens]
    nb = sum(need) + 3
    ids = rng.permutation(nb).astype(np.int32)
    table = np.full((len(lens), max(need + [0]) + 1), 10 ** 6, dtype=np.int32)
    used = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[used:used + n]
        used += n
    T = sum(n for _, n in lens) + pad
    qq = rnd(seed, (T, nh, hd), dtype, qs).cuda()
    if interleave:
        both = rnd(seed + 1, (nb, 2, nkv, S, hd), dtype).cuda()
        k, v = both[:, 0], both[:, 1]
    else:
        k, v = (rnd(seed + i, (nb, nkv, S, hd), dtype).cuda() for i in (1, 2))
    if poison:  # rows that no request holds
        free = torch.ones((nb, S), dtype=torch.bool)
        for r, (L, _) in enumerate(lens):
            j = np.arange(max(L, 0))
            free[table[r][j // S], j % S] = False
        mask = free.cuda()[:, None, :, None].expand(nb, nkv, S, hd)
        k[mask] = float("nan")
        v[mask] = float("nan")
    for r, c in bad:
        table[r, c] = -1 if (r + c) % 2 else nb
    wide = torch.zeros((len(lens), table.shape[1] + 3), dtype=torch.int32, device="cuda")
    dt = wide[:, :table.shape[1]]
    dt.copy_(torch.from_numpy(table))
    y = torch.full((T, nh, hd), 7.0, dtype=y_dtype, device="cuda")
    q.attn_paged(qq, q.PagedKV(k, v), dt, cu_of([n for _, n in lens]), i32(L for L, _ in lens), y=y)
    assert q.qmm_device_status(clear=True) == (q.QMM_DEV_BAD_BLOCK if bad else 0)
    want, b = ref.paged(num(qq), num(k), num(v), table, [(max(L, 0), n) for L, n in lens],
                        hd ** -0.5, tensor_core(dtype))
    assert_within(num(y), want, round_bound(want, b, y_dtype), f"{nh}/{nkv} d{hd} S{S} {dtype}")


DECODE = [(1, 1), (15, 1), (16, 1), (17, 1), (1000, 1), (0, 1), (128, 1), (129, 1), (511, 1)]
MIXED = [(700, 150), (64, 64), (300, 1), (129, 2), (5, 5), (257, 130), (40, 0), (0, 0), (33, 17)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd", SHAPES)
def test_paged_decode(dev, nh, nkv, hd, dtype):
    run_paged(DECODE, nh, nkv, hd, 16, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd", SHAPES)
def test_paged_chunks(dev, nh, nkv, hd, dtype):
    run_paged(MIXED, nh, nkv, hd, 32, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("S", [16, 32, 64, 128, 256])
def test_paged_block_sizes(dev, S, dtype):
    run_paged(MIXED + DECODE, 8, 2, 64, S, dtype, pad=4, interleave=S == 64)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd", [(2, 1, 4), (3, 3, 20), (4, 2, 132), (2, 1, 256), (2, 2, 260),
                                       (4, 1, 512), (70, 1, 64), (160, 1, 16)])
def test_paged_other_heads(dev, nh, nkv, hd, dtype):
    run_paged([(100, 20), (77, 1), (30, 1)], nh, nkv, hd, 16, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd", [(12, 1, 128), (32, 2, 64), (20, 1, 84), (32, 1, 36), (16, 2, 256),
                                       (13, 1, 200), (8, 1, 512), (5, 1, 260)])
def test_paged_rows_of_several_units(dev, nh, nkv, hd, dtype):
    """More query rows to a key/value head than one unit of the kernel for few
    rows takes: whole and ragged shares of a group, single tokens and several,
    rows that see no key, blocks outside the cache."""
    run_paged([(700, 1), (33, 1), (1, 1), (0, 1), (258, 1), (0, 0)], nh, nkv, hd, 16, dtype,
              bad=[(0, 2), (4, 16)])
    few = max(1, 32 // (nh // nkv) * 4 // 5) if hd <= 128 else 1
    run_paged([(700, few + 1), (few - 1, few), (64, few)], nh, nkv, hd, 32, dtype, pad=2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd", [(16, 4, 256), (8, 2, 512), (8, 8, 132)])
def test_paged_chunks_of_wide_heads(dev, nh, nkv, hd, dtype):
    run_paged(MIXED, nh, nkv, hd, 32, dtype, bad=[(0, 3), (2, 9)])
    run_paged([(300, 12), (12, 12), (5, 12)], nh, nh, hd, 16, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [3, 5, 7, 8])
def test_paged_few_tokens_each(dev, n, dtype):
    run_paged([(900, n), (n, n), (40, n), (2, n)], 8, 2, 128, 16, dtype, bad=[(0, 50)])
    run_paged([(900, n), (n, n), (40, n), (2, n)], 16, 2, 60, 64, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_paged_rows_that_see_no_key(dev, dtype):
    """Fewer cache rows than new tokens: the first of them see nothing."""
    run_paged([(3, 10), (0, 4), (130, 140), (1, 300), (-5, 2)], 4, 2, 64, 16, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_paged_bad_blocks(dev, dtype):
    run_paged([(200, 1), (300, 40), (16, 1), (100, 1)], 4, 2, 64, 16, dtype,
              bad=[(0, 0), (0, 5), (1, 3), (1, 18), (2, 0), (3, 6)])
    run_paged([(300, 300), (700, 1)], 4, 1, 128, 64, dtype, bad=[(0, 0), (1, 10)])


@pytest.mark.parametrize("dtype,y_dtype", [(F32, BF16), (BF16, BF16)])
def test_paged_output_types(dev, dtype, y_dtype):
    run_paged(MIXED, 8, 2, 128, 16, dtype, y_dtype, pad=2)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_paged_long_contexts(dev, dtype):
    """One long context split over every worker, alone and beside short ones."""
    run_paged([(20000, 1)], 4, 1, 64, 64, dtype)
    run_paged([(6001, 3), (1, 1), (9000, 1), (50, 50)], 4, 2, 128, 128, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_paged_many_requests(dev, dtype):
    rng = np.random.default_rng(5)
    run_paged([(int(L), 1) for L in rng.integers(1, 200, 400)], 4, 2, 64, 16, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_paged_sharp_scores(dev, dtype):
    run_paged([(900, 1), (400, 100)], 4, 2, 64, 16, dtype, qs=100.0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_paged_captured_step_replays_with_other_lengths(dev, dtype):
    nh, nkv, hd, S, nb = 4, 2, 64, 16, 200
    qq = rnd(1, (3, nh, hd), dtype).cuda()
    k, v = (rnd(2 + i, (nb, nkv, S, hd), dtype).cuda() for i in range(2))
    cache, cu = q.PagedKV(k, v), cu_of([1, 1, 1])
    table = torch.from_numpy(np.random.default_rng(7).permutation(nb)[:189].astype(np.int32)
                             .reshape(3, 63)).cuda()
    kvl = i32([5, 900, 33])
    y = torch.empty((3, nh, hd), device="cuda")
    ws = torch.empty((q.qmm_attn_paged_workspace_bytes(qq, cache, 3),), dtype=torch.uint8,
                     device="cuda")
    call = lambda out: q.attn_paged(qq, cache, table, cu, kvl, y=out, workspace=ws)
    call(y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(y)
    for lens in ([5, 900, 33], [1000, 1, 17], [0, 500, 1008]):
        kvl.copy_(i32(lens))
        g.replay()
        torch.cuda.synchronize()
        eager = torch.empty_like(y)
        call(eager)
        assert torch.equal(y, eager)
        want, b = ref.paged(num(qq), num(k), num(v), table.cpu().numpy(), [(L, 1) for L in lens],
                            hd ** -0.5, tensor_core(dtype))
        assert_within(num(y), want, round_bound(want, b, F32))


def test_prompt_and_paged_agree(dev):
    """A prompt in one call, in chunks over the cache, and token by token."""
    n, nh, nkv, hd, S = 150, 4, 2, 64, 16
    for dtype in (F32, BF16):
        qq, k, v = (rnd(s, (n, h, hd), dtype).cuda() for s, h in ((1, nh), (2, nkv), (3, nkv)))
        nb = -(-n // S)
        table = torch.arange(nb, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
        cache = q.PagedKV(*(torch.zeros((nb, nkv, S, hd), dtype=dtype, device="cuda")
                            for _ in range(2)))
        for t in (k, v):
            c = cache.k if t is k else cache.v
            for j in range(n):
                c[int(table[0, j // S]), :, j % S] = t[j]
        whole, b = ref.prompt(num(qq), num(k), num(v), [n], hd ** -0.5, tensor_core(dtype))
        for cuts in ([n], [70, 80], [1] * n):
            done, out = 0, []
            for m in cuts:
                done += m
                out.append(q.attn_paged(qq[done - m:done], cache, table, cu_of([m]), i32([done])))
            assert_within(num(torch.cat(out)), whole, b + ref.U * np.abs(whole))


# -------------------------------------------------- the layer and the example

def test_layer_step_within_the_decode_oracles_bound(dev):
    """One decode step of a layer over a paged fp32 cache, beside another
    request, against the oracle of the single-sequence decode step: the same
    weights, token, position and earlier cache rows."""
    import oracle
    import synth

    D, nh, nkv, hd, S, pos, max_seq = 256, 8, 2, 32, 16, 70, 128
    r = synth.normal
    ow = [oracle.quantize(r(5, i, n * kk, 0.05).reshape(n, kk), 8, 64)
          for i, (n, kk) in enumerate(((nh * hd, D), (nkv * hd, D), (nkv * hd, D), (D, nh * hd)))]

    def weight(os_):
        cat = [np.concatenate([getattr(o, f).reshape(o.N, -1) for o in os_])
               for f in ("codes", "scales", "zps")]
        t = [torch.from_numpy(np.ascontiguousarray(c)).cuda() for c in (cat[0].view(np.int8), *cat[1:])]
        return q.QWeight(8, 64, sum(o.N for o in os_), os_[0].K, *t)

    wqkv, wo = weight(ow[:3]), weight(ow[3:])
    oc, os_ = oracle.rope_table(max_seq, hd, 10000.0)
    cos, sin = q.rope_table(max_seq, hd, device=dev)
    old = r(6, 1, 2 * nkv * max_seq * hd).reshape(2, nkv, max_seq, hd)
    cache = q.PagedKV(*(torch.zeros((12, nkv, S, hd), device="cuda") for _ in range(2)))
    used = [7, 0, 9, 4, 11]  # the request's earlier blocks
    for b, i in enumerate(used):
        for t, c in ((0, cache.k), (1, cache.v)):
            c[i] = torch.from_numpy(old[t][:, b * S:(b + 1) * S].copy()).cuda()
    table = torch.full((2, 6), -1, dtype=torch.int32, device="cuda")
    table[0, :5] = torch.tensor(used)
    xs = np.stack([r(7, 1, D), r(7, 2, D)])
    plan = q.kv_plan(i32([pos, 0]), i32([1, 1]), table, i32([3, 5]), S, 2)
    y = q.attn_layer_paged(torch.from_numpy(xs).cuda(), wqkv, wo, nh, cos, sin, cache, plan, table)
    assert plan.blocks_used.tolist() == [1] and table[1, 0] == 3
    for row, (p, c) in enumerate(((pos, old), (0, np.zeros_like(old)))):
        want, bound, kv, kvb = oracle.attn_decode(xs[row], p, nh, nkv, hd, *ow, oc, os_, c)
        assert_within(num(y[row]), want, bound, f"row {row}")
        slot = int(plan.slots[row])
        for t, got in ((0, cache.k), (1, cache.v)):
            assert_within(num(got[slot // S, :, slot % S]), kv[t], kvb[t], f"cache {row}")


@pytest.mark.parametrize("dtype", (F32, BF16))
def test_memory_of_a_call_on_another_stream_is_recorded_there(dev, monkeypatch, dtype):
    """Every tensor that a call allocates belongs to the current stream; a call
    on another one has to record them all there, or their memory could be
    handed out again while that stream still uses it."""
    D, nh, nkv, hd, S, T = 128, 4, 2, 32, 16, 12
    g = torch.Generator().manual_seed(3)

    def weight(N, K):
        return q.qmm_quantize_groupwise(torch.randn((N, K), generator=g).cuda(), 8, 64)

    wqkv, wo = weight((nh + 2 * nkv) * hd, D), weight(D, nh * hd)
    cos, sin = q.rope_table(64, hd, device=dev)
    cache = q.paged_kv(4, nkv, S, hd, dtype=dtype, device=dev)
    table = torch.full((2, 2), -1, dtype=torch.int32, device="cuda")
    x = torch.randn((T, D), generator=g).to(dtype).cuda()
    args = i32([0, 0]), i32([5, 7]), table, i32([0, 1, 2, 3]), S, T
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    made, seen, empty, record = [], set(), torch.empty, q._on_stream

    def spy_empty(*a, **kw):
        t = empty(*a, **kw)
        made.append(t)  # kept, so that no address comes twice
        return t

    def spy_record(stream, *ts):
        seen.update(t.data_ptr() for t in ts if t is not None and stream is not None)
        record(stream, *ts)

    monkeypatch.setattr(torch, "empty", spy_empty)
    monkeypatch.setattr(q, "_on_stream", spy_record)
    plan = q.kv_plan(*args, stream=s)
    for prompts in (True, False):
        q.attn_layer_paged(x, wqkv, wo, nh, cos, sin, cache, plan, table, prompts=prompts, stream=s)
    s.synchronize()
    missing = [(t.shape, t.dtype) for t in made if t.numel() and t.data_ptr() not in seen]
    assert len(made) >= 5 and not missing, missing


def test_layer_without_tokens(dev):
    nh, nkv, hd, S = 4, 2, 32, 16
    w = [q.qmm_quantize_groupwise(torch.ones((n, k), device="cuda"), 8, 64) for n, k in ((256, 128), (128, 128))]
    cos, sin = q.rope_table(16, hd, device=dev)
    cache = q.paged_kv(2, nkv, S, hd, dtype=F32, device=dev)
    table = torch.full((1, 1), -1, dtype=torch.int32, device="cuda")
    plan = q.kv_plan(i32([0]), i32([0]), table, i32([0, 1]), S, 0)
    x = torch.zeros((0, 128), device="cuda")
    for prompts in (True, False):
        y = q.attn_layer_paged(x, *w, nh, cos, sin, cache, plan, table, prompts=prompts)
        assert y.shape == (0, 128)
    assert plan.blocks_used.tolist() == [0]


def test_example_serves_requests(dev):
    """examples/serve_paged.py: prompts, decoding and a chunked prompt through
    the cache agree with each whole sequence at once.  Both round the same
    values to bf16 at the same places (queries, keys, values, weights, rows),
    so a row differs by a few of those roundings, each at most 2^-8 of what it
    rounds: 4 x 2^-8."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "serve_paged.py")
    spec = importlib.util.spec_from_file_location("serve_paged", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main(["--quiet", "--width", "1024", "--heads", "8", "--kv-heads", "2"]) <= 4 * 2.0 ** -8


# ------------------------------------------------------------- further edges

@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_requests_and_given_scale(dev, dtype):
    run_prompt([], 4, 2, 64, dtype, pad=2)
    run_paged([], 4, 2, 64, 16, dtype, pad=3)
    n, nh, nkv, hd = 140, 4, 2, 64
    qq, k, v = (rnd(s, (n, h, hd), dtype).cuda() for s, h in ((1, nh), (2, nkv), (3, nkv)))
    y = q.attn_prompt(qq, k, v, cu_of([n]), scale=0.3)
    want, b = ref.prompt(num(qq), num(k), num(v), [n], float(np.float32(0.3)), tensor_core(dtype))
    assert_within(num(y), want, round_bound(want, b, F32))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_cache_offsets_beyond_32_bits(dev, dtype):
    """A cache of more than 2^31 elements (and 2^32 bytes), the requests'
    blocks at its end: written by rope_append, read by attn_paged."""
    nh, nkv, hd, S, nb, n = 8, 8, 128, 16, 140000, 40
    assert nb * nkv * S * hd > 2 ** 31
    cache = q.paged_kv(nb, nkv, S, hd, dtype)
    x = rnd(1, (n, (nh + 2 * nkv) * hd), dtype).cuda()
    cos, sin = q.rope_table(n, hd, device=dev)
    table = torch.tensor([[nb - 1, nb - 3, 131072]], dtype=torch.int32, device="cuda")
    plan = q.kv_plan(i32([0]), i32([n]), torch.full((1, 3), -1, dtype=torch.int32, device="cuda"),
                     table[0].contiguous(), S, n)
    gq, gk, gv = q.rope_append(x, nh, plan.positions, plan.slots, cos, sin, cache, keep_kv=True)
    for j in (0, 15, 16, 39):
        b = int(table[0, j // S])
        assert torch.equal(cache.k[b, :, j % S], gk[j]) and torch.equal(cache.v[b, :, j % S], gv[j])
    y = q.attn_paged(gq, cache, table, plan.cu_new, plan.kv_lens)
    want, b = ref.prompt(num(gq), num(gk), num(gv), [n], hd ** -0.5, tensor_core(dtype))
    assert_within(num(y), want, round_bound(want, b, F32))
    last = q.attn_paged(gq[-1:], cache, table, cu_of([1]), plan.kv_lens)
    assert_within(num(last), want[-1:], round_bound(want, b, F32)[-1:])


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_captured_serving_step(dev, dtype):
    """kv_plan, rope_append and attn_paged in one graph, replayed step by step
    with the lengths updated in place, against the same steps run eagerly."""
    nh, nkv, hd, S, R = 4, 2, 64, 16, 3
    cos, sin = q.rope_table(256, hd, device=dev)
    free = torch.arange(40, dtype=torch.int32, device="cuda")

    def server():
        cache = q.PagedKV(*(torch.zeros((40, nkv, S, hd), dtype=dtype, device="cuda") for _ in range(2)))
        table = torch.full((R, 40), -1, dtype=torch.int32, device="cuda")
        return cache, table, i32([0, 0, 0]), i32([1, 1, 1]), free.clone(), \
            torch.empty((R, (nh + 2 * nkv) * hd), dtype=dtype, device="cuda")

    def step(s, plan=None, y=None, ws=None):
        cache, table, ctx, new, pool, x = s
        p = q.kv_plan(ctx, new, table, pool, S, R, out=plan)
        gq, _, _ = q.rope_append(x, nh, p.positions, p.slots, cos, sin, cache)
        return p, q.attn_paged(gq, cache, table, p.cu_new, p.kv_lens, y=y, workspace=ws)

    a, b = server(), server()
    plan, y = q.alloc_kv_plan(R, R), torch.empty((R, nh, hd), device="cuda")
    x0 = rnd(50, tuple(b[5].shape), dtype).cuda()
    b[5].copy_(x0)
    ws = torch.empty((q.qmm_attn_paged_workspace_bytes(
        torch.empty((R, nh, hd), dtype=dtype, device="cuda"), b[0], R),), dtype=torch.uint8, device="cuda")
    step(b, plan, y, ws)  # warm-up; the lengths stay as they are
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(b, plan, y, ws)
    for t in range(40):
        x = rnd(100 + t, tuple(x0.shape), dtype).cuda()
        for s in (a, b):
            s[5].copy_(x)
        p, want = step(a)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(a[1], b[1])
        assert torch.equal(a[0].k, b[0].k) and torch.equal(a[0].v, b[0].v)
        used = int(p.blocks_used)
        for s in (a, b):
            s[2].copy_(p.kv_lens)
            s[4].copy_(torch.roll(s[4], -used))
    assert a[2].tolist() == [40, 40, 40]
