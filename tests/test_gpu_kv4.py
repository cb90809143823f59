"""The paged cache held in 4 bits on the GPU, against plain numpy
(tests/kv4_reference.py, which derives the bounds): stored bytes exactly,
attention within its bound, everything a call does not own left as it was."""
import numpy as np
import pytest
import torch

import group_quantized_moe_gb300 as q
import kv4_reference as ref
import paged_reference as pref
from parity_checks import assert_within
from test_gpu_paged import BF16, DECODE, F32, MIXED, cu_of, dev, i32, num, rnd, round_bound  # noqa: F401 (dev: fixture)

pytestmark = pytest.mark.gpu


def filled(nb, nkv, hd, group, S, seed):
    """A cache of quantised random rows, as bytes."""
    rng = np.random.default_rng(seed)
    gain, mean = np.exp(0.5 * rng.standard_normal((2, nkv, 1, hd))), 0.4 * rng.standard_normal((2, nkv, 1, hd))
    x = [(rng.standard_normal((nb, nkv, S, hd)) * gain[i] + mean[i]).astype(np.float32) for i in range(2)]
    (kc, kz, ks), (vc, vz, vs) = (ref.quantise(t, group) for t in x)
    return pack((kc, kz, ks), (vc, vz, vs), hd, group, S)


def pack(keys, vals, hd, group, S):
    nb, nkv = keys[0].shape[:2]
    nc, G, strip = ref.chunks(hd), -(-hd // group), ref.strip_bytes(hd, group)
    out = np.zeros((nb, nkv, S // 16, strip), dtype=np.uint8)
    pad = lambda c: np.pad(c, ((0, 0),) * 3 + ((0, 32 * nc - hd),)).reshape(nb, nkv, S // 16, 16, nc, 32)
    kc = pad(keys[0]).reshape(nb, nkv, S // 16, 16, nc, 4, 8).swapaxes(4, 5)
    vc = pad(vals[0]).reshape(nb, nkv, S // 16, 2, 4, 2, nc, 8, 4).transpose(0, 1, 2, 3, 7, 4, 6, 5, 8)
    at = 0
    for c in (kc, vc):
        b = (c[..., 0::2] | c[..., 1::2] << 4).reshape(nb, nkv, S // 16, 256 * nc)
        out[..., at:at + 256 * nc] = b
        at += 256 * nc
    for _, z, s in (keys, vals):
        w = z.astype(np.float16).view(np.uint16).astype(np.uint32) | np.where(
            np.isnan(s), np.uint32(0x7FC00000), s.astype(np.float32).view(np.uint32))
        out[..., at:at + 64 * G] = np.ascontiguousarray(w).view(np.uint8).reshape(nb, nkv, S // 16, 64 * G)
        at += 64 * G
    return out.reshape(nb, nkv, -1)


# -------------------------------------------------------------------- append

def run_append(nh, nkv, hd, group, S, xd, yd, keep, x=None, T=37, seed=1, interleave=False):
    rng = np.random.default_rng(seed)
    nb, max_seq = 9, 300
    cos, sin = q.rope_table(max_seq, hd, device="cuda")
    pos = rng.integers(0, max_seq, T).astype(np.int32)
    slot = rng.permutation(nb * S)[:T].astype(np.int64)
    pos[3 % T], slot[5 % T] = -1, -1  # a padding row with a slot, a row without one
    row = (nh + 2 * nkv) * hd
    x = rnd(seed, (T, row), xd, 3.0) if x is None else x
    wide = torch.zeros((T, row + 16), dtype=xd, device="cuda")
    wide[:, :row] = x.cuda()
    n = q.qmm_kv4_block_bytes(nkv, hd, group, S) // nkv
    base = torch.from_numpy(rng.integers(0, 256, (nb, 2, nkv, n), dtype=np.uint8)).cuda()
    data = base[:, 1] if interleave else base[:, 1].contiguous()
    want = data.cpu().numpy().copy()
    cache = q.PagedKV4(data, hd, group, S)
    gq, gk, gv = q.rope_append(wide[:, :row], nh, torch.from_numpy(pos).cuda(), torch.from_numpy(slot).cuda(), cos,
                               sin, cache, keep_kv=keep, y_dtype=yd)
    turned = ref.rope32(x.float().numpy().reshape(T, nh + 2 * nkv, hd), pos, cos.cpu().numpy(), sin.cpu().numpy(),
                        nh + nkv)
    turned[pos < 0] = 0
    for t in range(T):
        if pos[t] >= 0 and slot[t] >= 0:
            ref.put(want, hd, group, S, int(slot[t]), turned[t, nh:nh + nkv], turned[t, nh + nkv:])
    np.testing.assert_array_equal(data.cpu().numpy(), want)
    if interleave:
        assert base[:, 0].cpu().numpy().any()
    # the same queries, keys and values as over the other caches
    pq, pk, pv = q.rope_append(wide[:, :row], nh, torch.from_numpy(pos).cuda(), None, cos, sin, None, keep_kv=True,
                               n_kv=nkv, y_dtype=yd)
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert same(gq, pq)
    if keep:
        assert same(gk, pk) and same(gv, pv)
    else:
        assert gk is None and gv is None
    # and read back
    slots = torch.from_numpy(rng.permutation(np.concatenate([slot, [-1, -5]]))).cuda()
    parts = ref.unpack(want, hd, group, S)
    idx = slots.cpu().numpy()
    with np.errstate(all="ignore"):
        for y_dtype in (F32, BF16):
            for got, part in zip(q.kv4_read(cache, slots, y_dtype=y_dtype), parts):
                # in fp32: exact for rows that were stored; the row with a slot and no
                # position holds random bytes, whose difference is rounded
                v = ref.values([t.astype(np.float32) for t in part], group)[idx // S, :, idx % S]
                v[idx < 0] = 0
                np.testing.assert_array_equal(got.float().cpu().numpy(),
                                              torch.from_numpy(v).float().to(y_dtype).float().numpy())
    assert q.qmm_device_status(clear=True) == 0


@pytest.mark.parametrize("nh,nkv,hd,group,S,xd,yd,keep", [
    (4, 2, 128, 64, 16, F32, BF16, True), (6, 1, 128, 32, 64, BF16, BF16, False), (3, 3, 8, 32, 32, F32, F32, True),
    (5, 5, 40, 64, 16, BF16, F32, True), (8, 2, 256, 64, 16, F32, F32, False), (7, 7, 80, 32, 128, BF16, BF16, True),
    (2, 1, 80, 64, 256, F32, BF16, False), (4, 4, 96, 64, 16, BF16, F32, False), (3, 1, 160, 32, 32, F32, BF16, True),
    (2, 2, 200, 64, 16, BF16, BF16, False), (9, 3, 64, 64, 64, F32, F32, True), (16, 16, 32, 32, 16, BF16, BF16, True)])
def test_append_bytes(dev, nh, nkv, hd, group, S, xd, yd, keep):
    run_append(nh, nkv, hd, group, S, xd, yd, keep, interleave=hd == 80)


@pytest.mark.parametrize("T", [1, 2, 150])
def test_append_tokens(dev, T):
    run_append(4, 2, 64, 32, 64, F32, BF16, False, T=T, seed=T)


@pytest.mark.parametrize("group", [32, 64])
def test_append_unusual_groups(dev, group):
    """Zeros, constants, one sign, a narrow range far from zero, ties, tiny and
    huge values, NaN and infinities, in the values (which are not turned) and,
    at position 0 of a table whose angle is 0, in the keys."""
    nh, nkv, hd = 2, 2, 128
    rng = np.random.default_rng(5)
    rows = [np.zeros(hd), np.full(hd, 3.25), np.full(hd, -1e-20), 100 + rng.random(hd), -5 - rng.random(hd),
            1e4 + 1e-3 * rng.random(hd), np.arange(hd) % 16 - 7.5, (np.arange(hd) % 31) * 0.5,
            rng.standard_normal(hd) * 1e-38, rng.standard_normal(hd) * 1e-44, rng.standard_normal(hd) * 1e38,
            np.where(np.arange(hd) % 2, 3.4e38, -3.4e38), rng.standard_normal(hd) * 1e-30]
    for bad in (np.nan, np.inf, -np.inf):
        for at in (0, 63, 127):
            r = rng.standard_normal(hd)
            r[at] = bad
            rows.append(r)
    x = np.stack([np.concatenate([rng.standard_normal(2 * hd), r, r[::-1], r[::-1], r]) for r in rows])
    x = torch.from_numpy(x.astype(np.float32))
    T = len(x)
    cos, sin = torch.ones((4, hd // 2), device="cuda"), torch.zeros((4, hd // 2), device="cuda")
    cache = q.paged_kv4(2, nkv, 16, hd, group)
    cache.data.zero_()
    want = cache.data.cpu().numpy().copy()
    slots = torch.arange(T, device="cuda")
    q.rope_append(x.cuda(), nh, torch.zeros(T, dtype=torch.int32, device="cuda"), slots, cos, sin, cache)
    with np.errstate(all="ignore"):
        turned = ref.rope32(x.numpy().reshape(T, nh + 2 * nkv, hd), [0] * T, cos.cpu().numpy(), sin.cpu().numpy(), 4)
        for t in range(T):
            ref.put(want, hd, group, 16, t, turned[t, nh:nh + nkv], turned[t, nh + nkv:])
        np.testing.assert_array_equal(cache.data.cpu().numpy(), want)
        for got, part in zip(q.kv4_read(cache, slots), ref.unpack(want, hd, group, 16)):
            v = ref.values(part, group)[slots.cpu().numpy() // 16, :, slots.cpu().numpy() % 16].astype(np.float32)
            np.testing.assert_array_equal(got.cpu().numpy(), v)
    # a value is off by at most half a scale (a whole one at the clamped end), its own scale's rounding apart
    k, v = q.kv4_read(cache, slots)
    vs = ref.unpack(want, hd, group, 16)[1][2][slots.cpu().numpy() // 16, :, slots.cpu().numpy() % 16]
    vs = np.repeat(vs, group, -1)[..., :hd]
    real = turned[:, nh + nkv:]
    fine = np.isfinite(vs)
    err = np.abs(v.cpu().numpy().astype(np.float64) - real)
    assert (err[fine] <= vs[fine] * (0.5 + 2.0 ** -8) + 1e-30).all()
    assert fine.sum() > 0.5 * fine.size


def test_append_and_read_out_of_range(dev):
    nh, nkv, hd, S = 2, 1, 8, 16
    cos, sin = q.rope_table(10, hd, device=dev)
    cache = q.paged_kv4(2, nkv, S, hd, 32)
    cache.data.zero_()
    x = torch.ones((3, (nh + 2 * nkv) * hd), device=dev)
    gq, _, _ = q.rope_append(x, nh, i32([9, 10, 1]), torch.tensor([32, 0, 31], device=dev), cos, sin, cache)
    assert q.qmm_device_status(clear=True) == q.QMM_DEV_BAD_POSITION | q.QMM_DEV_BAD_BLOCK
    assert (gq[1] == 0).all() and (gq[0] != 0).any() and gq.dtype == BF16
    k, v = q.kv4_read(cache, torch.tensor([0, 31, 15, 16], device=dev))
    assert q.qmm_device_status(clear=True) == 0
    assert (v[1] - 1).abs().max() < 1e-3 and v.count_nonzero() == hd and not k[0].any()
    k, v = q.kv4_read(cache, torch.tensor([31, 32, 1 << 40, -1], device=dev), y_dtype=BF16)
    assert q.qmm_device_status(clear=True) == q.QMM_DEV_BAD_BLOCK
    assert v[0].all() and not v[1:].any() and not k[1:].any()


# -------------------------------------------------------------------- attend

def run_attend(lens, nh, nkv, hd, group, S, dtype, y_dtype=F32, seed=1, pad=0, bad=(), qs=2.0, nan_rows=(),
               interleave=False, strided=False):
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
    data = filled(nb, nkv, hd, group, S, seed)
    # rows that no request holds: NaN scales and zero points, any codes
    free = np.ones((nb, S), dtype=bool)
    for r, (L, _) in enumerate(lens):
        j = np.arange(max(L, 0))
        free[table[r][j // S], j % S] = False
    strip, nc, G = ref.strip_bytes(hd, group), ref.chunks(hd), -(-hd // group)
    for b, row in zip(*np.nonzero(free)):
        for part in range(2):
            at = row // 16 * strip + 512 * nc + 64 * G * part + 4 * G * (row % 16)
            data[b, :, at:at + 4 * G] = 0xFF
    for r, c in bad:
        table[r, c] = -1 if (r + c) % 2 else nb
    if strided:
        buf = rnd(seed, (T, nh * hd + 24), dtype, qs).cuda()
        qq = buf[:, :nh * hd].view(T, nh, hd)
    else:
        qq = rnd(seed, (T, nh, hd), dtype, qs).cuda()
    wide = torch.zeros((len(lens), table.shape[1] + 3), dtype=torch.int32, device="cuda")
    dt = wide[:, :table.shape[1]]
    dt.copy_(torch.from_numpy(table))
    t = torch.from_numpy(data).cuda()
    if interleave:
        t = torch.stack([t, torch.full_like(t, 0xFF)], 1)[:, 0]
    y = torch.full((T, nh, hd), 7.0, dtype=y_dtype, device="cuda")
    q.attn_paged(qq, q.PagedKV4(t, hd, group, S), dt, cu_of([n for _, n in lens]), i32(L for L, _ in lens), y=y)
    assert q.qmm_device_status(clear=True) == (q.QMM_DEV_BAD_BLOCK if bad else 0)
    with np.errstate(all="ignore"):
        want, b = ref.paged(num(qq), data, group, S, table, [(max(L, 0), n) for L, n in lens], hd ** -0.5,
                            dtype == F32)
    assert_within(num(y), want, round_bound(want, b, y_dtype), f"{nh}/{nkv} d{hd} g{group} S{S} {dtype}")


HEADS = [(4, 4, 64, 64), (8, 2, 128, 64), (6, 1, 128, 32), (7, 1, 32, 32), (16, 2, 64, 32), (2, 2, 80, 32),
         (12, 4, 96, 64), (3, 1, 8, 64), (4, 2, 160, 32), (4, 1, 256, 64), (8, 8, 200, 64), (2, 1, 256, 32),
         (10, 1, 96, 32), (32, 2, 40, 64)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd,group", HEADS)
def test_attend_decode(dev, nh, nkv, hd, group, dtype):
    run_attend(DECODE, nh, nkv, hd, group, 16, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd,group", HEADS)
def test_attend_chunks(dev, nh, nkv, hd, group, dtype):
    run_attend(MIXED, nh, nkv, hd, group, 32, dtype, strided=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("S", [16, 32, 64, 128, 256])
def test_attend_block_sizes(dev, S, dtype):
    run_attend(MIXED + DECODE, 8, 2, 64, 64, S, dtype, pad=4, interleave=S == 64)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,hd,group", [(12, 1, 128, 64), (70, 1, 64, 32), (160, 1, 16, 32), (20, 1, 88, 64),
                                             (13, 1, 200, 32), (32, 1, 128, 32)])
def test_attend_many_heads_to_one(dev, nh, nkv, hd, group, dtype):
    run_attend([(700, 1), (33, 1), (1, 1), (0, 1), (258, 1), (0, 0)], nh, nkv, hd, group, 16, dtype,
               bad=[(0, 2), (4, 16)])
    run_attend([(300, 5), (3, 4), (64, 3)], nh, nkv, hd, group, 32, dtype, pad=2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n", [2, 3, 5, 8, 17])
def test_attend_few_tokens_each(dev, n, dtype):
    run_attend([(900, n), (n, n), (40, n), (2, n)], 8, 2, 128, 64, 16, dtype, bad=[(0, 50)])


@pytest.mark.parametrize("nh,nkv,hd,group", [(8, 2, 128, 64), (28, 4, 80, 32), (32, 1, 64, 32), (4, 4, 32, 32)])
def test_attend_chunks_beside_single_tokens(dev, nh, nkv, hd, group):
    """Long chunks and short requests in one call: each goes to its own kernel."""
    run_attend([(1, 1), (700, 600), (33, 1), (900, 1), (300, 300), (0, 1), (64, 3), (12, 40), (0, 0), (512, 200)],
               nh, nkv, hd, group, 16, BF16, BF16, pad=3, bad=[(1, 9), (3, 20)])
    if hd == 128:  # several units to a worker, of two query tiles and of one, some divided
        run_attend([(700, 200)] * 24, nh, nkv, hd, group, 16, BF16, BF16)
    run_attend([(1500, 1200), (40, 1)], nh, nkv, hd, group, 64, BF16)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attend_rows_that_see_no_key(dev, dtype):
    run_attend([(3, 10), (0, 4), (130, 140), (1, 300), (-5, 2)], 4, 2, 64, 32, 16, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attend_bad_blocks(dev, dtype):
    run_attend([(200, 1), (300, 40), (16, 1), (100, 1)], 4, 2, 64, 64, 16, dtype,
               bad=[(0, 0), (0, 5), (1, 3), (1, 18), (2, 0), (3, 6)])
    run_attend([(300, 300), (700, 1)], 4, 1, 128, 64, 64, dtype, bad=[(0, 0), (1, 10)])


@pytest.mark.parametrize("dtype,y_dtype", [(F32, BF16), (BF16, BF16)])
def test_attend_output_types(dev, dtype, y_dtype):
    run_attend(MIXED, 8, 2, 128, 64, 16, dtype, y_dtype, pad=2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("qs", [0.0, 1e-3, 100.0])
def test_attend_flat_and_sharp_scores(dev, dtype, qs):
    run_attend([(5000, 1), (1200, 30), (400, 1)], 4, 2, 128, 64, 64, dtype, qs=qs)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attend_long(dev, dtype):
    run_attend([(20000, 1), (9000, 2), (1, 1)], 8, 1, 128, 64, 128, dtype)


def test_attend_nothing(dev):
    cache = q.paged_kv4(4, 2, 16, 64)
    none, table = i32([]), torch.zeros((0, 3), dtype=torch.int32, device="cuda")
    y = q.attn_paged(torch.ones((3, 4, 64), device="cuda"), cache, table, i32([0]), none)
    assert not y.any()
    assert q.attn_paged(torch.ones((0, 4, 64), device="cuda"), cache, table, i32([0]), none).shape == (0, 4, 64)
    empty = q.paged_kv4(0, 2, 16, 64)
    y = q.attn_paged(torch.ones((1, 4, 64), device="cuda"), empty, i32([0]).view(1, 1), i32([0, 1]), i32([1]))
    assert not y.any() and q.qmm_device_status(clear=True) == q.QMM_DEV_BAD_BLOCK
    k, v = q.kv4_read(cache, torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert k.shape == v.shape == (0, 2, 64)


def scaled_cache(scales, hd=64, S=16):
    """One request of len(scales) rows whose values have scale 2^scales."""
    rng = np.random.default_rng(7)
    L, nkv = len(scales), 1
    nb = -(-L // S)
    x = rng.standard_normal((nb, nkv, S, hd)).astype(np.float32)
    keys, vals = ref.quantise(x, 32), list(ref.quantise(x[:, :, ::-1].copy(), 32))
    e = np.zeros(nb * S)
    e[:L] = scales
    vals[2] = (vals[2].astype(np.float64) * 2.0 ** e.reshape(nb, 1, S, 1)).astype(np.float32)
    return pack(keys, tuple(vals), hd, 32, S), keys


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("scales", [[-90.0] * 400, [100.0] * 400, list(np.round(np.linspace(-60, 60, 400))),
                                    list(np.round(np.linspace(60, -60, 400))), [60.0 * (i % 37 == 0) for i in range(400)],
                                    [0.0] * 399 + [110.0], [110.0] + [0.0] * 399])
def test_attend_value_scales_far_apart(dev, dtype, scales):
    """Scales of values over hundreds of powers of two, growing, shrinking, and
    of a row whose weight is small."""
    data, _ = scaled_cache(scales)
    table = np.arange(data.shape[0], dtype=np.int32)[None]
    for qs in (1.0, 20.0):
        qq = rnd(3, (1, 2, 64), dtype, qs).cuda()
        y = q.attn_paged(qq, q.PagedKV4(torch.from_numpy(data).cuda(), 64, 32, 16), torch.from_numpy(table).cuda(),
                         i32([0, 1]), i32([400]))
        want, b = ref.paged(num(qq), data, 32, 16, table, [(400, 1)], 64 ** -0.5, dtype == F32)
        assert_within(num(y), want, round_bound(want, b, F32), f"{dtype} {qs}")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nh,nkv,n", [(4, 2, 1), (4, 2, 6), (32, 2, 40), (8, 8, 200)])
def test_attend_unseen_nans_do_not_matter(dev, dtype, nh, nkv, n):
    """A row of the cache with a NaN reaches the queries that see it, and only
    them; a NaN group of a value only its own dimensions."""
    hd, S, L = 64, 16, 260
    data = filled(17, nkv, hd, 32, S, 3)
    table = torch.arange(17, dtype=torch.int32, device="cuda")[None]
    qq = rnd(2, (n, nh, hd), dtype).cuda()
    call = lambda d: q.attn_paged(qq, q.PagedKV4(torch.from_numpy(d).cuda(), hd, 32, S), table, i32([0, n]), i32([L]))
    clean = call(data)
    nan = np.frombuffer(np.uint32(0x7FC00000).tobytes(), np.uint8)
    # The power of two that holds a row's weights in 16 bits goes by the largest
    # weight times scale of all groups, so without a group's it may be another one:
    # parts below fp16's normal range are then rounded elsewhere, each by at most
    # 2^-29 of the largest, times a code of at most 15; and the sums of fp32 (2 u a
    # term) round those other parts.
    codes, zp, sc = ref.unpack(data, hd, 32, S)[1]
    near = L * 2.0 ** -29 * 15 * sc.max() + 2 * (L + 64) * 2 * ref.U * ((15 + np.abs(zp)) * sc).max()
    for j in (0, 100, L - n, L - 1):
        first = max(0, j - (L - n))  # the first query that sees row j
        for part in range(2):
            d = data.copy()
            at = j % 16 * 8 + 512 * 2 + 128 * part
            d[j // 16, :, at:at + 4] = nan  # group 0
            y = call(d)
            assert torch.equal(y[:first], clean[:first]), (j, part)
            if part:
                assert y[first:, :, :32].isnan().all()
                assert (y[first:, :, 32:] - clean[first:, :, 32:]).abs().max() <= near
            else:
                assert y[first:].isnan().all()


def test_attend_nonfinite_queries(dev):
    data = torch.from_numpy(filled(4, 1, 64, 64, 16, 3)).cuda()
    for dtype in (F32, BF16):
        qq = rnd(2, (2, 4, 64), dtype).cuda()
        qq[0, 1, 5], qq[1, 2, 7] = float("nan"), float("inf")
        y = q.attn_paged(qq, q.PagedKV4(data, 64, 64, 16), i32([0, 1, 2, 3]).view(1, 4), i32([0, 2]), i32([60]))
        assert y[0, 1].isnan().all() and y[1, 2].isnan().all()
        assert y[0, [0, 2, 3]].isfinite().all() and y[1, [0, 1, 3]].isfinite().all()


def test_attend_offsets_beyond_32_bits(dev):
    """Blocks whose first byte lies beyond 2^32."""
    nkv, hd, S, L = 2, 64, 256, 700
    n = q.qmm_kv4_block_bytes(nkv, hd, 64, S) // nkv
    nb = (5 << 30) // (nkv * n)
    big = torch.empty((nb, nkv, n), dtype=torch.uint8, device="cuda")
    small = filled(3, nkv, hd, 64, S, 5)
    ids = [nb - 1, nb - 7, 2]
    for i, b in enumerate(ids):
        big[b] = torch.from_numpy(small[i]).cuda()
    qq = rnd(1, (1, 4, hd), BF16).cuda()
    y = q.attn_paged(qq, q.PagedKV4(big, hd, 64, S), i32(ids).view(1, 3), i32([0, 1]), i32([L]))
    want, b = ref.paged(num(qq), small, 64, S, np.arange(3)[None], [(L, 1)], hd ** -0.5, False)
    assert_within(num(y), want, round_bound(want, b, F32))
    cos, sin = q.rope_table(10, hd, device="cuda")
    x = rnd(2, (2, 6 * hd), F32).cuda()
    slots = torch.tensor([nb * S - 1, (nb - 9) * S], device="cuda")
    cache = q.PagedKV4(big, hd, 64, S)
    q.rope_append(x, 2, i32([0, 1]), slots, cos, sin, cache)
    _, v = q.kv4_read(cache, slots)
    assert (v - x[:, 4 * hd:].view(2, nkv, hd)).abs().max() < 0.3


def test_attend_repeats_bit_for_bit_on_any_stream(dev):
    data = torch.from_numpy(filled(40, 2, 128, 64, 32, 3)).cuda()
    cache, table = q.PagedKV4(data, 128, 64, 32), torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    for dtype, n in ((F32, 1), (BF16, 1), (BF16, 70)):
        qq = rnd(1, (2 * n, 8, 128), dtype).cuda()
        args = (qq, cache, table, i32([0, n, 2 * n]), i32([600, 333]))
        a = q.attn_paged(*args)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        b = q.attn_paged(*args, stream=s)
        s.synchronize()
        assert torch.equal(a, b)


# ----------------------------------------------------------- used together

@pytest.mark.parametrize("dtype,group,hd", [(BF16, 64, 128), (F32, 32, 80)])
def test_a_serving_run(dev, dtype, group, hd):
    """Prompts, decoding and a prompt in chunks through kv_plan, rope_append and
    attn_paged: the cache's bytes and every step's rows."""
    nh, nkv, S, R, nb, max_seq = 6, 2, 16, 3, 40, 300
    cos, sin = q.rope_table(max_seq, hd, device="cuda")
    cache = q.paged_kv4(nb, nkv, S, hd, group)
    cache.data.zero_()
    want = cache.data.cpu().numpy().copy()
    free = torch.arange(nb, dtype=torch.int32, device="cuda")
    table = torch.full((R, 20), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(R, dtype=torch.int32, device="cuda")
    steps = [[20, 0, 5], [1, 33, 1], [1, 1, 1], [0, 40, 1], [1, 1, 0], [17, 2, 3]]
    for i, new in enumerate(steps):
        T = sum(new) + (i % 2)  # every second step padded
        p = q.kv_plan(lens, i32(new), table, free, S, T)
        x = rnd(100 + i, (T, (nh + 2 * nkv) * hd), dtype).cuda()
        qq, _, _ = q.rope_append(x, nh, p.positions, p.slots, cos, sin, cache, y_dtype=dtype)
        y = q.attn_paged(qq, cache, table, p.cu_new, p.kv_lens, y_dtype=dtype)
        pos, slots = p.positions.tolist(), p.slots.tolist()
        turned = ref.rope32(x.float().cpu().numpy().reshape(T, -1, hd), pos, cos.cpu().numpy(), sin.cpu().numpy(),
                            nh + nkv)
        for t in range(T):
            if pos[t] >= 0:
                ref.put(want, hd, group, S, slots[t], turned[t, nh:nh + nkv], turned[t, nh + nkv:])
        np.testing.assert_array_equal(cache.data.cpu().numpy(), want)
        wy, b = ref.paged(num(qq), want, group, S, table.cpu().numpy(), list(zip(p.kv_lens.tolist(), new)),
                          hd ** -0.5, dtype == F32)
        assert_within(num(y), wy, round_bound(wy, b, dtype), f"step {i}")
        free, lens = free[int(p.blocks_used):], p.kv_lens
    assert q.qmm_device_status(clear=True) == 0


def test_a_captured_step(dev):
    """A captured decode step (plan, append, attention), replayed with other
    lengths, tables and inputs in the same buffers; two graphs, each with its
    own workspace, replayed in turn."""
    nh, nkv, hd, S, R, nb = 8, 2, 128, 16, 4, 64  # and blocks to hand out behind them
    cos, sin = q.rope_table(400, hd, device="cuda")
    start = filled(2 * nb, nkv, hd, 64, S, 9)
    row = (nh + 2 * nkv) * hd

    def make(n_new):
        cache = q.PagedKV4(torch.from_numpy(start).cuda(), hd, 64, S)
        table = torch.arange(nb, dtype=torch.int32, device="cuda").view(R, nb // R).contiguous()
        ctx, new = i32([5] * R), i32([n_new] * R)
        x = torch.zeros((n_new * R, row), dtype=BF16, device="cuda")
        plan = q.alloc_kv_plan(R, n_new * R)
        ws = torch.empty(q.qmm_attn_paged_workspace_bytes(x[:, :nh * hd].view(-1, nh, hd), cache, R),
                         dtype=torch.uint8, device="cuda")
        out, qb = torch.empty((n_new * R, nh, hd), device="cuda"), torch.empty((n_new * R, nh, hd), dtype=BF16, device="cuda")

        def step():
            q.kv_plan(ctx, new, table, free0, S, n_new * R, out=plan)
            q.rope_append(x, nh, plan.positions, plan.slots, cos, sin, cache, q=qb)
            q.attn_paged(qb, cache, table, plan.cu_new, plan.kv_lens, y=out, workspace=ws)

        return cache, ctx, x, out, step

    free0 = torch.arange(nb, 2 * nb, dtype=torch.int32, device="cuda")
    sides = [make(1), make(3)]
    graphs = []
    for side in sides:
        side[4]()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            side[4]()
        graphs.append(g)
    for i, lens in enumerate(([5, 200, 17, 32], [100, 0, 251, 64], [16, 15, 1, 249])):
        for (cache, ctx, x, out, step), g in zip(sides, graphs):
            ctx.copy_(i32(lens))
            x.copy_(rnd(i, tuple(x.shape), BF16))
            cache.data.copy_(torch.from_numpy(start))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [(s[0].data.clone(), s[3].clone()) for s in sides]
        for (cache, ctx, x, out, step), (data, y) in zip(sides, got):
            cache.data.copy_(torch.from_numpy(start))
            out.fill_(9)
            step()
            assert torch.equal(cache.data, data) and torch.equal(out, y), lens
    assert q.qmm_device_status(clear=True) == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("prompts", [False, True])
def test_layer(dev, dtype, prompts):
    """attn_layer_paged over a 4-bit cache is its parts, in the type of x."""
    D, nh, nkv, hd, S = 256, 8, 2, 32, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn((nh + 2 * nkv) * hd, D, device="cuda", generator=g) / 16
    wqkv = q.qmm_quantize_groupwise(w, 8, 64)
    wo = q.qmm_quantize_groupwise(torch.randn(D, nh * hd, device="cuda", generator=g) / 16, 8, 64)
    cos, sin = q.rope_table(200, hd)
    x = torch.randn(40, D, device="cuda", generator=g).to(dtype)
    made = []
    for _ in range(2):
        cache = q.paged_kv4(20, nkv, S, hd, 32)
        cache.data.zero_()
        table = torch.full((2, 8), -1, dtype=torch.int32, device="cuda")
        p = q.kv_plan(i32([0, 0]), i32([30, 10]), table, torch.arange(20, dtype=torch.int32, device="cuda"), S, 40)
        made.append((cache, table, p))
    (c0, t0, p0), (c1, t1, p1) = made
    y = q.attn_layer_paged(x, wqkv, wo, nh, cos, sin, c0, p0, t0, prompts=prompts)
    qkv = q.qmm_linear_batched(x, wqkv)
    qq, k, v = q.rope_append(qkv, nh, p1.positions, p1.slots, cos, sin, c1, keep_kv=True, y_dtype=dtype)
    assert qq.dtype == dtype
    a = (q.attn_prompt(qq, k, v, p1.cu_new, y_dtype=dtype) if prompts
         else q.attn_paged(qq, c1, t1, p1.cu_new, p1.kv_lens, y_dtype=dtype))
    assert torch.equal(c0.data, c1.data)
    assert torch.equal(y, q.qmm_linear_batched(a.flatten(1), wo))
    # and near the layer over an fp32 cache: four bits of keys and values
    c2 = q.paged_kv(20, nkv, S, hd, F32)
    z = q.attn_layer_paged(x.float(), wqkv, wo, nh, cos, sin, c2, p0, t0, prompts=prompts)
    assert (y.float() - z).norm() < 0.2 * z.norm()


def test_example_serves_from_a_4_bit_cache(dev):
    """examples/serve_paged.py --four-bit runs, and its rows are those of the whole
    sequences but for four bits of keys and values: a step is a fifteenth of a
    group's range, some five deviations, so a value is off by a tenth of one."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_paged.py")
    spec = importlib.util.spec_from_file_location("serve_paged", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    worst = m.main(["--quiet", "--four-bit", "--width", "1024", "--heads", "8", "--kv-heads", "2"])
    assert 1e-3 < worst < 0.5


def test_two_streams_at_once(dev):
    """Two calls on two streams, each with its own workspace, give what they give alone."""
    data = torch.from_numpy(filled(60, 2, 128, 64, 32, 3)).cuda()
    cache, table = q.PagedKV4(data, 128, 64, 32), torch.arange(60, dtype=torch.int32, device="cuda").view(3, 20)
    sides = []
    for n, dtype in ((1, BF16), (90, BF16), (2, F32)):
        qq = rnd(n, (3 * n, 8, 128), dtype).cuda()
        args = (qq, cache, table, i32([0, n, 2 * n, 3 * n]), i32([600, 333, 640]))
        ws = torch.empty(q.qmm_attn_paged_workspace_bytes(qq, cache, 3), dtype=torch.uint8, device="cuda")
        sides.append((args, ws, q.attn_paged(*args, workspace=ws).clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        out = [q.attn_paged(*a, workspace=ws, stream=s) for a, ws, _, s in sides]
        torch.cuda.synchronize()
        for y, (_, _, want, _) in zip(out, sides):
            assert torch.equal(y, want)


@pytest.mark.parametrize("dtype,n", [(BF16, 1), (F32, 1), (BF16, 64)])
def test_repeated_calls_agree(dev, dtype, n):
    """Many units to a worker, whole and divided, the same bits every time."""
    rng = np.random.default_rng(2)
    lens = [int(v) for v in rng.integers(1, 1500, 64)]
    need = [-(-v // 16) for v in lens]
    data = torch.from_numpy(filled(sum(need), 2, 64, 32, 16, 3)).cuda()
    table, used = np.full((64, max(need)), -1, dtype=np.int32), 0
    for r, k in enumerate(need):
        table[r, :k] = np.arange(used, used + k)
        used += k
    qq = rnd(1, (64 * n, 8, 64), dtype, 2.0).cuda()
    args = (qq, q.PagedKV4(data, 64, 32, 16), torch.from_numpy(table).cuda(), cu_of([n] * 64), i32(lens))
    first = q.attn_paged(*args)
    for _ in range(30):
        assert torch.equal(q.attn_paged(*args), first)
    assert q.qmm_device_status(clear=True) == 0


@pytest.mark.parametrize("lens", [
    [(300, 8)] * 3, [(300, 9)] * 3,                                    # 32 rows a request, 36
    [(200, 1)] * 4 + [(500, 140)], [(200, 1)] * 5 + [(500, 140)],      # five requests, six
    [(90, 1)] * 30 + [(400, 128)], [(90, 1)] * 30 + [(400, 129)],      # 508 rows beyond a token each, 512
    [(90, 1)] * 40 + [(400, 256)], [(90, 1)] * 40 + [(400, 257)],      # ... 1020, 1024, at most 32 on average
    [(60, 8), (60, 9)] * 16 + [(700, 300)], [(40, 40)] * 8,
])
def test_attend_around_the_rules_that_choose(dev, lens):
    run_attend(lens, 8, 2, 128, 64, 32, BF16, pad=1)


def test_a_captured_call_whose_requests_change_kernels(dev):
    """One captured call of 400 tokens in eight requests, replayed with the tokens
    spread anew, and two such graphs that share a workspace of any contents."""
    nh, nkv, hd, S, R, T = 8, 2, 128, 32, 8, 400
    data = filled(R * 20, nkv, hd, 64, S, 11)
    cache = q.PagedKV4(torch.from_numpy(data).cuda(), hd, 64, S)
    table = torch.arange(R * 20, dtype=torch.int32, device="cuda").view(R, 20)
    ws = torch.full((q.qmm_attn_paged_workspace_bytes(torch.empty((T, nh, hd), dtype=BF16, device="cuda"), cache, R),),
                    0xFF, dtype=torch.uint8, device="cuda")
    sides = []
    for seed in (1, 2):
        qq = rnd(seed, (T, nh, hd), BF16, 2.0).cuda()
        cu, kv, y = cu_of([50] * R), i32([100] * R), torch.empty((T, nh, hd), device="cuda")
        call = lambda qq=qq, cu=cu, kv=kv, y=y: q.attn_paged(qq, cache, table, cu, kv, y=y, workspace=ws)
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        sides.append((qq, cu, kv, y, g))
    spreads = [[1, 1, 1, 393, 1, 1, 1, 1], [50] * R, [0, 0, 400, 0, 0, 0, 0, 0], [1, 8, 9, 300, 1, 1, 70, 0], [1] * R]
    for i, new in enumerate(spreads):
        have = [[0, 600, 17, 640, 333, 1, 128, 64], [640] * R][i % 2]
        lens = [(min(640, max(h, n)), n) for h, n in zip(have, new)]
        for qq, cu, kv, y, g in sides:
            cu.copy_(cu_of(new))
            kv.copy_(i32(L for L, _ in lens))
            y.fill_(9)
        ws.fill_(0xFF)
        for side in sides:
            side[4].replay()
        torch.cuda.synchronize()
        for qq, cu, kv, y, g in sides:
            want, b = ref.paged(num(qq), data, 64, S, table.cpu().numpy(), lens, hd ** -0.5, False)
            assert_within(num(y), want, round_bound(want, b, F32), str(new))
    assert q.qmm_device_status(clear=True) == 0


@pytest.mark.parametrize("order", ["up", "down", "from 1", "swapped", "twice"])
@pytest.mark.parametrize("hd,group,n_kv", [(128, 64, 2), (96, 32, 1), (200, 64, 3)])
def test_rows_in_any_order(dev, order, hd, group, n_kv):
    """Neighbours in the cache share words of values: pairs of rows the right way
    round, the other way round, and rows that only look like pairs."""
    S, n = 16, 64
    at = np.arange(n)
    slots = {"up": at, "down": at[::-1], "from 1": (at + 1) % n, "swapped": at ^ 1, "twice": at // 2}[order]
    data = filled(n // S, n_kv, hd, group, S, 13)
    cache = q.PagedKV4(torch.from_numpy(data).cuda(), hd, group, S)
    where = torch.from_numpy(np.ascontiguousarray(slots)).cuda()
    for got, part in zip(q.kv4_read(cache, where), ref.unpack(data, hd, group, S)):
        want = ref.values([t.astype(np.float32) for t in part], group)[slots // S, :, slots % S]
        np.testing.assert_array_equal(got.cpu().numpy(), want)
    if order == "twice":
        return  # (tokens do not share a slot)
    x = rnd(4, (n, 4 * n_kv * hd), F32)
    cos, sin = q.rope_table(8, hd, device="cuda")
    q.rope_append(x.cuda(), 2 * n_kv, i32([0] * n), where, cos, sin, cache)
    want = data.copy()
    rows = x.numpy().reshape(n, -1, hd)  # position 0 turns nothing
    for t in range(n):
        ref.put(want, hd, group, S, int(slots[t]), rows[t, 2 * n_kv:3 * n_kv], rows[t, 3 * n_kv:])
    np.testing.assert_array_equal(cache.data.cpu().numpy(), want)
