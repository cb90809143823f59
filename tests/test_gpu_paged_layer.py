"""attn_layer_paged with fp32 and bf16 tokens over fp32 and bf16 caches: each
value is rounded where the layer says and nowhere else.

The layer is held to the 64-bit oracle's projections and to an attention in
64 bits, with a bound from its roundings (a half step of bf16 is 2^-8, of fp32
2^-24 = u):
  projections   the oracle's bound, 1e-5 sum |x w| + 1e-6
  q, k          that bound turned by the rotation, 4 u of the products, then a
                half step of the cache's type
  v             the projection's bound, then a half step of the cache's type
  score         ds = scale (|q| . dk + dq . |k| + dq . dk) and fp32 arithmetic,
                scale (hd + 8) u |q| . |k|, both with the errors added to |q|, |k|
  weight        p_j within [exp(-ds_j) / sum p exp(ds), exp(ds_j) / sum p exp(-ds)],
                and its own half step of bf16 on the tensor cores, 2^-20 of the
                exponential, 2 (L + 64) u of the sums
  result        sum p_j (E_j (|v_j| + dv_j) + dv_j), then a half step of the type
                of x
  output        |W| da + the oracle's bound
"""
import numpy as np
import pytest
import torch

import group_quantized_moe_gb300 as q
import oracle
import paged_reference as ref
import synth
from parity_checks import assert_within
from test_gpu_paged import BF16, F32, dev, i32, num  # noqa: F401 (dev: fixture)

pytestmark = pytest.mark.gpu

D, NH, NKV, HD, S, MAX_SEQ = 256, 8, 2, 32, 16, 256


def half_step(dtype):
    return ref.HALF_BF16 if dtype == BF16 else ref.U


def weights():
    """The oracle's quantised wqkv and wo, and the same on the device."""
    r = synth.normal
    row = (NH + 2 * NKV) * HD
    out = []
    for o in (oracle.quantize(r(11, 1, row * D, 0.05).reshape(row, D), 8, 64),
              oracle.quantize(r(11, 2, D * NH * HD, 0.05).reshape(D, NH * HD), 8, 64)):
        codes = np.ascontiguousarray(o.codes.reshape(o.N, -1).view(np.int8))
        out.append((o, q.QWeight(8, 64, o.N, o.K, *(torch.from_numpy(t).cuda()
                                                    for t in (codes, o.scales, o.zps)))))
    return out


def turn(x, dx, pos):
    """Rows x [n, heads, HD] with errors dx turned by their positions' angles."""
    c, s = (t[pos][:, None, :] for t in map(np.asarray, oracle.rope_table(MAX_SEQ, HD, 10000.0)))
    c, s = c.astype(np.float64), s.astype(np.float64)
    y, dy = np.empty_like(x), np.empty_like(x)
    a, b, da, db = x[..., 0::2], x[..., 1::2], dx[..., 0::2], dx[..., 1::2]
    y[..., 0::2], y[..., 1::2] = a * c - b * s, a * s + b * c
    # the device's table is within an fp32 ulp (2 u) of the oracle's
    slop = 4 * ref.U * (np.abs(a) + da + np.abs(b) + db)
    dy[..., 0::2] = np.abs(c) * da + np.abs(s) * db + slop
    dy[..., 1::2] = np.abs(s) * da + np.abs(c) * db + slop
    return y, dy


def attend(x, dx, k, dk, v, dv, tensor_core):
    """Causal attention of one request's rows and the bound described above."""
    n, scale = len(x), HD ** -0.5
    y, b = np.empty_like(x), np.empty_like(x)
    vis = np.tril(np.ones((n, n), dtype=bool))
    for h in range(NH):
        kv = h // (NH // NKV)
        qa, da, ka, dka = x[:, h], dx[:, h], k[:, kv], dk[:, kv]
        s = np.where(vis, scale * (qa @ ka.T), -np.inf)
        ds = scale * (np.abs(qa) @ dka.T + da @ np.abs(ka).T + da @ dka.T)
        ds += scale * (HD + 8) * ref.U * ((np.abs(qa) + da) @ (np.abs(ka) + dka).T)
        p = np.exp(s - s.max(axis=1, keepdims=True))
        p /= p.sum(axis=1, keepdims=True)
        E = np.exp(ds) / (p * np.exp(-ds)).sum(axis=1, keepdims=True) - 1
        E = (1 + E) * (1 + 2.0 ** -20 + 2 * (n + 64) * ref.U + (ref.HALF_BF16 if tensor_core else 0)) - 1
        y[:, h] = p @ v[:, kv]
        b[:, h] = (p * E) @ (np.abs(v[:, kv]) + dv[:, kv]) + p @ dv[:, kv]
    return y, b


@pytest.mark.parametrize("x_dtype,cache_dtype", [(F32, BF16), (BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("prompts", [True, False])
def test_layer_within_the_bound_of_its_roundings(dev, x_dtype, cache_dtype, prompts):
    """Two requests, 5 and 3 tokens (the projections' fp32 kernels, whose
    products are exact to fp32 for bf16 rows as well), then one token more each."""
    (oqkv, wqkv), (oo, wo) = weights()
    cos, sin = q.rope_table(MAX_SEQ, HD, device=dev)
    cache = q.paged_kv(6, NKV, S, HD, dtype=cache_dtype, device=dev)
    for t in (cache.k, cache.v):
        t.fill_(float("nan"))
    table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    free, ctx = i32([4, 1, 5, 0]), i32([0, 0])
    xs, got = [[], []], [[], []]
    for step, new in enumerate(([5, 3], [1, 1], [1, 1])):
        T = sum(new)
        x = torch.from_numpy(synth.normal(12, step, T * D)).view(T, D).to(x_dtype)
        p = q.kv_plan(ctx, i32(new), table, free, S, T)
        y = q.attn_layer_paged(x.cuda(), wqkv, wo, NH, cos, sin, cache, p, table,
                               prompts=prompts and step == 0)
        free, ctx = free[int(p.blocks_used):].contiguous(), p.kv_lens
        for r, (a, b) in enumerate(((0, new[0]), (new[0], T))):
            xs[r].append(num(x[a:b]))
            got[r].append(num(y[a:b]))
    for r in range(2):
        x = np.concatenate(xs[r])
        n = len(x)
        qkv = oracle.linear_fused(x, oqkv).reshape(n, -1, HD)
        d = oracle.linear_bound(x, oqkv).reshape(n, -1, HD)
        rot, drot = turn(qkv[:, :NH + NKV], d[:, :NH + NKV], np.arange(n))
        hc = half_step(cache_dtype)
        drot = drot + hc * (np.abs(rot) + drot)
        v, dv = qkv[:, NH + NKV:], d[:, NH + NKV:]
        dv = dv + hc * (np.abs(v) + dv)
        a, da = attend(rot[:, :NH], drot[:, :NH], rot[:, NH:], drot[:, NH:], v, dv, cache_dtype == BF16)
        da = da + half_step(x_dtype) * (np.abs(a) + da)
        a, da = a.reshape(n, -1), da.reshape(n, -1)
        w = oracle.dequantize(oo).astype(np.float64)
        want = a @ w.T
        bound = da @ np.abs(w).T + 1e-5 * ((np.abs(a) + da) @ np.abs(w).T) + 1e-6
        assert_within(np.concatenate(got[r]), want, bound, f"request {r}")


@pytest.mark.parametrize("x_dtype,cache_dtype", [(F32, BF16), (BF16, BF16), (BF16, F32), (F32, F32)])
def test_layer_rounds_once_before_the_cache_and_in_the_type_of_x(dev, x_dtype, cache_dtype):
    """The layer's steps one by one, with fp32 projections into rope_append."""
    (_, wqkv), (_, wo) = weights()
    cos, sin = q.rope_table(MAX_SEQ, HD, device=dev)
    lens, T = [20, 47], 67
    x = torch.from_numpy(synth.normal(13, 1, T * D)).view(T, D).to(x_dtype).cuda()

    def fresh():
        c = q.paged_kv(6, NKV, S, HD, dtype=cache_dtype, device=dev)
        table = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
        return c, table, q.kv_plan(i32([0, 0]), i32(lens), table, i32([4, 1, 5, 0, 2, 3]), S, T)

    for prompts in (True, False):
        cache, table, plan = fresh()
        y = q.attn_layer_paged(x, wqkv, wo, NH, cos, sin, cache, plan, table, prompts=prompts)
        c2, table, plan = fresh()
        qkv = q.qmm_linear_batched(x, wqkv, y_dtype=F32)
        qq, k, v = q.rope_append(qkv, NH, plan.positions, plan.slots, cos, sin, c2, keep_kv=True)
        if prompts:
            a = q.attn_prompt(qq, k, v, plan.cu_new, y_dtype=x_dtype)
        else:
            a = q.attn_paged(qq, c2, table, plan.cu_new, plan.kv_lens, y_dtype=x_dtype)
        assert torch.equal(y, q.qmm_linear_batched(a.flatten(1), wo))
        rows = plan.slots.cpu()
        for got, want in ((cache.k, c2.k), (cache.v, c2.v)):
            assert torch.equal(got[rows // S, :, rows % S], want[rows // S, :, rows % S])
