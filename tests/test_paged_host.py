"""Refusals of the paged-cache entry points, on the CPU: the C ABI's status
codes (with addresses that are never dereferenced, and only where no GPU is
visible) and the binding's checks of every tensor before any library call."""
import ctypes

import numpy as np
import pytest
import torch

import group_quantized_moe_gb300 as q
import paged_reference as ref
from group_quantized_moe_gb300 import build_lib

P = 0x7F0000000000
BIG = 1 << 62


@pytest.fixture(scope="module")
def L():
    if torch.cuda.is_available():
        pytest.skip("fake device pointers are only passed where no GPU is visible")
    build_lib.build()
    return q.lib()


def _call(fn, names, ok, **kw):
    a = list(ok)
    for k, v in kw.items():
        a[names.index(k)] = v
    return fn(*a)


def test_kv_plan_refuses(L):
    names = ["ctx", "new", "R", "S", "table", "stride", "cols", "free", "nfree", "T", "cu", "kvl",
             "pos", "slots", "used", "s"]
    ok = (P, P, 4, 16, P, 8, 8, P, 10, 20, P, P, P, P, P, None)
    call = lambda **kw: _call(L.qmm_kv_plan, names, ok, **kw)
    for bad in (dict(R=-1), dict(T=-1), dict(T=1 << 31), dict(cols=-1), dict(nfree=-1),
                dict(stride=7), dict(stride=(1 << 31) + 1)):
        assert call(**bad) == q.QMM_ERR_SHAPE, bad
    for S in (0, 8, 24, 512, -16):
        assert call(S=S) == q.QMM_ERR_UNSUPPORTED
    assert call(R=16385) == q.QMM_ERR_UNSUPPORTED
    for k in ("ctx", "new", "table", "free", "cu", "kvl", "pos", "slots", "used"):
        assert call(**{k: None}) == q.QMM_ERR_INVALID_ARG, k
        assert q.qmm_last_error()


def _cache(dtype=q.QMM_BF16, nkv=2, hd=64, S=16, nb=10, k=P, v=P, stride=None):
    return q._KvCache(dtype, nkv, hd, S, nb, k, v, nkv * S * hd if stride is None else stride)


BAD_CACHES = [(dict(dtype=3), q.QMM_ERR_INVALID_ARG), (dict(nkv=0), q.QMM_ERR_SHAPE),
              (dict(hd=6), q.QMM_ERR_UNSUPPORTED), (dict(hd=516), q.QMM_ERR_UNSUPPORTED),
              (dict(S=48), q.QMM_ERR_UNSUPPORTED), (dict(S=8), q.QMM_ERR_UNSUPPORTED),
              (dict(nb=-1), q.QMM_ERR_SHAPE), (dict(stride=100), q.QMM_ERR_SHAPE),
              (dict(stride=BIG), q.QMM_ERR_SHAPE), (dict(k=None), q.QMM_ERR_INVALID_ARG),
              (dict(v=P + 8), q.QMM_ERR_ALIGN), (dict(stride=2 * 16 * 64 + 4), q.QMM_ERR_ALIGN)]


def test_rope_append_refuses(L):
    names = ["x", "xd", "T", "stride", "nh", "nkv", "hd", "pos", "slots", "cos", "sin", "max", "cache",
             "q", "k", "v", "yd", "s"]
    ok = (P, q.QMM_F32, 3, 512, 4, 2, 64, P, P, P, P, 100, ctypes.byref(_cache()), P, P, P,
          q.QMM_BF16, None)
    call = lambda **kw: _call(L.qmm_rope_append, names, ok, **kw)
    assert call(T=0, x=None, q=None) == q.QMM_OK
    for kw, code in BAD_CACHES:
        assert call(cache=ctypes.byref(_cache(**kw))) == code, kw
    for kw, code in ((dict(nh=0), q.QMM_ERR_SHAPE), (dict(nh=5), q.QMM_ERR_SHAPE),
                     (dict(nh=2050), q.QMM_ERR_UNSUPPORTED), (dict(hd=62), q.QMM_ERR_UNSUPPORTED),
                     (dict(xd=2), q.QMM_ERR_INVALID_ARG), (dict(yd=q.QMM_F32), q.QMM_ERR_SHAPE),
                     (dict(nkv=4), q.QMM_ERR_SHAPE), (dict(hd=128), q.QMM_ERR_SHAPE),
                     (dict(T=-1), q.QMM_ERR_SHAPE), (dict(max=-1), q.QMM_ERR_SHAPE),
                     (dict(stride=511), q.QMM_ERR_SHAPE), (dict(stride=514), q.QMM_ERR_ALIGN),
                     (dict(x=P + 4), q.QMM_ERR_ALIGN), (dict(k=P + 8), q.QMM_ERR_ALIGN),
                     (dict(cos=P + 8), q.QMM_ERR_ALIGN),
                     (dict(x=None), q.QMM_ERR_INVALID_ARG), (dict(pos=None), q.QMM_ERR_INVALID_ARG),
                     (dict(slots=None), q.QMM_ERR_INVALID_ARG), (dict(sin=None), q.QMM_ERR_INVALID_ARG),
                     (dict(q=None), q.QMM_ERR_INVALID_ARG)):
        assert call(**kw) == code, kw


def test_attn_prompt_refuses(L):
    names = ["q", "k", "v", "dt", "T", "sq", "sk", "sv", "nh", "nkv", "hd", "cu", "B", "scale", "y",
             "yd", "ws", "wsb", "s"]
    need = L.qmm_attn_prompt_workspace_bytes(q.QMM_BF16, 5, 4, 2, 64, 1)
    assert need > 0
    ok = (P, P, P, q.QMM_BF16, 5, 256, 128, 128, 4, 2, 64, P, 1, 0.0, P, q.QMM_F32, P, need, None)
    call = lambda **kw: _call(L.qmm_attn_prompt, names, ok, **kw)
    assert call(T=0, q=None, y=None, ws=None) == q.QMM_OK
    for kw, code in ((dict(nh=3), q.QMM_ERR_SHAPE), (dict(nkv=0), q.QMM_ERR_SHAPE),
                     (dict(hd=2), q.QMM_ERR_UNSUPPORTED), (dict(hd=66), q.QMM_ERR_UNSUPPORTED),
                     (dict(dt=2), q.QMM_ERR_INVALID_ARG), (dict(yd=-1), q.QMM_ERR_INVALID_ARG),
                     (dict(T=-1), q.QMM_ERR_SHAPE), (dict(T=1 << 31), q.QMM_ERR_SHAPE),
                     (dict(B=-1), q.QMM_ERR_SHAPE), (dict(scale=-1.0), q.QMM_ERR_INVALID_ARG),
                     (dict(scale=float("nan")), q.QMM_ERR_INVALID_ARG),
                     (dict(scale=float("inf")), q.QMM_ERR_INVALID_ARG),
                     (dict(sq=255), q.QMM_ERR_SHAPE), (dict(sk=127), q.QMM_ERR_SHAPE),
                     (dict(sv=BIG), q.QMM_ERR_SHAPE), (dict(sq=258), q.QMM_ERR_ALIGN),
                     (dict(sk=130), q.QMM_ERR_ALIGN), (dict(q=P + 2), q.QMM_ERR_ALIGN),
                     (dict(y=P + 8), q.QMM_ERR_ALIGN), (dict(v=P + 8), q.QMM_ERR_ALIGN),
                     (dict(k=None), q.QMM_ERR_INVALID_ARG), (dict(cu=None), q.QMM_ERR_INVALID_ARG),
                     (dict(ws=None), q.QMM_ERR_WORKSPACE), (dict(wsb=need - 1), q.QMM_ERR_WORKSPACE),
                     (dict(ws=P + 16), q.QMM_ERR_ALIGN)):
        assert call(**kw) == code, kw
    assert call(dt=q.QMM_F32, sq=258, wsb=1 << 30) == q.QMM_ERR_ALIGN
    assert L.qmm_attn_prompt_workspace_bytes(q.QMM_BF16, 5, 3, 2, 64, 1) == 0


def test_attn_paged_refuses(L):
    names = ["q", "T", "sq", "nh", "cache", "table", "stride", "cols", "cu", "kvl", "R", "scale", "y",
             "yd", "ws", "wsb", "s"]
    c = _cache()
    need = L.qmm_attn_paged_workspace_bytes(ctypes.byref(c), 3, 4, 3)
    ok = (P, 3, 256, 4, ctypes.byref(c), P, 9, 9, P, P, 3, 0.0, P, q.QMM_F32, P, need, None)
    call = lambda **kw: _call(L.qmm_attn_paged, names, ok, **kw)
    assert call(T=0, q=None, y=None, ws=None) == q.QMM_OK
    for kw, code in BAD_CACHES:
        assert call(cache=ctypes.byref(_cache(**kw))) == code, kw
    for kw, code in ((dict(nh=3), q.QMM_ERR_SHAPE), (dict(cache=None), q.QMM_ERR_INVALID_ARG),
                     (dict(table=None), q.QMM_ERR_INVALID_ARG), (dict(kvl=None), q.QMM_ERR_INVALID_ARG),
                     (dict(cu=None), q.QMM_ERR_INVALID_ARG), (dict(cols=-1), q.QMM_ERR_SHAPE),
                     (dict(stride=8), q.QMM_ERR_SHAPE), (dict(R=-1), q.QMM_ERR_SHAPE),
                     (dict(sq=200), q.QMM_ERR_SHAPE), (dict(sq=258), q.QMM_ERR_ALIGN),
                     (dict(scale=-0.5), q.QMM_ERR_INVALID_ARG), (dict(yd=9), q.QMM_ERR_INVALID_ARG),
                     (dict(wsb=0), q.QMM_ERR_WORKSPACE), (dict(ws=P + 128), q.QMM_ERR_ALIGN)):
        assert call(**kw) == code, kw


# ---------------------------------------------------------------- the binding

DEVICE_MSG = "CUDA device"


def _raises(exc, fn, *a, **kw):
    with pytest.raises(exc) as e:
        fn(*a, **kw)
    return str(e.value)


def test_binding_stops_host_tensors_and_wrong_sizes():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    ok = (i(3), i(3), i(3, 5), i(9), 16, 7)
    assert DEVICE_MSG in _raises(ValueError, q.kv_plan, *ok)
    for n, bad, exc in ((0, torch.zeros(3), TypeError), (1, i(4), ValueError), (2, i(2, 5), ValueError),
                        (2, i(3, 5).long(), TypeError), (2, i(15), TypeError),
                        (3, torch.zeros(9), TypeError)):
        a = list(ok)
        a[n] = bad
        _raises(exc, q.kv_plan, *a)
    cos = torch.zeros(50, 32)
    x = torch.zeros(4, 8 * 64)
    assert DEVICE_MSG in _raises(ValueError, q.rope_append, x, 4, i(4), i(4).long(), cos, cos, None,
                                 n_kv=2)
    _raises(ValueError, q.rope_append, torch.zeros(4, 500), 4, i(4), None, cos, cos, None, n_kv=2)
    _raises(ValueError, q.rope_append, x, 4, i(4), None, cos, torch.zeros(49, 32), None, n_kv=2)
    _raises(ValueError, q.rope_append, x, 4, i(4), None, cos, cos, None)
    host = q.PagedKV(torch.zeros(2, 2, 16, 64), torch.zeros(2, 2, 16, 64))
    assert DEVICE_MSG in _raises(ValueError, q.rope_append, x, 4, i(4), i(4).long(), cos, cos, host)
    qq, k = torch.zeros(4, 4, 64), torch.zeros(4, 2, 64)
    assert DEVICE_MSG in _raises(ValueError, q.attn_prompt, qq, k, k, i(2))
    _raises(ValueError, q.attn_prompt, torch.zeros(4, 256), k, k, i(2))
    assert DEVICE_MSG in _raises(ValueError, q.attn_paged, qq, host, i(1, 2), i(2), i(1))


def test_paged_cache_descriptor_checks(monkeypatch):
    """k and v share shape, type and strides; rows of a block lie together."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    z = lambda *s, **kw: torch.zeros(s, **kw)
    d = q.PagedKV(z(5, 2, 16, 8), z(5, 2, 16, 8))._desc()
    assert (d.num_blocks, d.n_kv, d.block_size, d.head_dim, d.block_stride) == (5, 2, 16, 8, 256)
    both = z(5, 2, 2, 16, 8)
    assert q.PagedKV(both[:, 0], both[:, 1])._desc().block_stride == 512
    for k, v in ((z(5, 2, 16, 8), z(4, 2, 16, 8)), (z(5, 2, 16), z(5, 2, 16)),
                 (z(5, 2, 16, 8), z(5, 2, 16, 8, dtype=torch.bfloat16)),
                 (z(5, 16, 2, 8).transpose(1, 2), z(5, 16, 2, 8).transpose(1, 2)),
                 (both[:, 0], z(5, 2, 16, 8))):
        _raises(ValueError, q.PagedKV(k, v)._desc)
    cache = q.PagedKV(z(5, 2, 16, 8), z(5, 2, 16, 8))
    first = cache._desc()
    assert cache._desc() is first
    cache.k = z(6, 2, 16, 8)
    cache.v = z(6, 2, 16, 8)
    assert cache._desc().num_blocks == 6
    # the calls' own checks, device check aside
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    qq = z(3, 4, 8)
    for a, exc in (((z(3, 4, 12), cache, i(2, 4), i(3), i(2)), ValueError),
                   ((qq.bfloat16(), cache, i(2, 4), i(3), i(2)), ValueError),
                   ((qq, cache, i(3, 4), i(3), i(2)), ValueError),
                   ((qq, cache, i(2, 4), i(4), i(2)), ValueError),
                   ((qq, cache, i(2, 4).long(), i(3), i(2)), TypeError),
                   ((qq, cache, i(4, 2).t(), i(3), i(2)), ValueError),
                   ((qq.transpose(0, 1), cache, i(2, 4), i(3), i(2)), ValueError),
                   ((qq, cache, i(2, 4), i(3), i(2).float()), TypeError)):
        _raises(exc, q.attn_paged, *a)
    _raises(ValueError, q.attn_paged, qq, cache, i(2, 4), i(3), i(2), y=z(3, 4, 9))
    _raises(ValueError, q.attn_paged, qq, cache, i(2, 4), i(6)[::2], i(2))
    cos, x = z(50, 4), z(3, 64)
    for a in ((i(6)[::2], i(3).long(), cos, cos), (i(3), i(6).long()[::2], cos, cos),
              (i(3), i(3).long(), z(50, 8)[:, ::2], cos), (i(3), i(3).long(), cos, z(50, 8)[:, ::2])):
        _raises(ValueError, q.rope_append, x, 4, *a, cache)
    _raises(ValueError, q.kv_plan, i(4)[::2], i(2), i(2, 4), i(9), 16, 5)
    _raises(ValueError, q.kv_plan, i(2), i(2), i(2, 4), i(18)[::2], 16, 5)
    _raises(TypeError, q.attn_paged, qq, cache, i(2, 4), i(3), i(2), y=z(3, 4, 8).half())


# -------------------------------------------------- the reference's own checks

def test_reference_attention_by_hand():
    """Two keys with scores 0 and log 3: weights 1/4 and 3/4; a key a row does
    not see stays out of it."""
    qq = np.array([[[1.0, 0, 0, 0]], [[1.0, 0, 0, 0]]])
    k = np.zeros((2, 1, 4))
    k[1, 0, 0] = np.log(3.0)
    v = np.array([[[4.0, 0, 0, 8]], [[8.0, 4, 0, 0]]])
    y, b = ref.prompt(qq, k, v, [2], 1.0)
    np.testing.assert_allclose(y, [[[4, 0, 0, 8]], [[7, 3, 0, 2]]], rtol=1e-14)
    assert (b > 0).all() and (b < 1e-3).all()
    cache = lambda a: np.stack([a[1:], a[:1]]).transpose(0, 2, 1, 3)  # one row a block, reversed
    y2, _ = ref.paged(qq, cache(k), cache(v), np.array([[1, 0]]), [(2, 2)], 1.0)
    np.testing.assert_array_equal(y, y2)
    y3, _ = ref.paged(qq, cache(k), cache(v), np.array([[7, 0]]), [(2, 2)], 1.0)
    np.testing.assert_allclose(y3, [[[0, 0, 0, 0]], [[8, 4, 0, 0]]])


def test_reference_plan_by_hand():
    table = np.array([[9, -7, -7], [-7, -7, -7]], dtype=np.int32)
    t, cu, kvl, pos, slot, used, short = ref.plan([15, 0], [2, 17], table, [3, 4, 5], 16, 20)
    assert t.tolist() == [[9, 3, -7], [4, 5, -7]] and cu == [0, 2, 19] and kvl == [17, 17]
    assert pos == [15, 16] + list(range(17)) + [-1] and used == 3 and not short
    assert slot == [9 * 16 + 15, 3 * 16] + list(range(64, 80)) + [80, -1]
