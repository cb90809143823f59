"""Refusals of the 4-bit cache's entry points, on the CPU (see
tests/test_paged_host.py), and the reference's own checks."""
import ctypes

import numpy as np
import pytest
import torch

import group_quantized_moe_gb300 as q
import kv4_reference as ref
from test_paged_host import BIG, P, L, _call, _raises  # noqa: F401 (L: fixture)
from test_stream_memory import _Log


def _cache(nkv=2, hd=64, group=64, S=16, nb=10, data=P, stride=2 * (1024 + 128)):
    return q._Kv4Cache(nkv, hd, group, S, nb, data, stride)


BAD_CACHES = [(dict(nkv=0), q.QMM_ERR_SHAPE), (dict(nkv=2000, stride=BIG), q.QMM_ERR_UNSUPPORTED),
              (dict(hd=60), q.QMM_ERR_UNSUPPORTED), (dict(hd=4), q.QMM_ERR_UNSUPPORTED),
              (dict(hd=264), q.QMM_ERR_UNSUPPORTED), (dict(group=16), q.QMM_ERR_UNSUPPORTED),
              (dict(group=128), q.QMM_ERR_UNSUPPORTED), (dict(S=48), q.QMM_ERR_UNSUPPORTED),
              (dict(S=8), q.QMM_ERR_UNSUPPORTED), (dict(S=512), q.QMM_ERR_UNSUPPORTED),
              (dict(nb=-1), q.QMM_ERR_SHAPE), (dict(nb=1 << 31), q.QMM_ERR_SHAPE),
              (dict(stride=2 * 1152 - 16), q.QMM_ERR_SHAPE), (dict(stride=BIG), q.QMM_ERR_SHAPE),
              (dict(data=None), q.QMM_ERR_INVALID_ARG), (dict(data=P + 8), q.QMM_ERR_ALIGN),
              (dict(stride=2 * 1152 + 8), q.QMM_ERR_ALIGN)]


def test_block_bytes(L):
    for hd, nc in ((8, 1), (32, 1), (40, 2), (96, 3), (128, 4), (136, 6), (192, 6), (200, 8), (256, 8)):
        for group in (32, 64):
            strip = 512 * nc + 128 * -(-hd // group)
            assert ref.strip_bytes(hd, group) == strip
            for S in (16, 64, 256):
                assert q.qmm_kv4_block_bytes(3, hd, group, S) == 3 * S // 16 * strip
    for bad in ((3, 12, 64, 16), (0, 64, 64, 16), (3, 64, 48, 16), (3, 64, 64, 17), (3, 288, 64, 16)):
        assert L.qmm_kv4_block_bytes(*bad) == 0
        with pytest.raises(q.QmmError):
            q.qmm_kv4_block_bytes(*bad)


def test_append_refuses(L):
    names = ["x", "xd", "T", "stride", "nh", "pos", "slots", "cos", "sin", "max", "cache", "q", "k", "v", "yd", "s"]
    ok = (P, q.QMM_F32, 3, 512, 4, P, P, P, P, 100, ctypes.byref(_cache()), P, P, P, q.QMM_BF16, None)
    call = lambda **kw: _call(L.qmm_rope_append_kv4, names, ok, **kw)
    assert call(T=0, x=None, q=None) == q.QMM_OK
    assert call(cache=None) == q.QMM_ERR_INVALID_ARG
    for kw, code in BAD_CACHES:
        assert call(cache=ctypes.byref(_cache(**kw))) == code, kw
    for kw, code in ((dict(nh=0), q.QMM_ERR_SHAPE), (dict(nh=5), q.QMM_ERR_SHAPE),
                     (dict(nh=2050), q.QMM_ERR_UNSUPPORTED), (dict(xd=2), q.QMM_ERR_INVALID_ARG),
                     (dict(yd=3), q.QMM_ERR_INVALID_ARG), (dict(T=-1), q.QMM_ERR_SHAPE),
                     (dict(max=-1), q.QMM_ERR_SHAPE), (dict(stride=511), q.QMM_ERR_SHAPE),
                     (dict(stride=BIG), q.QMM_ERR_SHAPE), (dict(stride=514), q.QMM_ERR_ALIGN),
                     (dict(stride=516, xd=q.QMM_BF16), q.QMM_ERR_ALIGN), (dict(x=P + 4), q.QMM_ERR_ALIGN),
                     (dict(k=P + 8), q.QMM_ERR_ALIGN), (dict(cos=P + 8), q.QMM_ERR_ALIGN),
                     (dict(pos=P + 2), q.QMM_ERR_ALIGN), (dict(slots=P + 4), q.QMM_ERR_ALIGN),
                     (dict(x=None), q.QMM_ERR_INVALID_ARG), (dict(pos=None), q.QMM_ERR_INVALID_ARG),
                     (dict(slots=None), q.QMM_ERR_INVALID_ARG), (dict(sin=None), q.QMM_ERR_INVALID_ARG),
                     (dict(q=None), q.QMM_ERR_INVALID_ARG)):
        assert call(**kw) == code, kw
        assert q.qmm_last_error()


def test_read_refuses(L):
    names = ["cache", "slots", "n", "k", "v", "yd", "s"]
    ok = (ctypes.byref(_cache()), P, 3, P, P, q.QMM_F32, None)
    call = lambda **kw: _call(L.qmm_kv4_read, names, ok, **kw)
    assert call(n=0, slots=None, k=None, v=None) == q.QMM_OK
    for kw, code in BAD_CACHES:
        assert call(cache=ctypes.byref(_cache(**kw))) == code, kw
    for kw, code in ((dict(n=-1), q.QMM_ERR_SHAPE), (dict(slots=None), q.QMM_ERR_INVALID_ARG),
                     (dict(k=None, v=None), q.QMM_ERR_INVALID_ARG), (dict(yd=2), q.QMM_ERR_INVALID_ARG),
                     (dict(k=P + 8), q.QMM_ERR_ALIGN), (dict(slots=P + 4), q.QMM_ERR_ALIGN)):
        assert call(**kw) == code, kw


def test_attend_refuses(L):
    names = ["q", "qd", "T", "sq", "nh", "cache", "table", "stride", "cols", "cu", "kvl", "R", "scale", "y", "yd",
             "ws", "wsb", "s"]
    c = _cache()
    for dt in (q.QMM_F32, q.QMM_BF16):
        need = L.qmm_attn_paged_kv4_workspace_bytes(ctypes.byref(c), dt, 3, 4, 3)
        assert need > 0
        ok = (P, dt, 3, 256, 4, ctypes.byref(c), P, 9, 9, P, P, 3, 0.0, P, q.QMM_F32, P, need, None)
        call = lambda **kw: _call(L.qmm_attn_paged_kv4, names, ok, **kw)
        assert call(T=0, q=None, y=None, ws=None) == q.QMM_OK
        for kw, code in BAD_CACHES:
            assert call(cache=ctypes.byref(_cache(**kw))) == code, kw
        for kw, code in ((dict(nh=3), q.QMM_ERR_SHAPE), (dict(cache=None), q.QMM_ERR_INVALID_ARG),
                         (dict(table=None), q.QMM_ERR_INVALID_ARG), (dict(kvl=None), q.QMM_ERR_INVALID_ARG),
                         (dict(cu=None), q.QMM_ERR_INVALID_ARG), (dict(cols=-1), q.QMM_ERR_SHAPE),
                         (dict(stride=8), q.QMM_ERR_SHAPE), (dict(R=-1), q.QMM_ERR_SHAPE),
                         (dict(T=-1), q.QMM_ERR_SHAPE), (dict(T=1 << 30), q.QMM_ERR_UNSUPPORTED),
                         (dict(sq=200), q.QMM_ERR_SHAPE), (dict(sq=258), q.QMM_ERR_ALIGN),
                         (dict(scale=-0.5), q.QMM_ERR_INVALID_ARG), (dict(scale=float("nan")), q.QMM_ERR_INVALID_ARG),
                         (dict(yd=9), q.QMM_ERR_INVALID_ARG), (dict(qd=2), q.QMM_ERR_INVALID_ARG),
                         (dict(wsb=0), q.QMM_ERR_WORKSPACE), (dict(wsb=need - 1), q.QMM_ERR_WORKSPACE),
                         (dict(ws=P + 128), q.QMM_ERR_ALIGN), (dict(cu=P + 2), q.QMM_ERR_ALIGN)):
            assert call(**kw) == code, kw
    assert L.qmm_attn_paged_kv4_workspace_bytes(ctypes.byref(c), 2, 3, 4, 3) == 0
    assert L.qmm_attn_paged_kv4_workspace_bytes(ctypes.byref(c), 0, 3, 5, 3) == 0


# ---------------------------------------------------------------- the binding

def test_binding_refuses(monkeypatch, L):
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    n = 1152
    host = q.PagedKV4(torch.zeros(5, 2, n, dtype=torch.uint8), 64, 64, 16)
    cos, x, qq = torch.zeros(50, 32), torch.zeros(4, 8 * 64), torch.zeros(4, 4, 64)
    for call in (lambda: q.rope_append(x, 4, i(4), i(4).long(), cos, cos, host),
                 lambda: q.attn_paged(qq, host, i(1, 2), i(2), i(1)), lambda: q.kv4_read(host, i(3).long())):
        assert "CUDA device" in _raises(ValueError, call)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    z = lambda *s: torch.zeros(s, dtype=torch.uint8)
    d = q.PagedKV4(z(5, 2, n), 64, 64, 16)._desc()
    assert (d.num_blocks, d.n_kv, d.head_dim, d.group, d.block_size, d.block_stride) == (5, 2, 64, 64, 16, 2 * n)
    assert q.PagedKV4(z(5, 3, 2, n)[:, 1], 64, 64, 16)._desc().block_stride == 6 * n
    for data, form, exc in ((z(5, 2, n + 16), (64, 64, 16), ValueError), (z(5, 2, n), (64, 32, 16), ValueError),
                            (z(5, 2, n).float(), (64, 64, 16), TypeError), (z(5, 2 * n), (64, 64, 16), TypeError),
                            (z(5, n, 2).transpose(1, 2), (64, 64, 16), ValueError),
                            (z(5, 2, n), (60, 64, 16), q.QmmError), (z(5, 2, n), (64, 64, 24), q.QmmError)):
        _raises(exc, q.PagedKV4(data, *form)._desc)
    cache = q.PagedKV4(z(5, 2, n), 64, 64, 16)
    assert cache._desc() is cache._desc()
    cache.data = z(6, 2, n)
    assert cache._desc().num_blocks == 6
    # a tensor of another device than the current one
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    for call in (lambda: q.rope_append(x, 4, i(4), i(4).long(), cos, cos, cache),
                 lambda: q.attn_paged(qq, cache, i(1, 2), i(2), i(1)), lambda: q.kv4_read(cache, i(3).long())):
        assert "current CUDA device" in _raises(ValueError, call)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    for a, exc in (((torch.zeros(4, 4, 72), cache, i(2, 4), i(3), i(2)), ValueError),
                   ((qq.half(), cache, i(2, 4), i(3), i(2)), TypeError),
                   ((qq, cache, i(3, 4), i(3), i(2)), ValueError), ((qq, cache, i(2, 4), i(4), i(2)), ValueError),
                   ((qq, cache, i(2, 4).long(), i(3), i(2)), TypeError),
                   ((qq.transpose(0, 1), cache, i(2, 4), i(3), i(2)), ValueError)):
        _raises(exc, q.attn_paged, *a)
    ok = (x, 4, i(4), i(4).long(), cos, cos, cache)
    for at, bad, exc in ((0, torch.zeros(4, 500), ValueError), (2, i(5), ValueError), (3, i(4), TypeError),
                         (3, None, ValueError), (4, torch.zeros(50, 16), ValueError)):
        a = list(ok)
        a[at] = bad
        _raises(exc, q.rope_append, *a)
    _raises(ValueError, q.rope_append, *ok, n_kv=4)
    _raises(TypeError, q.rope_append, *ok, y_dtype=torch.float16)
    _raises(TypeError, q.rope_append, *ok, q=torch.zeros(4, 4, 64))  # bf16 unless y_dtype says otherwise
    _raises(ValueError, q.rope_append, *ok, k=torch.zeros(4, 2, 72).bfloat16())
    _raises(TypeError, q.kv4_read, cache, i(3))
    _raises(TypeError, q.kv4_read, cache, i(3).long(), y_dtype=torch.float16)
    _raises(ValueError, q.kv4_read, cache, i(3).long(), k=torch.zeros(3, 2, 72))
    _raises(TypeError, q.kv4_read, cache, i(3).long(), v=torch.zeros(3, 2, 64).bfloat16())


def test_memory_of_another_stream(monkeypatch):
    """Outputs and workspaces of a call on another stream come from its pool."""
    log = _Log(monkeypatch)
    monkeypatch.setattr(torch.Tensor, "get_device", lambda t: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(q, "qmm_kv4_block_bytes", lambda *a: 2 * 1152)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    cache = q.PagedKV4(torch.zeros(5, 2, 1152, dtype=torch.uint8), 64, 64, 16)
    cos, x, qq = torch.zeros(50, 32), torch.zeros(4, 8 * 64), torch.zeros(4, 4, 64)
    for call in (lambda: q.rope_append(x, 4, i(4), i(4).long(), cos, cos, cache, keep_kv=True, stream=77),
                 lambda: q.attn_paged(qq, cache, i(1, 2), i(2), i(1), stream=77),
                 lambda: q.kv4_read(cache, i(3).long(), stream=77)):
        log.made.clear()
        call()
        assert log.made and all(where == ("stream", 77) for _, where in log.made)


# -------------------------------------------------- the reference's own checks

def test_quantise_by_hand():
    """Two groups: -1 .. 2 in steps of a fifth (scale 0.2, the next bf16 0.2002);
    a constant, which its zero point holds."""
    x = np.concatenate([np.linspace(-1, 2, 32), np.full(32, 5.0)]).astype(np.float32)
    c, z, s = ref.quantise(x, 32)
    assert s[0] == 0.2001953125 and z[0] == 5 and c[0] == 0 and c[31] == 15
    assert s[1] == np.float32(5 / 2048) and z[1] == -2048 and (c[32:] == 0).all()
    v = ref.values((c.astype(float), z.astype(float), s.astype(float)), 32)
    assert np.abs(v[:32] - x[:32]).max() <= 0.1002 and (v[32:] == 5).all()
    c, z, s = ref.quantise(np.array([0.0] * 31 + [np.inf], np.float32), 32)
    assert not c.any() and z[0] == 0 and np.isnan(s[0])


@pytest.mark.parametrize("hd,group,S", [(128, 64, 32), (80, 32, 16), (160, 32, 16), (8, 64, 16)])
def test_layout_round_trip(hd, group, S):
    rng = np.random.default_rng(1)
    nb, nkv = 2, 2
    x = [rng.standard_normal((nb * S, nkv, hd)).astype(np.float32) for _ in range(2)]
    data = np.full((nb, nkv, S // 16 * ref.strip_bytes(hd, group)), 0xA5, dtype=np.uint8)
    for slot in rng.permutation(nb * S):
        ref.put(data, hd, group, S, int(slot), x[0][slot], x[1][slot])
    for got, want in zip(ref.unpack(data, hd, group, S), x):
        codes, zp, s = ref.quantise(want, group)
        back = lambda t: t.reshape(nb, S, nkv, -1).swapaxes(1, 2)
        assert (got[0] == back(codes)).all() and (got[1] == back(zp)).all() and (got[2] == back(s)).all()
