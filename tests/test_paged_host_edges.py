"""Further refusals of the paged-cache entry points, on the CPU (see
tests/test_paged_host.py: addresses that are never dereferenced, and only
where no GPU is visible)."""
import ctypes

import pytest
import torch

import group_quantized_moe_gb300 as q
from test_paged_host import L  # noqa: F401 (fixture)

P = 0x7F0000000000
GAP = 1 << 32
NAMES = ["ctx", "new", "R", "S", "table", "stride", "cols", "free", "nfree", "T", "cu", "kvl", "pos",
         "slots", "used", "s"]
BYTES = dict(ctx=16, new=16, free=40, cu=20, kvl=16, pos=80, slots=160, used=4)
OUT = ("cu", "kvl", "pos", "slots", "used")


def _plan(L, **kw):
    """qmm_kv_plan of 4 requests, 20 token rows, a table of 4 x 8 in rows of 12."""
    a = dict(R=4, S=16, stride=12, cols=8, nfree=10, T=20, s=None)
    for i, k in enumerate(("ctx", "new", "table", "free") + OUT):
        a[k] = P + i * GAP
    a.update(kw)
    return L.qmm_kv_plan(*(a[k] for k in NAMES)), a


@pytest.mark.parametrize("out", OUT)
def test_kv_plan_refuses_outputs_on_its_inputs(L, out):
    base = _plan(L)[1]
    for other in BYTES:
        if other == out:
            continue
        word = 8 if "slots" in (out, other) else 4  # (slots lie at multiples of 8)
        size = {k: -(-BYTES[k] // word) * word for k in (out, other)}
        for at in (0, size[other] - word, word - size[out]):  # same start, its last word, our last word
            rc, _ = _plan(L, **{out: base[other] + at})
            assert rc == q.QMM_ERR_INVALID_ARG and "overlaps" in q.qmm_last_error(), (out, other, at)
        for at in (size[other], -size[out]):  # side by side: nothing shared
            rc, _ = _plan(L, **{out: base[other] + at})
            assert rc == q.QMM_ERR_CUDA, (out, other, at, q.qmm_last_error())


@pytest.mark.parametrize("name", sorted(BYTES))
def test_kv_plan_refuses_vectors_in_the_table(L, name):
    t = _plan(L)[1]["table"]
    n = BYTES[name]
    word = 8 if name == "slots" else 4
    for at in (0, 31, 48, 3 * 48 + 28, word - n):
        at -= at % word
        assert _plan(L, **{name: t + at})[0] == q.QMM_ERR_INVALID_ARG, (name, at)
    for at in (3 * 48 + 32, -n):  # behind the last row's columns, before the first
        assert _plan(L, **{name: t + at})[0] == q.QMM_ERR_CUDA, (name, at)
    if n <= 16:  # between two rows' columns
        assert _plan(L, **{name: t + 48 + 32})[0] == q.QMM_ERR_CUDA, name


def test_kv_plan_without_rows_overlaps_nothing(L):
    """Vectors of no elements have no memory."""
    p = P + 100 * GAP
    assert _plan(L, R=0, T=0, nfree=0, ctx=p, new=p, kvl=p, pos=p, slots=p, free=p, table=p)[0] \
        == q.QMM_ERR_CUDA


def test_misaligned_integer_arrays_are_refused(L):
    for name in ("ctx", "new", "table", "free", "cu", "kvl", "pos", "used"):
        for at in (1, 2):
            assert _plan(L, **{name: _plan(L)[1][name] + at})[0] == q.QMM_ERR_ALIGN, name
    assert _plan(L, slots=_plan(L)[1]["slots"] + 4)[0] == q.QMM_ERR_ALIGN
    cache = q._KvCache(q.QMM_BF16, 2, 64, 16, 10, P, P, 2 * 16 * 64)
    c = ctypes.byref(cache)

    def append(pos=P, slots=P):
        return L.qmm_rope_append(P, q.QMM_F32, 3, 512, 4, 2, 64, pos, slots, P, P, 100, c, P, P, P,
                                 q.QMM_BF16, None)
    assert append(pos=P + 2) == append(slots=P + 4) == q.QMM_ERR_ALIGN
    assert append() == q.QMM_ERR_CUDA

    def prompt(cu=P):
        n = L.qmm_attn_prompt_workspace_bytes(q.QMM_BF16, 5, 4, 2, 64, 1)
        return L.qmm_attn_prompt(P, P, P, q.QMM_BF16, 5, 256, 128, 128, 4, 2, 64, cu, 1, 0.0, P, q.QMM_F32,
                                 P, n, None)
    assert prompt(P + 1) == q.QMM_ERR_ALIGN and prompt() == q.QMM_ERR_CUDA

    def paged(table=P, cu=P, kvl=P):
        n = L.qmm_attn_paged_workspace_bytes(c, 3, 4, 3)
        return L.qmm_attn_paged(P, 3, 256, 4, c, table, 9, 9, cu, kvl, 3, 0.0, P, q.QMM_F32, P, n, None)
    assert paged(table=P + 2) == paged(cu=P + 2) == paged(kvl=P + 1) == q.QMM_ERR_ALIGN
    assert paged() == q.QMM_ERR_CUDA


# ---------------------------------------------------------------- the binding

def _ints(*s):
    return torch.zeros(s, dtype=torch.int32)


def test_attention_refuses_other_output_types(monkeypatch):
    """A type that the library cannot write is a TypeError before any memory is made."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    monkeypatch.setattr(q, "_new", lambda *a: pytest.fail("allocated"))
    x, kv = torch.zeros(3, 4, 64), torch.zeros(3, 2, 64)
    cache = q.PagedKV(torch.zeros(2, 2, 16, 64), torch.zeros(2, 2, 16, 64))
    for bad in (torch.float16, torch.float64, torch.int32, None):
        with pytest.raises(TypeError, match="float32 or bfloat16"):
            q.attn_prompt(x, kv, kv, _ints(2), y_dtype=bad)
        with pytest.raises(TypeError, match="float32 or bfloat16"):
            q.attn_paged(x, cache, _ints(1, 2), _ints(2), _ints(1), y_dtype=bad)


def test_cache_of_one_head_may_have_any_stride_there(monkeypatch):
    """[blocks, rows, 1, columns] seen as [blocks, 1, rows, columns] is the same memory."""
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
    rows = [torch.zeros(5, 16, 1, 64) for _ in range(2)]
    k, v = (t.transpose(1, 2) for t in rows)
    assert k.stride(1) == 64 and k.is_contiguous()
    d = q.PagedKV(k, v)._desc()
    assert (d.num_blocks, d.n_kv, d.block_size, d.head_dim, d.block_stride) == (5, 1, 16, 64, 1024)
    both = torch.zeros(5, 2, 16, 1, 64)
    d = q.PagedKV(both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2))._desc()
    assert d.block_stride == 2048
    for t in (torch.zeros(5, 16, 2, 64).transpose(1, 2), torch.zeros(5, 1, 64, 16).transpose(2, 3),
              torch.zeros(5, 1, 16, 128)[..., ::2]):
        with pytest.raises(ValueError):
            q.PagedKV(t, t)._desc()
