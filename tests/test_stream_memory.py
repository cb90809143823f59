"""Calls on another stream than the current one: where their memory comes from.

A call with ``stream=s`` has to allocate from s's own pool.  Memory of the
current stream's pool may have been freed a moment ago with its last kernel
still queued there, and nothing orders s behind that kernel.  What the call
hands out is recorded on the current stream too, where the caller reads it.

The CPU tests run the binding with a library that does nothing and with
stand-ins for torch's streams that note what was allocated where.
"""
import contextlib

import pytest
import torch

import group_quantized_moe_gb300 as q

F32, I32 = torch.float32, torch.int32


class _Nothing:
    """A library whose calls succeed without doing anything."""

    def __getattr__(self, name):
        return lambda *a: 64 if name.endswith("_bytes") else 0


class _Log:
    def __init__(self, monkeypatch):
        self.now, self.made, self.recorded = [], [], []
        empty, log = torch.empty, self

        @contextlib.contextmanager
        def on(stream):
            log.now.append(stream)
            yield
            log.now.pop()

        def spy(*a, **kw):
            t = empty(*a, **kw)
            log.made.append((t, log.now[-1] if log.now else "current"))
            return t

        monkeypatch.setattr(q, "lib", lambda: _Nothing())
        monkeypatch.setattr(torch, "empty", spy)
        monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda t: True))
        monkeypatch.setattr(torch.Tensor, "record_stream",
                            lambda t, s: log.recorded.append((t.data_ptr(), s)))
        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, *a: ("stream", h))
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: "the caller's")
        monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: "default")
        # not there before a CUDA build of torch is initialised
        monkeypatch.setattr(q, "_stream", lambda stream: 0 if stream is None else int(stream))


@pytest.fixture
def log(monkeypatch):
    return _Log(monkeypatch)


def _weight(N, K):
    G = K // 64
    return q.QWeight(8, 64, N, K, torch.zeros((N, K), dtype=torch.int8), torch.zeros((N, G)),
                     torch.zeros((N, G), dtype=I32))


def _experts(E, H, I):
    z = lambda *s, dt=F32: torch.zeros(s, dtype=dt)
    m = lambda r, c: (z(E, r, c, dt=torch.int8), z(E, r, c // 64), z(E, r, c // 64, dt=I32))
    return q.MoeExperts(E, H, I, 8, 64, *m(I, H), *m(I, H), *m(H, I))


def _cases():
    i = lambda *s: torch.zeros(s, dtype=I32)
    z = lambda *s: torch.zeros(s)
    nh, nkv, hd, D, T = 4, 2, 32, 128, 5
    cos = z(16, hd // 2)
    w = lambda: _weight((nh + 2 * nkv) * hd, D)
    cache = lambda: q.PagedKV(z(3, nkv, 16, hd), z(3, nkv, 16, hd))
    plan = lambda: q.KVPlan(i(3), i(2), i(T), i(T).long(), i(1))
    layer = lambda: q.AttnLayer(nh, nkv, hd, 16, _weight(nh * hd, D), _weight(nkv * hd, D),
                                _weight(nkv * hd, D), _weight(D, nh * hd), cos, cos)
    return {
        "kv_plan": lambda s: q.kv_plan(i(2), i(2), i(2, 3), i(6), 16, T, stream=s),
        "rope_append": lambda s: q.rope_append(z(T, 8 * hd), nh, i(T), i(T).long(), cos, cos, cache(),
                                               keep_kv=True, stream=s),
        "attn_prompt": lambda s: q.attn_prompt(z(T, nh, hd), z(T, nkv, hd), z(T, nkv, hd), i(2), stream=s),
        "attn_paged": lambda s: q.attn_paged(z(T, nh, hd), cache(), i(2, 3), i(3), i(2), stream=s),
        "attn_layer_paged": lambda s: q.attn_layer_paged(z(T, D), w(), _weight(D, nh * hd), nh, cos, cos,
                                                         cache(), plan(), i(2, 3), stream=s),
        "attn_layer_paged, prompts": lambda s: q.attn_layer_paged(
            z(T, D), w(), _weight(D, nh * hd), nh, cos, cos, cache(), plan(), i(2, 3), prompts=True,
            stream=s),
        "qmm_quantize_groupwise": lambda s: q.qmm_quantize_groupwise(z(16, 64), 8, 64, stream=s),
        "qmm_linear": lambda s: q.qmm_linear(z(T, D), w(), stream=s),
        "qmm_linear_batched": lambda s: q.qmm_linear_batched(z(T, D), w(), stream=s),
        "moe_route_topk": lambda s: q.moe_route_topk(z(T, D), z(8, D), None, 2, stream=s),
        "moe_route_topk_noalloc": lambda s: q.moe_route_topk_noalloc(z(T, D), z(8, D), None, 2, stream=s),
        "moe_route_load_stats": lambda s: q.moe_route_load_stats(i(8), 3, stream=s),
        "moe_ffn_forward": lambda s: q.moe_ffn_forward(z(T, D), i(T, 2), z(T, 2), _experts(2, D, 64),
                                                       stream=s),
        "moe_decode_forward": lambda s: q.moe_decode_forward(z(T, D), z(2, D), None, 2,
                                                             _experts(2, D, 64), stream=s),
        "rope_table": lambda s: q.rope_table(16, hd, device="cpu", stream=s),
        "quantize_attn_layer": lambda s: q.quantize_attn_layer(
            z(nh * hd, D), z(nkv * hd, D), z(nkv * hd, D), z(D, nh * hd), nh, nkv, hd, 16, stream=s),
        "attn_decode": lambda s: q.attn_decode(z(D), 0, layer(), z(2, nkv, 16, hd), stream=s),
    }


@pytest.mark.parametrize("name", sorted(_cases()))
def test_memory_of_a_call_comes_from_its_streams_pool(log, name):
    call = _cases()[name]
    call(None)
    assert log.made and all(where == "current" for _, where in log.made) and not log.recorded
    log.made.clear()
    call(4096)
    assert log.made and all(where == ("stream", 4096) for _, where in log.made), \
        [(tuple(t.shape), where) for t, where in log.made]
    # ... and what it hands out is the caller's stream's to read
    missing = [tuple(t.shape) for t, _ in log.made if t.numel()
               and (t.data_ptr(), "the caller's") not in log.recorded]
    assert not missing, missing


def test_default_stream_handle(log):
    """Handle 0 is the default stream, not a new one."""
    q.rope_table(16, 32, device="cpu", stream=0)
    assert [where for _, where in log.made] == ["default", "default"]


def test_stacked_projections_are_made_where_they_are_read(log, monkeypatch):
    """The copy that stacks wq, wk and wv runs on the call's stream."""
    cat, seen = torch.cat, []
    monkeypatch.setattr(torch, "cat", lambda *a, **kw: (seen.append(list(log.now)), cat(*a, **kw))[1])
    _cases()["quantize_attn_layer"](4096)
    assert seen == [[("stream", 4096)]]


@pytest.mark.gpu
def test_memory_freed_on_the_current_stream_is_not_handed_to_another():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from group_quantized_moe_gb300 import build_lib
    build_lib.build()
    T, nh, hd = 2048, 8, 128
    x = [torch.randn((T, nh, hd), device="cuda") for _ in range(3)]
    cu = torch.tensor([0, T], dtype=I32, device="cuda")
    want = q.attn_prompt(*x, cu)
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        torch.cuda.synchronize()
        freed = [torch.empty((T, nh, hd), device="cuda") for _ in range(4)]
        spans = [(t.data_ptr(), t.data_ptr() + t.nbytes) for t in freed]
        del freed
        y = q.attn_prompt(*x, cu, stream=stream)
        assert not any(a < y.data_ptr() + y.nbytes and y.data_ptr() < b for a, b in spans)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(y, want)
    z = q.attn_prompt(*x, cu, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(z, want)
