"""The binding's own work, without a GPU: what it allocates and where, and what
it keeps in a cache."""
import contextlib
import copy
import io
import pickle

import pytest
import torch

import sliding_window_kv_swa_gb300 as nd


class FakeLibrary:
    """Sizes are 4096, statuses ND_OK; nothing is launched."""
    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("_size") else 0


class OtherStream(torch.cuda.Stream if torch.cuda.is_available() else object):
    cuda_stream = 77


def calls(stream):
    """Every entry point that makes a workspace or an output when it is given none."""
    B, T, Hq, Hkv, d = 2, 16, 4, 2, 64
    x = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    cache, prefix = nd.KVCache.empty(B, Hkv, d, 4, 8, device="cpu"), nd.KVCache.empty(1, Hkv, d, 600, 0, device="cpu")
    comp = nd.CompressedCache.empty(B, Hkv, d, 4, 8, 4, device="cpu")
    q, k, Q, K = x(B, Hq, d), x(B, Hkv, d), x(B, T, Hq, d), x(B, T, Hkv, d)
    kw = dict(stream=stream)
    return {
        "nd_kv_cache_from_prefill": lambda: nd.nd_kv_cache_from_prefill(cache, K, K, i32(B), **kw),
        "nd_swa_sink_decode": lambda: nd.nd_swa_sink_decode(q, cache, 8, **kw),
        "nd_swa_sink_decode_step": lambda: nd.nd_swa_sink_decode_step(q, cache, k, k, 8, **kw),
        "nd_swa_sink_decode_step_host": lambda: nd.nd_swa_sink_decode_step_host(q, cache, k, k, 8, x(B, Hq, d), **kw),
        "nd_swa_sink_decode_step_host_packed":
            lambda: nd.nd_swa_sink_decode_step_host_packed(x(B * (Hq + 2 * Hkv) * d), cache, Hq, 8, x(B, Hq, d), **kw),
        "nd_kv_cache_read": lambda: nd.nd_kv_cache_read(cache, 8, **kw),
        "nd_shared_prefix_decode": lambda: nd.nd_shared_prefix_decode(q, prefix, cache, 8, **kw),
        "nd_qk_norm_rope": lambda: nd.nd_qk_norm_rope(Q, K, **kw),
        "nd_qk_norm_rope_append": lambda: nd.nd_qk_norm_rope_append(q, cache, k, k, **kw),
        "nd_compressed_decode_step": lambda: nd.nd_compressed_decode_step(q, comp, k, k, 8, **kw),
        "nd_swa_sink_prefill": lambda: nd.nd_swa_sink_prefill(Q, K, K, **kw),
        "nd_compressed_prefill": lambda: nd.nd_compressed_prefill(Q, K, K, 8, 4, **kw),
        "nd_swa_sink_chunk_prefill": lambda: nd.nd_swa_sink_chunk_prefill(Q, K, K, cache, 8, **kw),
        "nd_rope_apply": lambda: nd.nd_rope_apply(Q, **kw),
        "nd_kv_compress_pool": lambda: nd.nd_kv_compress_pool(K, K, 4, **kw),
        "nd_kv_compress_pool_rope": lambda: nd.nd_kv_compress_pool_rope(K, K, 4, 1e4, **kw),
    }


@pytest.mark.parametrize("name", sorted(calls(None)))
def test_what_a_call_makes_belongs_to_the_stream_it_runs_on(name, monkeypatch):
    """A workspace from another stream's memory would be handed on, when the call returns, to that stream's next tensor
    while the call's kernels still use it."""
    stream, inside, made = OtherStream.__new__(OtherStream), [], []

    @contextlib.contextmanager
    def on(s):
        inside.append(s)
        yield
        inside.pop()

    def watched(fn):
        def make(*a, **kw):
            made.append(bool(inside) and inside[-1].cuda_stream == stream.cuda_stream)
            return fn(*a, **kw)
        return make

    m = nd.nd
    call = calls(stream)[name]
    monkeypatch.setattr(m, "_lib", FakeLibrary)
    monkeypatch.setattr(m, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(m, "_here", lambda t: -1)   # the index that a host tensor gives
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: stream)
    monkeypatch.setattr(torch, "empty", watched(torch.empty))
    monkeypatch.setattr(torch, "empty_like", watched(torch.empty_like))
    call()
    assert made and all(made), f"{made.count(False)} of {len(made)} tensors made on the current stream"


def test_a_cache_that_a_call_has_seen_can_be_copied_and_saved():
    """deepcopy, pickle and torch.save of a cache after its address was kept for the calls; the copy's own address."""
    cache = nd.KVCache.empty(2, 2, 64, 4, 8, device="cpu")
    cache.k_codes.random_(-127, 128)
    before = set(vars(cache))
    cache.struct_ref()
    for copied in (copy.deepcopy(cache), pickle.loads(pickle.dumps(cache)), copy.copy(cache), saved(cache)):
        assert set(vars(copied)) == before and (copied.sink_cap, copied.ring_cap) == (4, 8)
        assert torch.equal(copied.k_codes, cache.k_codes)
        s = copied.struct_ref()._obj
        assert s.k_codes == copied.k_codes.data_ptr() and s.seq_len == copied.seq_len.data_ptr()
    assert cache.struct_ref() is cache.struct_ref()
    comp = nd.CompressedCache.empty(2, 2, 64, 4, 8, 4, device="cpu")
    comp.kv.struct_ref()
    copy.deepcopy(comp), pickle.dumps(comp)


def saved(cache):
    f = io.BytesIO()
    torch.save(cache, f)
    return torch.load(io.BytesIO(f.getvalue()), weights_only=False)


@pytest.mark.parametrize("field", ["k_codes", "v_codes", "k_scale", "v_scale", "sink_len", "ring_start", "ring_len", "seq_len"])
def test_a_cache_whose_tensors_are_not_in_the_layout_is_refused(field):
    """The kernels go by the sizes alone: a tensor that is shorter would be read past its end, one with other strides
    or another type read wrongly."""
    def changed(make):
        cache = nd.KVCache.empty(2, 2, 64, 4, 8, device="cpu")
        setattr(cache, field, make(getattr(cache, field)))
        return cache

    wrong = [lambda t: t[:1], lambda t: t.repeat_interleave(2, -1)[..., ::2], lambda t: t.double(), lambda t: t.to("meta")]
    for make in wrong:
        with pytest.raises(ValueError):
            changed(make).struct_ref()
    assert changed(torch.clone).struct_ref()._obj.batch == 2


def test_a_cache_whose_capacities_are_not_its_tensors_is_refused():
    for sinks, ring in ((5, 8), (4, 7), (8, 4), (12, 0), (13, -1)):
        cache = nd.KVCache.empty(2, 2, 64, 4, 8, device="cpu")
        cache.sink_cap, cache.ring_cap = sinks, ring
        if sinks + ring == 12 and ring >= 0:
            assert cache.struct_ref()._obj.sink_cap == sinks
        else:
            with pytest.raises(ValueError):
                cache.struct_ref()
