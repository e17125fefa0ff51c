"""Refusals of the shared-prefix decode, the per-head norm with rotation, its
append and the cache read-back: every bad argument is answered on the host, with
the status the header gives, before anything is enqueued (no GPU is needed)."""
import ctypes

import pytest
import torch

import sliding_window_kv_swa_gb300 as nd

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = range(5)
P, Z, F, L = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float, ctypes.c_int64
A, BAD = P(4096), P(4104)   # aligned and misaligned addresses; nothing is read


def cache(B=1, Hkv=2, d=64, S=4, W=8, ptr=4096):
    return nd.nd._Cache(B, Hkv, d, S, W, *([ptr] * 8))


def lib():
    return nd.nd._lib()


def test_shared_prefix_decode():
    def call(prefix=cache(S=100), own=cache(), Hq=8, window=8, q=A, out=A, ws=A, size=1 << 30):
        ref = lambda c: None if c is None else ctypes.byref(c)
        return lib().nd_shared_prefix_decode(q, ref(prefix), ref(own), Hq, window, out, None, ws, Z(size), None)

    assert call(prefix=None) == INVALID and call(own=None) == INVALID
    assert call(prefix=cache(B=2, S=100)) == INVALID and call(prefix=cache(B=0, S=100)) == INVALID
    assert call(prefix=cache(S=0)) == INVALID
    assert call(prefix=cache(Hkv=1, S=100)) == INVALID and call(prefix=cache(d=128, S=100)) == INVALID
    assert call(prefix=cache(S=100, ptr=0)) == INVALID and call(own=cache(ptr=4104)) == INVALID
    assert call(window=0) == INVALID and call(Hq=7) == INVALID and call(Hq=0) == INVALID
    assert call(Hq=18) == UNSUPPORTED                      # nine query heads per KV head
    assert call(prefix=cache(d=96, S=100), own=cache(d=96)) == UNSUPPORTED
    assert call(own=cache(S=0, W=0)) == INVALID
    assert call(q=None) == INVALID and call(q=BAD) == INVALID and call(out=BAD) == INVALID and call(out=None) == INVALID
    need = nd.nd_shared_prefix_decode_workspace_size(1, 8, 2, 64, 1000, 12)
    assert need > 0
    long = cache(S=1000)
    assert call(long, ws=None) == WORKSPACE and call(long, size=need - 1) == WORKSPACE and call(long, ws=BAD) == WORKSPACE
    assert call(own=cache(B=1 << 22)) == UNSUPPORTED
    assert call(own=cache(B=0)) == OK


def test_shared_prefix_workspace_size_of_bad_arguments_is_zero():
    size = nd.nd_shared_prefix_decode_workspace_size
    assert size(0, 8, 2, 64, 100, 12) == 0 and size(1, 8, 3, 64, 100, 12) == 0 and size(1, 8, 2, 64, 0, 12) == 0
    assert size(1, 8, 2, 64, 100, 0) == 0 and size(1, 0, 2, 64, 100, 12) == 0 and size(1, 8, 2, 0, 100, 12) == 0


def test_qk_norm_rope():
    def call(q=A, k=A, dtype=1, B=2, T=3, Hq=4, Hk=2, d=64, qs=None, ks=None, wq=A, wk=None, eps=1e-6, theta=1e4, pos=None,
             qo=A, ko=A):
        qs, ks = Hq * d if qs is None else qs, Hk * d if ks is None else ks
        return lib().nd_qk_norm_rope(q, k, dtype, B, T, Hq, Hk, d, L(qs), L(ks), wq, wk, F(eps), F(theta), pos, qo, ko, None)

    assert call(dtype=2) == INVALID and call(B=-1) == INVALID and call(T=-1) == INVALID and call(Hq=-1) == INVALID
    assert call(Hk=70000) == INVALID
    assert call(d=48) == INVALID and call(d=0) == INVALID and call(d=96) == UNSUPPORTED and call(d=512) == UNSUPPORTED
    assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID and call(eps=float("inf")) == INVALID
    assert call(theta=-1.0) == INVALID and call(theta=float("nan")) == INVALID and call(theta=float("inf")) == INVALID
    for name in ("q", "k", "qo", "ko"):
        assert call(**{name: BAD}) == INVALID and call(**{name: None}) == INVALID
    assert call(wq=BAD) == INVALID and call(wk=BAD) == INVALID
    assert call(qs=4 * 64 - 8) == INVALID and call(qs=4 * 64 + 4) == INVALID and call(ks=0) == INVALID
    assert call(dtype=0, qs=4 * 64 + 2) == INVALID
    assert call(B=0) == OK and call(T=0) == OK and call(Hq=0, Hk=0, q=None, k=None) == OK


def test_qk_norm_rope_append():
    def call(c=cache(), q=A, k=A, v=A, Hq=4, qs=256, ks=128, vs=128, wq=None, wk=None, eps=1e-6, theta=1e4, sink=0, qo=A):
        return lib().nd_qk_norm_rope_append(q, None if c is None else ctypes.byref(c), k, v, Hq, L(qs), L(ks), L(vs), wq, wk,
                                            F(eps), F(theta), None, sink, qo, None)

    assert call(c=None) == INVALID and call(c=cache(ptr=4104)) == INVALID and call(c=cache(d=48)) == INVALID
    assert call(c=cache(d=96)) == UNSUPPORTED
    assert call(Hq=0) == INVALID and call(Hq=1 << 20) == INVALID
    assert call(c=cache(W=0)) == INVALID and call(c=cache(S=0), sink=1) == INVALID
    for name in ("q", "k", "v", "qo"):
        assert call(**{name: BAD}) == INVALID and call(**{name: None}) == INVALID
    assert call(qs=248) == INVALID and call(ks=127) == INVALID and call(vs=130) == INVALID
    assert call(eps=float("nan")) == INVALID and call(theta=-2.0) == INVALID and call(wq=BAD) == INVALID
    assert call(c=cache(B=0)) == OK


def test_kv_cache_read():
    def call(c=cache(), window=8, dtype=1, rows=12, k=A, v=A):
        return lib().nd_kv_cache_read(None if c is None else ctypes.byref(c), window, dtype, rows, k, v, None, None, None)

    assert call(c=None) == INVALID and call(window=0) == INVALID and call(dtype=3) == INVALID
    assert call(rows=11) == INVALID and call(window=5, rows=8) == INVALID and call(rows=-1) == INVALID
    assert call(c=cache(d=96)) == UNSUPPORTED and call(c=cache(B=70000)) == UNSUPPORTED
    assert call(k=None) == INVALID and call(v=BAD) == INVALID
    assert call(c=cache(B=0)) == OK and call(c=cache(S=0, W=0), rows=0) == OK


def test_the_binding_refuses_host_tensors_and_wrong_shapes():
    t = torch.zeros(1, 3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nd.nd_qk_norm_rope(t, t)
    with pytest.raises(ValueError):
        nd.nd_qk_norm_rope(None, None)
    c = nd.KVCache.empty(1, 2, 64, 4, 8, device="cpu")
    with pytest.raises(ValueError):
        nd.nd_kv_cache_read(c, 8)
    with pytest.raises(ValueError):
        nd.nd_qk_norm_rope_append(t[0, :1], c, t[0, :1, :2], t[0, :1, :2])
    with pytest.raises(ValueError):
        nd.nd_shared_prefix_decode(t[0, :1], c, c, 8)
