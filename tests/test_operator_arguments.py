"""Arguments of the operators' C entry points at the edges of what the header
allows.  Every call is refused or has nothing to do, so nothing is launched."""
import ctypes

import sliding_window_kv_swa_gb300 as nd

OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = range(5)
P, F, L = ctypes.c_void_p, ctypes.c_float, ctypes.c_int64
A, BAD = P(4096), P(4104)   # aligned and misaligned addresses; nothing is read


def lib():
    return nd.nd._lib()


def test_a_side_without_heads_has_no_weight_either():
    def call(Hq=4, Hk=2, wq=A, wk=A, B=0):
        return lib().nd_qk_norm_rope(A, A, 1, B, 3, Hq, Hk, 64, L(Hq * 64), L(Hk * 64), wq, wk, F(1e-6), F(1e4), None, A, A, None)

    assert call(Hk=0, wk=BAD) == OK and call(Hq=0, wq=BAD) == OK and call(Hq=0, Hk=0, wq=BAD, wk=BAD) == OK
    assert call(wk=BAD) == INVALID and call(wq=BAD) == INVALID
    assert call(Hk=0, wq=BAD) == INVALID and call(Hq=0, wk=BAD) == INVALID


def cache(B=1, Hkv=2, d=64, S=4, W=8):
    return nd.nd._Cache(B, Hkv, d, S, W, *([4096] * 8))


TOP = 2 ** 31 - 1


def test_regions_at_the_end_of_the_int_range_are_refused():
    def call(prefix, own):
        return lib().nd_shared_prefix_decode(A, ctypes.byref(prefix), ctypes.byref(own), 8, 8, A, None, A,
                                             ctypes.c_size_t(1 << 62), None)

    for many in (cache(S=TOP, W=0), cache(S=TOP - 63, W=0), cache(S=1 << 30, W=1 << 30)):
        assert call(many, cache()) == UNSUPPORTED
    for many in (cache(S=TOP, W=0), cache(S=TOP - 15, W=0), cache(S=1 << 30, W=1 << 30), cache(S=TOP, W=TOP)):
        assert call(cache(S=600), many) == UNSUPPORTED
    size = nd.nd_shared_prefix_decode_workspace_size
    assert size(1, 8, 2, 64, TOP, 12) == 0 and size(1, 8, 2, 64, 600, TOP) == 0


def test_heads_past_what_an_append_takes_are_refused():
    def call(Hkv):
        return lib().nd_qk_norm_rope_append(A, ctypes.byref(cache(Hkv=Hkv)), A, A, 4, L(256), L(Hkv * 64), L(Hkv * 64), None,
                                            None, F(1e-6), F(1e4), None, 0, A, None)

    assert call(1 << 17) == INVALID and call(TOP) == INVALID
