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
