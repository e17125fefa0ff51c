"""Refusals of the tree operators and of the rotation at positions: every bad
argument is answered on the host, with the status the header gives, before
anything is enqueued (no GPU is needed); and what the binding makes."""
import contextlib
import copy
import ctypes
import os
import pickle
import subprocess
import sys

import pytest
import torch

import sliding_window_kv_swa_gb300 as nd

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, CUDA, WORKSPACE = range(5)
P, Z, F, L = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float, ctypes.c_int64
A, BAD = P(4096), P(4104)   # aligned and misaligned addresses; nothing is read


def cache(B=1, Hkv=2, d=64, S=4, W=8, ptr=4096):
    return nd.nd._Cache(B, Hkv, d, S, W, *([ptr] * 8))


def lib():
    return nd.nd._lib()


def test_tree_layout():
    def call(parents=A, B=2, n=5, window=4, depth=A, mask=A):
        return lib().nd_tree_layout(parents, None, None, None, B, n, window, depth, None, mask, None)

    assert call(B=-1) == INVALID and call(n=-1) == INVALID and call(window=0) == INVALID
    assert call(n=257) == UNSUPPORTED and call(B=(1 << 24) + 1) == UNSUPPORTED
    assert call(parents=None) == INVALID and call(depth=None) == INVALID and call(mask=None) == INVALID
    assert call(B=0) == OK and call(n=0) == OK


def test_tree_accept():
    def call(parents=A, tokens=A, target=A, B=2, n=5, m=3, path=A, length=A):
        return lib().nd_tree_accept(parents, None, tokens, target, None, B, n, m, path, length, None, None)

    assert call(B=-1) == INVALID and call(n=-1) == INVALID and call(m=0) == INVALID
    assert call(n=257) == UNSUPPORTED and call(B=(1 << 24) + 1) == UNSUPPORTED
    assert call(m=65537) == UNSUPPORTED
    for name in ("parents", "tokens", "target", "path", "length"):
        assert call(**{name: None}) == INVALID
    assert call(B=0) == OK


def test_tree_commit():
    def call(c=cache(), k=A, v=A, ks=128, vs=128, n=5, path=A, length=A, m=3):
        return lib().nd_tree_commit(None if c is None else ctypes.byref(c), k, v, L(ks), L(vs), n, path, length, m, None)

    assert call(c=None) == INVALID and call(c=cache(ptr=4104)) == INVALID and call(c=cache(d=48)) == INVALID
    assert call(c=cache(W=0)) == INVALID and call(c=cache(d=96)) == UNSUPPORTED
    assert call(m=65537) == UNSUPPORTED and call(c=cache(Hkv=16384), m=65536, ks=1 << 20, vs=1 << 20) == UNSUPPORTED
    assert call(n=-1) == INVALID and call(n=257) == UNSUPPORTED and call(m=0) == INVALID
    for name in ("k", "v"):
        assert call(**{name: BAD}) == INVALID and call(**{name: None}) == INVALID
    assert call(path=None) == INVALID and call(length=None) == INVALID
    assert call(ks=120) == INVALID and call(vs=132) == INVALID and call(ks=-128) == INVALID
    assert call(c=cache(B=0)) == OK


def test_tree_decode():
    def call(c=cache(), q=A, k=A, v=A, ks=128, vs=128, depth=A, mask=A, n=5, Hq=8, window=8, out=A, ws=A, size=1 << 40):
        return lib().nd_tree_decode(q, None if c is None else ctypes.byref(c), k, v, L(ks), L(vs), depth, mask, n, Hq, window, out, None,
                                    ws, Z(size), None)

    assert call(c=None) == INVALID and call(c=cache(ptr=4104)) == INVALID and call(c=cache(d=48)) == INVALID
    assert call(c=cache(d=32)) == UNSUPPORTED and call(c=cache(d=256)) == UNSUPPORTED
    assert call(n=-1) == INVALID and call(n=257) == UNSUPPORTED and call(window=0) == INVALID
    assert call(Hq=7) == INVALID and call(Hq=0) == INVALID and call(Hq=18) == UNSUPPORTED
    for name in ("q", "k", "v", "out"):
        assert call(**{name: BAD}) == INVALID and call(**{name: None}) == INVALID
    assert call(depth=None) == INVALID and call(mask=None) == INVALID
    assert call(ks=120) == INVALID and call(vs=132) == INVALID and call(ks=-128) == INVALID
    assert call(c=cache(B=(1 << 19) + 1)) == UNSUPPORTED and call(c=cache(S=0, W=0)) == INVALID
    assert call(c=cache(S=2 ** 31 - 4097, W=2)) == UNSUPPORTED
    assert call(c=cache(B=0)) == OK and call(n=0) == OK
    need = nd.nd_tree_decode_workspace_size(1, 64, 8, 2, 64, 20000)
    if need:
        long = cache(S=20000, W=0)
        assert call(long, n=64, ws=None) == WORKSPACE and call(long, n=64, size=need - 1) == WORKSPACE and \
            call(long, n=64, ws=BAD) == WORKSPACE


def test_tree_decode_workspace_size_of_bad_arguments_is_zero():
    size = nd.nd_tree_decode_workspace_size
    assert size(0, 4, 8, 2, 64, 100) == 0 and size(1, 0, 8, 2, 64, 100) == 0 and size(1, 4, 8, 3, 64, 100) == 0
    assert size(1, 257, 8, 2, 64, 100) == 0 and size(1, 4, 0, 2, 64, 100) == 0 and size(1, 4, 8, 0, 64, 100) == 0
    assert size(1, 4, 8, 2, 0, 100) == 0 and size(1, 4, 8, 2, 64, 0) == 0


def test_tree_decode_refuses_what_the_workspace_size_is_no_answer_for():
    # 153 pairs of as many slots as leave 2^30 tiles: one region takes a tile less than the query allows for
    pairs, per = 153, (1 << 30) // 153
    W = (per - 1) * 128                     # and a tile of nodes: 153 * per < 2^30 <= 153 * (per + 1)
    assert pairs * per < 1 << 30 <= pairs * (per + 1) and W < 2 ** 31 - 4096
    assert nd.nd_tree_decode_workspace_size(pairs, 1, 1, 1, 64, W) == 0
    c = cache(B=pairs, Hkv=1, S=0, W=W)
    st = lib().nd_tree_decode(A, ctypes.byref(c), A, A, L(64), L(64), A, A, 1, 1, 8, A, None, None, Z(0), None)
    assert st == UNSUPPORTED
    assert nd.nd_tree_decode_workspace_size(pairs, 1, 1, 1, 64, W - 128) > 0


REFUSED_SHAPES = [(256, 80, 1, 64), (256, 128, 1, 128), (1, 9, 1, 64), (64, 18, 2, 128), (2, 2 ** 30, 1, 64), (5, 8, 2, 32),
                  (5, 8, 2, 96), (5, 8, 2, 256), (5, 8, 2, 2 ** 31 - 1)]    # n, Hq, Hkv, d


def test_tree_decode_workspace_size_of_refused_shapes_is_zero():
    # in a process of its own: a division by the CTAs that such groups leave (none) ends it
    code = f"import sliding_window_kv_swa_gb300 as nd; print([nd.nd_tree_decode_workspace_size(1, *s, 20000) for s in {REFUSED_SHAPES}])"
    done = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert done.returncode == 0 and done.stdout.strip() == str([0] * len(REFUSED_SHAPES)), (done.returncode, done.stdout, done.stderr)
    for n, Hq, Hkv, d in REFUSED_SHAPES[:-1]:
        c = cache(Hkv=Hkv, d=d, S=20000, W=0)
        st = lib().nd_tree_decode(A, ctypes.byref(c), A, A, L(Hkv * d), L(Hkv * d), A, A, n, Hq, 8, A, None, None, Z(0), None)
        assert st == UNSUPPORTED, (n, Hq, Hkv, d)


def rope_cfg(r=64, inter=0, inv=0, scaling=0, theta=1e4, factor=4.0, low=1.0, high=32.0, orig=4096.0, mag=1.0):
    return nd.nd._RopeCfg(r, inter, inv, scaling, theta, factor, low, high, orig, mag)


def test_rope_positions():
    def call(c=rope_cfg(), q=A, k=A, dtype=1, B=2, T=3, Hq=4, Hk=2, d=64, qs=None, ks=None, qo=A, ko=A):
        qs, ks = Hq * d if qs is None else qs, Hk * d if ks is None else ks
        return lib().nd_rope_positions(q, k, dtype, B, T, Hq, Hk, d, L(qs), L(ks), None if c is None else ctypes.byref(c), None, qo, ko,
                                       None)

    nan, inf = float("nan"), float("inf")
    assert call(c=None) == INVALID and call(dtype=2) == INVALID and call(B=-1) == INVALID and call(T=-1) == INVALID
    assert call(Hq=-1) == INVALID and call(Hk=70000) == INVALID
    assert call(d=48) == INVALID and call(d=0) == INVALID and call(d=96) == UNSUPPORTED and call(d=512) == UNSUPPORTED
    for bad in (dict(r=0), dict(r=-16), dict(r=80), dict(inter=2), dict(inv=-1), dict(scaling=3), dict(scaling=-1), dict(theta=0.0),
                dict(theta=nan), dict(theta=inf), dict(mag=0.0), dict(mag=-1.0), dict(mag=nan), dict(scaling=1, factor=0.0),
                dict(scaling=1, factor=nan), dict(scaling=2, factor=-1.0), dict(scaling=2, low=32.0), dict(scaling=2, low=-1.0),
                dict(scaling=2, high=nan), dict(scaling=2, high=inf), dict(scaling=2, orig=0.0), dict(scaling=2, orig=nan)):
        assert call(c=rope_cfg(**bad)) == INVALID, bad
    assert call(c=rope_cfg(r=24)) == UNSUPPORTED and call(c=rope_cfg(r=8)) == UNSUPPORTED
    assert call(c=rope_cfg(factor=nan, low=5.0, high=2.0, orig=-1.0), B=0) == OK   # fields that the scaling does not use
    for name in ("q", "k", "qo", "ko"):
        assert call(**{name: BAD}) == INVALID and call(**{name: None}) == INVALID
    assert call(qs=4 * 64 - 8) == INVALID and call(qs=4 * 64 + 4) == INVALID and call(ks=0) == INVALID
    assert call(dtype=0, qs=4 * 64 + 2) == INVALID
    assert call(B=0) == OK and call(T=0) == OK and call(Hq=0, Hk=0, q=None, k=None) == OK
    assert call(B=1 << 16, T=1 << 15) == UNSUPPORTED


def test_rope_positions_takes_every_finite_value():
    def call(**kw):
        return lib().nd_rope_positions(A, A, 1, 0, 3, 4, 2, 64, L(256), L(128), ctypes.byref(rope_cfg(**kw)), None, A, A, None)

    for x in (1e-45, 1e30, 3.4e38):
        for kw in (dict(theta=x), dict(mag=x), dict(scaling=1, factor=x), dict(scaling=2, factor=x), dict(scaling=2, orig=x)):
            assert call(**kw) == OK, kw
    assert call(scaling=2, high=1e30) == OK and call(scaling=2, low=1e30, high=3.4e38) == OK
    assert call(scaling=2, high=float("inf")) == INVALID and call(theta=float("inf")) == INVALID and call(mag=float("nan")) == INVALID


def test_the_binding_refuses_host_tensors_and_wrong_shapes():
    i = torch.zeros(1, 3, dtype=torch.int32)
    x = torch.zeros(1, 3, 2, 64, dtype=torch.bfloat16)
    c = nd.KVCache.empty(1, 2, 64, 4, 8, device="cpu")
    for call in (lambda: nd.nd_tree_layout(i, None, 4), lambda: nd.nd_tree_accept(i, i, i, 2),
                 lambda: nd.nd_tree_commit(c, x, x, i, i[:, 0]), lambda: nd.nd_tree_decode(x, c, x, x, i, i[:, :, None], 4),
                 lambda: nd.nd_rope_positions(x, x), lambda: nd.nd_rope_positions(None, None),
                 lambda: nd.RopeConfig(scaling="other").struct(64)):
        with pytest.raises(ValueError):
            call()


class FakeLibrary:
    """Sizes are 4096, statuses ND_OK; nothing is launched."""
    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("_size") else 0


class OtherStream(torch.cuda.Stream if torch.cuda.is_available() else object):
    cuda_stream = 77


@pytest.fixture
def on_the_host(monkeypatch):
    monkeypatch.setattr(nd.nd, "_lib", lambda: FakeLibrary())
    monkeypatch.setattr(nd.nd, "_here", lambda t: t.get_device())
    monkeypatch.setattr(nd.nd, "_on", lambda stream, dev: 0)


def calls(**kw):
    i = torch.zeros(2, 3, dtype=torch.int32)
    x = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    c = nd.KVCache.empty(2, 2, 64, 4, 8, device="cpu")
    return {"layout": lambda: nd.nd_tree_layout(i, None, 4, **kw), "accept": lambda: nd.nd_tree_accept(i, i, i, 2, **kw),
            "decode": lambda: nd.nd_tree_decode(x, c, x, x, i, i[:, :, None].contiguous(), 4, **kw),
            "rope": lambda: nd.nd_rope_positions(x, x, **kw)}


@pytest.mark.parametrize("name", sorted(calls()))
def test_what_a_call_makes_belongs_to_the_stream_it_runs_on(name, on_the_host, monkeypatch):
    stream, inside, made = OtherStream.__new__(OtherStream), [], []

    @contextlib.contextmanager
    def pool(s):
        inside.append(s)
        yield
        inside.pop()

    monkeypatch.setattr(nd.nd, "_pool", pool)
    for fn in ("empty", "empty_like"):
        real = getattr(torch, fn)
        monkeypatch.setattr(torch, fn, lambda *a, _real=real, **k: (made.append(list(inside)), _real(*a, **k))[1])
    calls(stream=stream)[name]()
    assert made and all(m == [stream] for m in made)


def test_the_binding_refuses_tensors_that_do_not_fit(on_the_host):
    i = torch.zeros(2, 3, dtype=torch.int32)
    x = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16)
    c = nd.KVCache.empty(2, 2, 64, 4, 8, device="cpu")
    mask = torch.zeros(2, 3, 1, dtype=torch.int32)
    nd.nd_tree_decode(x, c, x, x, i, mask, 4)
    for bad in (dict(depth=i[:, :2]), dict(mask=mask[:, :, 0]), dict(mask=mask.long()), dict(k_new=x[:, :2]), dict(v_new=x.float()),
                dict(q=x[:1]), dict(q=x.transpose(0, 1)), dict(out=x[:, :2])):
        args = dict(q=x, cache=c, k_new=x, v_new=x, depth=i, mask=mask, window=4) | bad
        with pytest.raises(ValueError):
            nd.nd_tree_decode(**args)
    for call in (lambda: nd.nd_tree_layout(i[0], None, 4), lambda: nd.nd_tree_layout(i, i, 4), lambda: nd.nd_tree_layout(i.long(), None, 4),
                 lambda: nd.nd_tree_accept(i, i[:, :2], i, 2), lambda: nd.nd_tree_accept(i, i, i, 0),
                 lambda: nd.nd_tree_commit(c, x, x, i[:1], i[:, 0].contiguous()), lambda: nd.nd_tree_commit(c, x, x, i, i),
                 lambda: nd.nd_tree_commit(c, x[:, :, :1], x[:, :, :1], i, i[:, 0].contiguous()),
                 lambda: nd.nd_rope_positions(x, x, positions=i.long()), lambda: nd.nd_rope_positions(x, x.float())):
        with pytest.raises(ValueError):
            call()


def test_a_rope_config_can_be_copied_and_pickled_after_a_call():
    c = nd.RopeConfig(rotary_dim=32, scaling="linear", factor=2.0)
    assert c.struct_ref(64) is c.struct_ref(64)
    assert copy.deepcopy(c) == c and pickle.loads(pickle.dumps(c)) == c
