"""GPU parity of the per-head RMS norm with rotation (prefill form and decode
append) against the formula in 64 bits.

Tolerances, from the roundings: a channel's fp32 value passes the sum of D
squares (at most D/16 additions in a lane and four across lanes; halved by the
square root), the reciprocal root, two products, the sine and cosine (2 ulp
each) and the rotation: below 16 roundings of 2^-24 each, so 2^-20 of the row's
largest magnitude.  A bf16 output adds half a step, 2^-8 of its value."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, dev_bf16, host, need_gpu, no_device_errors
from workloads import bf16_bits_to_f32, normal_bf16, philox, to_bf16_bits

pytestmark = pytest.mark.gpu

FIELDS = ("k_codes", "v_codes", "k_scale", "v_scale", "sink_len", "ring_start", "ring_len", "seq_len")


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    no_device_errors()


def nd():
    import sliding_window_kv_swa_gb300 as m
    return m


def formula(x, w, pos, eps, theta):
    """x [..., H, d], pos [...]: the norm and the rotation in fp64."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * np.asarray(w, np.float64)
    if theta == 0:
        return y
    freq = np.float64(theta) ** (-2.0 * np.arange(d // 2) / d)
    a = np.asarray(pos, np.float64)[..., None, None] * freq
    lo, hi = y[..., : d // 2], y[..., d // 2:]
    return np.concatenate([lo * np.cos(a) - hi * np.sin(a), hi * np.cos(a) + lo * np.sin(a)], -1)


def check(got, want, bf16, extra=0.0, what=""):
    top = np.abs(want).max(-1, keepdims=True)
    tol = (2.0 ** -20 + extra) * top + (2.0 ** -8 * np.abs(want) if bf16 else 0.0)
    bad = np.abs(got - want) > tol
    assert not bad.any(), f"{what}: {bad.sum()} channels off, worst {np.abs(got - want).max():.3e}"


def draw(rng, shape, f32):
    if f32:
        x = rng.standard_normal(shape, dtype=np.float32)
        return dev(x), x
    bits, x = normal_bf16(rng, shape)
    return dev_bf16(bits), x


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hk", [(1, 1, 1, 1), (2, 7, 4, 1), (3, 33, 5, 3), (1, 130, 32, 8)])
def test_norm_rope_matches_the_formula(d, f32, B, T, Hq, Hk):
    rng = philox(9000 + d + T)
    q, qf = draw(rng, (B, T, Hq, d), f32)
    k, kf = draw(rng, (B, T, Hk, d), f32)
    wq, wk = (rng.uniform(0.5, 1.5, d).astype(np.float32) for _ in range(2))
    qo, ko = nd().nd_qk_norm_rope(q, k, dev(wq), dev(wk), 1e-6, 10000.0)
    pos = np.broadcast_to(np.arange(T), (B, T))
    check(host(qo), formula(qf, wq, pos, 1e-6, 10000.0), not f32, what="q")
    check(host(ko), formula(kf, wk, pos, 1e-6, 10000.0), not f32, what="k")


@pytest.mark.parametrize("d,Hq,Hk", [(32, 33, 4), (64, 13, 4), (128, 7, 2), (256, 3, 2)])
@pytest.mark.parametrize("f32", [False, True])
def test_many_tokens(d, Hq, Hk, f32):
    """Enough rows that a warp takes a token; heads that do not fill its last batch; slices, positions, in place."""
    rng = philox(9050 + d)
    B, T = 3, 433
    x, xf = draw(rng, (B, T, Hq + Hk + 1, d), f32)
    q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
    wq, wk = (rng.uniform(0.5, 1.5, d).astype(np.float32) for _ in range(2))
    pos = rng.integers(-5, 100000, (B, T)).astype(np.int32)
    qo, ko = nd().nd_qk_norm_rope(q, k, dev(wq), dev(wk), 1e-6, 10000.0, positions=dev(pos))
    far = 1e5 * 2.0 ** -49
    check(host(qo), formula(xf[:, :, :Hq], wq, pos, 1e-6, 10000.0), not f32, far, "q")
    check(host(ko), formula(xf[:, :, Hq:Hq + Hk], wk, pos, 1e-6, 10000.0), not f32, far, "k")
    qc, kc = q.contiguous(), k.contiguous()
    nd().nd_qk_norm_rope(qc, kc, dev(wq), dev(wk), 1e-6, 10000.0, positions=dev(pos), q_out=qc, k_out=kc)
    assert torch.equal(qc, qo) and torch.equal(kc, ko)
    _, k2 = nd().nd_qk_norm_rope(None, q, None, dev(wq), 1e-6, 10000.0, positions=dev(pos))
    assert torch.equal(k2, qo)


def test_without_weights_without_rotation_and_one_tensor():
    rng = philox(9100)
    q, qf = draw(rng, (2, 5, 3, 64), False)
    qo, none = nd().nd_qk_norm_rope(q, None, eps=0.5)
    assert none is None
    check(host(qo), formula(qf, None, None, 0.5, 0), True)
    none, ko = nd().nd_qk_norm_rope(None, q, eps=0.5, rope_theta=500000.0)
    check(host(ko), formula(qf, None, np.broadcast_to(np.arange(5), (2, 5)), 0.5, 500000.0), True)


def test_zero_rows_large_and_small_values():
    """eps keeps a zero row 0; values near the ends of bf16's range keep their norm (squares stay in fp32)."""
    x = np.ones((1, 4, 1, 64), np.float32)
    x[0, 0] = 0.0
    x[0, 1] *= 2.0 ** 55
    x[0, 2] *= 2.0 ** -60
    bits = to_bf16_bits(x)
    qo, _ = nd().nd_qk_norm_rope(dev_bf16(bits), None, eps=1e-6)
    got = host(qo)
    assert (got[0, 0] == 0).all()
    check(got, formula(bf16_bits_to_f32(bits), None, None, 1e-6, 0), True)
    qo, _ = nd().nd_qk_norm_rope(dev_bf16(bits[:, 3:]), None, eps=0.0)
    check(host(qo), formula(bf16_bits_to_f32(bits[:, 3:]), None, None, 0.0, 0), True)


@pytest.mark.parametrize("top", [1 << 20, 1 << 24, (1 << 31) - 1])
def test_far_and_negative_positions(top):
    """The angle of a far position: the frequency in turns has 53 bits (2 pi 2^-53 < 2^-50 radians per position), the
    frequency and the product here another 2^-52 and 2^-53: below 2^-49 per position."""
    rng = philox(9200)
    B, T = 2, 19
    pos = rng.integers(-top, top, (B, T)).astype(np.int32)
    pos[0, :3] = (top, -top, 0)
    k, kf = draw(rng, (B, T, 2, 128), True)
    _, ko = nd().nd_qk_norm_rope(None, k, eps=1e-6, rope_theta=10000.0, positions=dev(pos))
    check(host(ko), formula(kf, None, pos, 1e-6, 10000.0), False, extra=top * 2.0 ** -49)


def test_slices_of_a_fused_projection_and_in_place():
    rng = philox(9300)
    B, T, Hq, Hk, d = 2, 21, 8, 2, 64
    x, xf = draw(rng, (B, T, Hq + 2 * Hk, d), False)
    keep = x.clone()
    q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
    qo, ko = nd().nd_qk_norm_rope(q, k, eps=1e-6, rope_theta=10000.0)
    assert torch.equal(x, keep) and qo.is_contiguous() and ko.is_contiguous()
    q2, k2 = nd().nd_qk_norm_rope(q.contiguous(), k.contiguous(), eps=1e-6, rope_theta=10000.0)
    assert torch.equal(qo, q2) and torch.equal(ko, k2)
    qc, kc = q.contiguous(), k.contiguous()
    nd().nd_qk_norm_rope(qc, kc, eps=1e-6, rope_theta=10000.0, q_out=qc, k_out=kc)
    assert torch.equal(qc, q2) and torch.equal(kc, k2)
    # one row of the batch, one token: strides of what is not there do not matter
    qo, _ = nd().nd_qk_norm_rope(q[:1, 3:4], None, eps=1e-6)
    want, _ = nd().nd_qk_norm_rope(q[:1, 3:4].contiguous(), None, eps=1e-6)
    assert torch.equal(qo, want)
    qo, _ = nd().nd_qk_norm_rope(q[:, 3:4], None, eps=1e-6)
    want, _ = nd().nd_qk_norm_rope(q[:, 3:4].contiguous(), None, eps=1e-6)
    assert torch.equal(qo, want)


def make_cache(B, Hkv, d, S, W):
    return nd().KVCache.empty(B, Hkv, d, S, W)


@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("B,Hq,Hkv", [(1, 1, 1), (5, 8, 2), (3, 48, 16)])
def test_append_equals_norm_rope_then_append(d, B, Hq, Hkv):
    """Bit for bit, through sinks, a filling ring and its wraps; and the query against the formula."""
    S, W, theta = 3, 4, 10000.0
    rng = philox(9400 + d)
    one, two = make_cache(B, Hkv, d, S, W), make_cache(B, Hkv, d, S, W)
    wq, wk = (dev(rng.uniform(0.5, 1.5, d).astype(np.float32)) for _ in range(2))
    base = torch.tensor([12345], dtype=torch.int32, device="cuda")
    for step in range(S + 2 * W + 1):
        x, xf = draw(rng, (B, Hq + 2 * Hkv, d), False)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        qo = nd().nd_qk_norm_rope_append(q, one, k, v, wq, wk, 1e-6, theta, pos_base=base, to_sink=step < S)
        pos = torch.full((B, 1), 12345 + step, dtype=torch.int32, device="cuda")
        q2, k2 = nd().nd_qk_norm_rope(q[:, None], k[:, None], wq, wk, 1e-6, theta, positions=pos)
        nd().nd_kv_append_quant(two, k2[:, 0].contiguous(), v.contiguous(), step < S)
        for f in FIELDS:
            assert torch.equal(getattr(one, f), getattr(two, f)), (f, step)
        assert torch.equal(qo, q2[:, 0])
        check(host(qo), formula(xf[:, :Hq], host(wq), np.full(B, 12345 + step), 1e-6, theta), True)


def test_append_without_base_weights_or_rotation_is_the_plain_append_of_normalised_keys():
    rng = philox(9500)
    cache = make_cache(2, 1, 64, 0, 2)
    x, xf = draw(rng, (2, 1, 64), False)
    nd().nd_qk_norm_rope_append(x, cache, x, x)
    ref = oracle.Cache(2, 1, 64, 0, 2)
    _, k2 = nd().nd_qk_norm_rope(None, x[:, None])
    oracle.kv_append(ref, host(k2[:, 0]).astype(np.float32), xf, False)
    for f in FIELDS:
        np.testing.assert_array_equal(host(getattr(cache, f)), getattr(ref, f))


def test_rejected_sink_append_and_bad_metadata_write_nothing():
    rng = philox(9600)
    cache = make_cache(3, 1, 64, 2, 4)
    cache.ring_len[0] = 1          # a ring token came first: a sink append is rejected
    cache.sink_len[1] = 7          # out of range
    x, _ = draw(rng, (3, 1, 64), False)
    q_out = torch.full((3, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    nd().nd_qk_norm_rope_append(x, cache, x, x, to_sink=True, q_out=q_out)
    torch.cuda.synchronize()
    assert nd().nd_device_errors(clear=True) == 2
    assert (q_out[:2] == 5.0).all() and not (q_out[2] == 5.0).any()
    assert (cache.k_codes[:2] == 0).all() and (cache.k_codes[2, :, 0] != 0).any()
    np.testing.assert_array_equal(host(cache.seq_len), [0, 0, 1])
    np.testing.assert_array_equal(host(cache.sink_len), [0, 7, 1])


def test_captured_and_on_another_stream():
    rng = philox(9700)
    cache, same = make_cache(4, 2, 64, 0, 8), make_cache(4, 2, 64, 0, 8)
    x, _ = draw(rng, (4, 8 + 4, 64), False)
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    out = torch.empty(4, 8, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        nd().nd_qk_norm_rope_append(q, same, k, v, rope_theta=10000.0, q_out=out)
    s.synchronize()
    want = [out.clone()]
    for _ in range(2):
        nd().nd_qk_norm_rope_append(q, same, k, v, rope_theta=10000.0, q_out=out)
        want.append(out.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nd().nd_qk_norm_rope_append(q, cache, k, v, rope_theta=10000.0, q_out=out)
    for w in want:
        g.replay()
        assert torch.equal(out, w)
    for f in FIELDS:
        assert torch.equal(getattr(cache, f), getattr(same, f)), f
