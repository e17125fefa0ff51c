"""Rotation at given positions against the formula in 64 bits.

Tolerances.  fp32: the angle is off by 2^-53 |p| turns (p < 2^20: nothing) and an fp32 rounding of half a turn, 9.4e-8
radians (2^-26 of a turn), sine and cosine by sincospif's 2 ulp (2.4e-7 at most below 1), each product by 2^-24 of itself:
|error| <= (9.4e-8 + 2.4e-7 + 2 * 6e-8) * 1.42 max(|a|, |b|) m < 7e-7 * max * m.  bf16 adds its own rounding, 2^-8 of the
value, and of a value below it as much as the fp32 error."""
import math

import numpy as np
import pytest
import torch

from gpu_util import need_gpu, no_device_errors
from workloads import philox

pytestmark = pytest.mark.gpu
F32 = 7e-7


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    no_device_errors()


def nd():
    import sliding_window_kv_swa_gb300 as m
    return m


def frequencies(c, r):
    f = float(np.float32(c.theta)) ** (-2.0 * np.arange(r // 2) / r)
    if c.scaling == "linear":
        return f / c.factor
    if c.scaling == "by_parts":
        g = np.clip((c.orig_len * f / (2 * math.pi) - c.low) / (c.high - c.low), 0, 1)
        return (1 - g) * f / c.factor + g * f
    return f


def formula(x, pos, c):
    d = x.shape[-1]
    r = c.rotary_dim or d
    a = pos.astype(np.float64)[..., None, None] * frequencies(c, r) * (-1 if c.inverse else 1)
    cos, sin = np.cos(a) * c.magnitude, np.sin(a) * c.magnitude
    y = x.astype(np.float64).copy()
    lo, hi = (slice(0, r, 2), slice(1, r, 2)) if c.interleaved else (slice(0, r // 2), slice(r // 2, r))
    y[..., lo] = x[..., lo] * cos - x[..., hi] * sin
    y[..., hi] = x[..., hi] * cos + x[..., lo] * sin
    return y


def check(got, x, pos, c):
    want = formula(x.double().cpu().numpy(), pos, c)
    got_ = got.double().cpu().numpy()
    r = c.rotary_dim or x.shape[-1]
    np.testing.assert_array_equal(got_[..., r:], want[..., r:])
    most = np.abs(want).max() * c.magnitude if want.size else 0
    tol = F32 * most * (1 if x.dtype == torch.float32 else 1.01) + (0 if x.dtype == torch.float32 else np.abs(want) * 2.0 ** -8)
    assert (np.abs(got_ - want) <= tol).all(), np.abs(got_ - want).max()


def make(rng, B, T, heads, d, dtype):
    return torch.from_numpy(rng.standard_normal((B, T, heads, d), dtype=np.float32)).cuda().to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d,r", [(32, 32), (32, 16), (64, 64), (64, 48), (64, 16), (128, 128), (128, 32), (128, 112), (256, 256),
                                 (256, 80)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaling,inverse", [("none", False), ("linear", True), ("by_parts", False), ("by_parts", True)])
def test_against_the_formula(dtype, d, r, interleaved, scaling, inverse):
    rng = philox(21000 + d + r)
    B, T, Hq, Hk = 2, 37, 5, 2
    c = nd().RopeConfig(rotary_dim=r, interleaved=interleaved, scaling=scaling, inverse=inverse, factor=8.0,
                        magnitude=1.0 if scaling == "none" else 1.2079)
    q, k = make(rng, B, T, Hq, d, dtype), make(rng, B, T, Hk, d, dtype)
    pos = rng.integers(0, 100000, (B, T)).astype(np.int32)
    gq, gk = nd().nd_rope_positions(q, k, c, positions=torch.from_numpy(pos).cuda())
    check(gq, q, pos, c)
    check(gk, k, pos, c)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,T,Hq,Hk,d", [(1, 1, 1, 1, 64), (1, 3, 32, 8, 128), (3, 700, 32, 8, 128), (2, 2500, 16, 2, 64), (1, 1500, 70, 3, 32),
                                         (1, 900, 9, 9, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_sizes_in_a_fused_projection(dtype, B, T, Hq, Hk, d, interleaved):
    rng = philox(21100 + T)
    c = nd().RopeConfig(rotary_dim=d // 2, interleaved=interleaved, theta=500000.0)
    x = make(rng, B, T, Hq + 2 * Hk, d, dtype)
    q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
    gq, gk = nd().nd_rope_positions(q, k, c)
    pos = np.tile(np.arange(T), (B, 1))
    check(gq, q, pos, c)
    check(gk, k, pos, c)
    assert gq.is_contiguous() and gk.is_contiguous()


def test_one_side_and_in_place():
    rng = philox(21200)
    for heads in (3, 64):
        q = make(rng, 2, 600, heads, 64, torch.float32)
        c = nd().RopeConfig(rotary_dim=32)
        pos = np.tile(np.arange(600), (2, 1))
        want, none = nd().nd_rope_positions(q, None, c)
        assert none is None
        check(want, q, pos, c)
        assert torch.equal(nd().nd_rope_positions(None, q, c)[1], want)
        kept = q.clone()
        nd().nd_rope_positions(kept, None, c, q_out=kept)
        assert torch.equal(kept, want)


def test_far_and_negative_positions():
    """Near the ends of the int32 range the fp64 frequency's last bit moves the angle by 2^-53 * 2^31 turns, 1.5e-6 rad; the
    formula's own argument p f (up to 2^31 rad) has as much: 2^-53 * 2^31 = 2.4e-7 rad and numpy's f a bit or two, 5e-7."""
    rng = philox(21300)
    pos = np.array([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, -987654321]], np.int32)
    q = make(rng, 1, pos.shape[1], 2, 128, torch.float32)
    for c in (nd().RopeConfig(), nd().RopeConfig(interleaved=True, inverse=True, scaling="linear", factor=32.0)):
        got, _ = nd().nd_rope_positions(q, None, c, positions=torch.from_numpy(pos).cuda())
        want = formula(q.double().cpu().numpy(), pos, c)
        assert np.abs(got.double().cpu().numpy() - want).max() <= (F32 + 2.5e-6) * np.abs(want).max()


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_gradient_is_the_inverse_call(interleaved):
    """<g, R(x + h e) - R(x - h e)> / 2h against the call's gradient: R is linear, so the difference quotient is exact but for
    roundings: each rotation is off by F32 * max |x| per channel, over 2h = 2 with 256 channels' worth of |g| <= 5."""
    rng = philox(21400)
    c = nd().RopeConfig(rotary_dim=48, interleaved=interleaved, scaling="by_parts", factor=4.0, magnitude=1.3)
    back = nd().RopeConfig(rotary_dim=48, interleaved=interleaved, scaling="by_parts", factor=4.0, magnitude=1.3, inverse=True)
    x, g = make(rng, 1, 4, 1, 64, torch.float32), make(rng, 1, 4, 1, 64, torch.float32)
    pos = torch.tensor([[3, 50, 1000, 70000]], dtype=torch.int32, device="cuda")
    turn = lambda t: nd().nd_rope_positions(t, None, c, positions=pos)[0].double()
    grad = nd().nd_rope_positions(g, None, back, positions=pos)[0].double()
    for t in range(4):
        for ch in (0, 1, 23, 24, 25, 47, 48, 63):
            e = torch.zeros_like(x)
            e[0, t, 0, ch] = 1.0
            diff = ((turn(x + e) - turn(x - e)) * g.double()).sum() / 2
            assert abs(float(diff - grad[0, t, 0, ch])) <= 2 * F32 * 7 * 1.3 * 5 * 4, (t, ch)


def test_whole_heads_equal_nd_qk_norm_ropes_rotation():
    """A row of ones times its own norm: the two kernels turn by the same angles, bit for bit."""
    x = torch.ones(1, 50, 4, 128, device="cuda")
    x[..., 1::2] = -1.0                                    # mean square 1: the norm (eps 0) leaves it
    a, _ = nd().nd_qk_norm_rope(x, None, eps=0.0, rope_theta=10000.0)
    b, _ = nd().nd_rope_positions(x, None, nd().RopeConfig())
    assert torch.equal(a, b)


def test_non_finite_channels_stay_in_their_pair():
    x = torch.zeros(1, 2, 1, 64, device="cuda")
    x[0, 1, 0, 3], x[0, 1, 0, 40] = float("inf"), float("nan")
    y, _ = nd().nd_rope_positions(x, None, nd().RopeConfig(rotary_dim=32))
    bad = {i for i in range(64) if not math.isfinite(float(y[0, 1, 0, i]))}
    assert bad == {3, 19, 40} and torch.isfinite(y[0, 0]).all()
