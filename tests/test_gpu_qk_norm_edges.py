"""The per-head norm with rotation where one side is absent, and the rotation's
angles by themselves."""
import numpy as np
import pytest
import torch

from gpu_util import dev, dev_bf16, need_gpu, no_device_errors
from workloads import normal_bf16, philox

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    no_device_errors()


def nd():
    import sliding_window_kv_swa_gb300 as m
    return m


@pytest.mark.parametrize("B,T", [(1, 3), (3, 433)])   # rows in a line; a warp to a token
def test_weights_of_a_side_that_is_absent(B, T):
    """Both weights are given, one side has no heads: its weight changes nothing, also where it is not aligned."""
    rng = philox(9250 + T)
    q = dev_bf16(normal_bf16(rng, (B, T, 13, 64))[0])
    wq, wk = (dev(rng.uniform(0.5, 1.5, 64).astype(np.float32)) for _ in range(2))
    odd = torch.full((65,), float("nan"), device="cuda")[1:]
    both_q, both_k = nd().nd_qk_norm_rope(q, q, wq, wk, 1e-6, 10000.0)
    for other in (wk, odd):
        one, none = nd().nd_qk_norm_rope(q, None, wq, other, 1e-6, 10000.0)
        assert none is None and torch.equal(one, both_q)
        none, one = nd().nd_qk_norm_rope(None, q, other, wk, 1e-6, 10000.0)
        assert none is None and torch.equal(one, both_k)


@pytest.mark.parametrize("d,theta", [(32, 10000.0), (128, 500000.0), (256, 2.0)])
def test_angles(d, theta):
    """A row of ones and zeros comes out as r (cos a, sin a).  The angle is rounded to fp32 in half turns, 24 bits of up
    to one: 2 pi 2^-26 off; its frequency by 2^-49 of the position; sine and cosine by 2 ulp, 2^-22; the norm's 17
    additions at D = 256, halved by the root, the root's and the two products' roundings, 12 of 2^-24.  Angles just
    beside half a turn, where the first of these is largest, are sought out among the positions."""
    rng = philox(9260 + d)
    top = 1 << 22
    freq = np.float64(theta) ** (-2.0 * np.arange(d // 2) / d)
    pos = rng.integers(-top, top, 200000)
    half = np.abs(np.abs(np.remainder(pos[:, None] * freq[:4] / (2 * np.pi), 1.0)) - 0.5).min(1)
    pos = np.concatenate([pos[np.argsort(half)[:1000]], pos[:1000], [0, 1, -1, top]]).astype(np.int32)
    x = torch.zeros(1, len(pos), 1, d, device="cuda")
    x[..., : d // 2] = 1.0
    _, y = nd().nd_qk_norm_rope(None, x, eps=0.0, rope_theta=theta, positions=dev(pos[None]))
    a = pos.astype(np.float64)[:, None] * freq
    want = np.concatenate([np.cos(a), np.sin(a)], -1) * np.sqrt(2.0)
    err = np.abs(y[0, :, 0].double().cpu().numpy() - want)
    assert err.max() <= np.sqrt(2.0) * (2 * np.pi * 2.0 ** -26 + top * 2.0 ** -49 + 2.0 ** -22 + 12 * 2.0 ** -24), err.max()
