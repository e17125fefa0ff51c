"""The per-head norm with rotation where one side is absent.  Results are compared bit for bit with the
same side's in a call that has both."""
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
