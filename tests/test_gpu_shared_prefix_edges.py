"""Shared-prefix decode where the rest of the suite does not look: groups of
query heads that lie across two row pairs of the prefix kernel.  Tolerances as
in test_gpu_shared_prefix.py."""
import pytest
import torch

from gpu_util import dev_bf16, host, need_gpu, no_device_errors
from test_gpu_shared_prefix import check, device_cache, nd, random_cache
from workloads import normal_bf16, philox

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    no_device_errors()


@pytest.mark.parametrize("Hq,Hkv,d,L", [(48, 8, 64, 600), (56, 8, 64, 200), (30, 5, 128, 600)])
def test_a_group_whose_heads_have_different_numbers_of_partials(Hq, Hkv, d, L):
    """Six or seven heads a group: some sequences' heads fall into two 256-row pairs, whose tiles lie in different
    numbers of CTAs, and the units of the last round are walked by the four warps of a CTA together.  The same bits
    every time."""
    rng = philox(11000 + Hq + L)
    B, W = 450, 40
    prefix = random_cache(rng, 1, Hkv, d, 600, 0, [(L, 0)])
    own = random_cache(rng, B, Hkv, d, 0, W, [(0, 2 * W), (0, 7), (0, 0), (0, W)])
    qb, q = normal_bf16(rng, (B, Hq, d))
    check(prefix, own, qb, q, W)
    p, c, qd = device_cache(prefix), device_cache(own), dev_bf16(qb)
    ws = torch.empty(nd().nd_shared_prefix_decode_workspace_size(B, Hq, Hkv, d, 600, W), dtype=torch.uint8, device="cuda")
    first = host(nd().nd_shared_prefix_decode(qd, p, c, W, workspace=ws))
    for _ in range(20):
        assert (host(nd().nd_shared_prefix_decode(qd, p, c, W, workspace=ws)) == first).all()
