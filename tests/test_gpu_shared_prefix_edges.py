"""Shared-prefix decode where the rest of the suite does not look: groups of
query heads that lie across two row pairs of the prefix kernel, calls on a
stream that is not the current one, scores that vanish, queries that are not
finite, values far smaller than others.  Tolerances as in
test_gpu_shared_prefix.py where nothing else is said."""
import math

import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev_bf16, host, need_gpu, no_device_errors
from test_gpu_shared_prefix import check, device_cache, joined, nd, random_cache, run
from workloads import normal_bf16, philox, to_bf16_bits

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


def test_a_call_on_another_stream_keeps_its_workspace():
    """The call's stream is held up behind a timed wait; meanwhile the current stream asks for memory of every size
    that the call used, and fills it."""
    rng = philox(11100)
    Hq, Hkv, d, B, L, W = 32, 8, 128, 20, 900, 32
    prefix = random_cache(rng, 1, Hkv, d, L, 0, [(L, 0)])
    own = random_cache(rng, B, Hkv, d, 0, W)
    p, c, qd = device_cache(prefix), device_cache(own), dev_bf16(normal_bf16(rng, (B, Hq, d))[0])
    size = nd().nd_shared_prefix_decode_workspace_size(B, Hq, Hkv, d, L, W)
    assert size > 0
    want = nd().nd_shared_prefix_decode(qd, p, c, W).clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(50_000_000)
        out = nd().nd_shared_prefix_decode(qd, p, c, W, stream=s)
        filled = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in (size, size, out.nbytes, out.nbytes)]
        torch.cuda.synchronize()
        assert torch.equal(out, want) and all((f == 0x7F).all() for f in filled)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("B", [3, 20, 70])   # rows of a KV head: up to 64, up to 128, more
@pytest.mark.parametrize("L", [601, 1])      # the last tile is partly behind the prefix
@pytest.mark.parametrize("keys", ["normal", "tiny", "zero"])
def test_queries_and_keys_that_are_zero_or_tiny(Hq, Hkv, d, B, L, keys):
    """Scores that are 0, or too small to be seen in fp32: the weights of all keys are then the same, and nothing that
    stands behind the prefix counts."""
    rng = philox(11200 + B + L + d)
    prefix = random_cache(rng, 1, Hkv, d, 900, 0, [(L, 0)])
    prefix.k_scale *= np.float32({"normal": 1.0, "tiny": 2.0 ** -30, "zero": 0.0}[keys])
    own = random_cache(rng, B, Hkv, d, 0, 16, [(0, 0), (0, 5), (0, 40)])
    q = normal_bf16(rng, (B, Hq, d))[1]
    q[:, 0] = 0.0
    q[:, 1] *= 2.0 ** -30
    q[0] = 0.0
    q[1] *= 2.0 ** -100
    check(prefix, own, to_bf16_bits(q), q, 16, f"{keys} keys")


def test_a_zeroed_prefix_and_a_zero_query():
    """What a warm-up or a padded session gives: uniform weights over values that are all 0."""
    n = nd()
    for B in (3, 20, 70):
        prefix, own = n.KVCache.empty(1, 2, 64, 900, 0), n.KVCache.empty(B, 2, 64, 0, 16)
        prefix.sink_len.fill_(601)
        lse = torch.empty(B, 8, device="cuda")
        out = n.nd_shared_prefix_decode(torch.zeros(B, 8, 64, dtype=torch.bfloat16, device="cuda"), prefix, own, 16, lse=lse)
        assert (out == 0).all()
        # the sum, 601 * 2^7, is exact; its log2 (16.2) within 2 ulp of 2^-19, the sum with the maximum and the product
        # with log 2 within half an ulp each: below 6e-6
        torch.testing.assert_close(lse, torch.full_like(lse, math.log(601.0)), rtol=0, atol=1e-5)


@pytest.mark.parametrize("Hq,Hkv,d,B,cap,L,W", [
    (8, 2, 64, 2, 64, 64, 16),        # a short prefix, read by each pair
    (8, 2, 128, 1, 300, 290, 600),    # the same in parts that a merge kernel joins
    (8, 2, 128, 1, 900, 900, 600),    # parts, and a prefix of its own kernel: two streams
    (8, 2, 64, 3, 900, 601, 24),      # two streams, a unit for a CTA
    (8, 2, 64, 20, 900, 601, 24),     # one row block
    (8, 2, 128, 70, 900, 601, 24),    # two row blocks
    (16, 8, 128, 480, 600, 600, 40),  # more pairs than warps
    (16, 8, 64, 480, 600, 601, 41)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_queries_that_are_not_finite(Hq, Hkv, d, B, cap, L, W, value):
    """As in nd_swa_sink_decode, out = 0 and lse = -inf for such a head, with and without own slots; the heads beside it
    keep their bits."""
    rng = philox(11300 + d + B)
    L = min(L, cap)
    prefix = random_cache(rng, 1, Hkv, d, cap, 0, [(L, 0)])
    own = random_cache(rng, B, Hkv, d, 0, W, [(0, W), (0, 0), (0, 2 * W)])
    q = dev_bf16(normal_bf16(rng, (B, Hq, d))[0])
    bad = torch.zeros(B, Hq, dtype=torch.bool, device="cuda")
    bad[:, 1] = bad[0, Hq - 1] = bad[B - 1, 0] = True
    qbad = q.clone()
    qbad[:, 1, 5] = qbad[0, Hq - 1, d - 1] = value
    qbad[B - 1, 0] = value
    p, c = device_cache(prefix), device_cache(own)
    lse, want_lse = torch.empty(B, Hq, device="cuda"), torch.empty(B, Hq, device="cuda")
    out = nd().nd_shared_prefix_decode(qbad, p, c, W, lse=lse)
    want = nd().nd_shared_prefix_decode(q, p, c, W, lse=want_lse)
    assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], want_lse[~bad])
    assert (out[bad] == 0).all() and (lse[bad] == -math.inf).all()
    whole = device_cache(joined(prefix, own))
    plain = nd().nd_swa_sink_decode(qbad, whole, W, lse=lse)
    assert (plain[bad] == 0).all() and (lse[bad] == -math.inf).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [3, 20, 70])
@pytest.mark.parametrize("at", [0, 300, 600])
@pytest.mark.parametrize("far", [12, 20, 28])
def test_small_values_beside_one_large_value(d, B, at, far):
    """A query that attends to small values only, with one key of the prefix, far from the query, whose value is 2^far
    times as large: each value is within 2^-10 of itself or 2^-28 of the largest.  All keys but the far one are the
    same, so their weights are, and the far one's is e^-64.  Compared head by head: the values' bound over their mean
    magnitude, the weights' rounding 2^-11 and the fp32 sums' 2^-14 likewise, and the output's own half step."""
    Hq, Hkv, L = 8, 2, 601
    rng = philox(11400 + d + at)
    prefix, own = random_cache(rng, 1, Hkv, d, 700, 0, [(L, 0)]), random_cache(rng, B, Hkv, d, 0, 8, [(0, 0)])
    prefix.k_codes[...] = 127
    prefix.k_codes[:, :, at] = -127
    prefix.k_scale[...] = 4.0 / 127 / np.sqrt(d / 64)     # score 4 * 8 or -4 * 8 for a query of ones
    prefix.v_scale[:, :, at] *= np.float32(2.0 ** far)
    q = np.ones((B, Hq, d), np.float32)
    out, _ = run(prefix, own, to_bf16_bits(q), 8)
    want, _ = oracle.decode(q[:1], joined(prefix, random_cache(rng, 1, Hkv, d, 0, 8, [(0, 0)])), 8)
    v = prefix.v_codes[0, :, :L].astype(np.float64) * np.repeat(prefix.v_scale[0, :, :L].astype(np.float64), 32, -1)
    small = np.delete(np.abs(v), at, 1).mean(1)            # [Hkv][d]
    largest = np.abs(v).max((1, 2))                        # [Hkv]
    tol = (2.0 ** -10 + 2.0 ** -11 + 2.0 ** -14) * small + 2.0 ** -28 * largest[:, None]
    err = np.abs(out - want)
    assert (err <= np.repeat(tol, Hq // Hkv, 0)[None] + 2.0 ** -8 * np.abs(want)).all(), err.max()


def parts_of(cache, b, window):
    """Sequence b's visible keys and values in fp64: [Hkv][keys][d] each, and the keys' scales [Hkv][keys][d/32]."""
    kpos, sink = oracle.slot_positions(cache, b)
    keep = oracle.decode_keep(int(cache.seq_len[b]) - 1, kpos, sink, window).astype(bool) & (kpos >= 0)
    k, v = (c[b][:, keep] * np.repeat(s[b][:, keep].astype(np.float64), 32, -1)
            for c, s in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)))
    return k, v, cache.k_scale[b][:, keep].astype(np.float64)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B", [4, 18, 40])        # rows of a KV head: up to 64, up to 128, more
@pytest.mark.parametrize("L", [400, 830])         # read by each pair; by the prefix kernel
@pytest.mark.parametrize("order", [1, -1])
def test_scores_that_grow_or_fall_along_the_prefix_row_by_row(d, B, L, order):
    """The running maximum moves by far more than a lazy rescale allows.  Every channel of every head is held to a bound
    from its own keys.  A key's score is off by at most e = 2^-10 sum |q_i k_i| / sqrt(d) in the prefix kernel, or where
    a pair walks it by the fp32 sums that carry 1152 sum q (four roundings of 2^-24 each): the larger, and 2^-20 for the
    scores' own fp32.  Weights p_j then become p_j exp(+-2e_j) after the division by their sum, at most, so the output
    moves by sum p_j (exp(2 e_j) - 1) |v_j - o|; the weights' and values' fp16 add 2^-11 and 2^-10, the sums 2^-14, of
    sum p_j |v_j|, and the output its half step.  lse moves by at most the weighted e."""
    Hq, Hkv, W = 8, 2, 8
    rng = philox(11500 + d + B + L)
    prefix, own = random_cache(rng, 1, Hkv, d, L, 0, [(L, 0)]), random_cache(rng, B, Hkv, d, 0, W)
    prefix.k_scale *= np.linspace(0.01, 8.0, L)[::order][None, None, :, None].astype(np.float32)
    qb, q = normal_bf16(rng, (B, Hq, d))
    out, lse = run(prefix, own, qb, W)
    whole = joined(prefix, own)
    want, wlse = oracle.decode(q, whole, W)
    for b in range(B):
        k, v, scale = parts_of(whole, b, W)
        k, v, scale = (np.repeat(x, Hq // Hkv, 0) for x in (k, v, scale))
        qh = q[b].astype(np.float64)
        s = np.einsum("hc,hjc->hj", qh, k) / np.sqrt(d)
        p = np.exp(s - s.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        e16 = 2.0 ** -10 * np.einsum("hc,hjc->hj", np.abs(qh), np.abs(k))
        e32 = 4 * 2.0 ** -24 * 1152 * np.einsum("hg,hjg->hj", np.abs(qh).reshape(Hq, -1, 32).sum(-1), scale)
        e = np.maximum(e16, e32) / np.sqrt(d) + 2.0 ** -20 * np.abs(s).max(-1, keepdims=True)
        tol = np.einsum("hj,hjc->hc", p * np.expm1(2 * e), np.abs(v - want[b][:, None]))
        tol += (2.0 ** -11 + 2.0 ** -10 + 2.0 ** -14) * np.einsum("hj,hjc->hc", p, np.abs(v)) + 2.0 ** -8 * np.abs(want[b])
        err = np.abs(out[b] - want[b])
        assert (err <= tol).all(), (b, err.max(), (err / tol).max())
        assert (np.abs(lse[b] - wlse[b]) <= (p * np.expm1(e)).sum(-1) + 2.0 ** -20 * np.abs(s).max(-1)).all()
