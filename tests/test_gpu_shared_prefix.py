"""Decode of a batch over one shared prefix, against the fp64 decode of caches
that each hold a copy of the prefix in front of their own sinks; outputs within
the bf16 tolerance of every attention here (max-abs 2e-2, mean-abs 2e-3).  lse:
the score of a key is off by at most 2^-10 sum |q_i k_i| / sqrt(d) (two fp16
roundings, 2^-11 each, of every key channel) plus the fp32 sums' roundings, and
the log of the sum by no more than the worst key's score; with N(0,1) values
the sum stays below 1.5 sqrt(d) for d >= 64: 2^-10 * 1.5 * sqrt(128) < 2e-2."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import assert_close_bf16, dev, dev_bf16, host, need_gpu, no_device_errors
from workloads import normal_bf16, philox

pytestmark = pytest.mark.gpu

FIELDS = ("k_codes", "v_codes", "k_scale", "v_scale", "sink_len", "ring_start", "ring_len", "seq_len")
LSE_TOL = 2e-2


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    no_device_errors()


def nd():
    import sliding_window_kv_swa_gb300 as m
    return m


def device_cache(ref):
    return nd().KVCache(*(dev(getattr(ref, f)) for f in FIELDS), ref.sink_cap, ref.ring_cap)


def random_cache(rng, B, Hkv, d, S, W, lens=None):
    """N(0,1) tokens through the codec; lens[b] = (sinks, ring tokens seen), default full."""
    ref = oracle.Cache(B, Hkv, d, S, W)
    for codes, scale in ((ref.k_codes, ref.k_scale), (ref.v_codes, ref.v_scale)):
        codes[...], scale[...] = oracle.quant_g32(normal_bf16(rng, codes.shape)[1])
    for b in range(B):
        sl, n = (S, W + int(rng.integers(0, W + 1))) if lens is None else lens[b % len(lens)]
        ref.sink_len[b], ref.ring_len[b], ref.seq_len[b] = sl, min(n, W), sl + n
        ref.ring_start[b] = n % W if W and n > W else 0
    return ref


def joined(prefix, own):
    """Each sequence's cache with the prefix's filled slots in front of its own sinks."""
    L = int(prefix.sink_len[0])
    c = oracle.Cache(own.B, own.Hkv, own.d, L + own.sink_cap, own.ring_cap)
    for f in ("k_codes", "v_codes", "k_scale", "v_scale"):
        getattr(c, f)[:, :, :L] = getattr(prefix, f)[:, :, :L]
        getattr(c, f)[:, :, L:] = getattr(own, f)
    c.sink_len[...] = own.sink_len + L
    c.seq_len[...] = own.seq_len + L
    c.ring_start[...], c.ring_len[...] = own.ring_start, own.ring_len
    return c


def run(prefix, own, q_bits, window, **kw):
    B, Hq, d = q_bits.shape
    lse = torch.empty((B, Hq), dtype=torch.float32, device="cuda")
    out = nd().nd_shared_prefix_decode(dev_bf16(q_bits), device_cache(prefix), device_cache(own), window, lse=lse, **kw)
    return host(out), host(lse)


def check(prefix, own, q_bits, q, window, what=""):
    out, lse = run(prefix, own, q_bits, window)
    # own.sink_len < sink_cap leaves a hole in the joined sink region: the oracle counts sinks as a prefix
    want, wlse = np.empty_like(out), np.empty(lse.shape)
    ref = joined(prefix, own)
    L = int(prefix.sink_len[0])
    for b in range(own.B):
        one = oracle.Cache(1, own.Hkv, own.d, ref.sink_cap, ref.ring_cap)
        for f in FIELDS:
            getattr(one, f)[...] = getattr(ref, f)[b:b + 1]
        w, l = oracle.decode(q[b:b + 1], one, window)
        want[b], wlse[b] = w[0], l[0]
    assert_close_bf16(out, want, what)
    seen = np.isfinite(wlse)
    np.testing.assert_array_equal(np.isfinite(lse), seen)
    assert (lse[~seen] == -np.inf).all() and (out[~seen] == 0).all()
    np.testing.assert_allclose(lse[seen], wlse[seen], atol=LSE_TOL, rtol=0)


LAYOUTS = [(8, 2, 64), (4, 4, 64), (8, 1, 64), (32, 8, 128), (3, 1, 128), (16, 2, 128)]


@pytest.mark.parametrize("Hq,Hkv,d", LAYOUTS)
@pytest.mark.parametrize("B,L,cap,S,W,window", [
    (1, 1, 1, 0, 1, 1),          # one key each
    (2, 64, 64, 0, 16, 16),      # whole tiles
    (5, 63, 70, 3, 20, 11),      # ends inside a tile, a hole behind it, a narrower window
    (9, 65, 65, 0, 33, 64),
    (33, 200, 333, 2, 7, 7)])
def test_matches_the_joined_caches(Hq, Hkv, d, B, L, cap, S, W, window):
    rng = philox(10000 + 7 * L + d + B)
    prefix = random_cache(rng, 1, Hkv, d, cap, 4, [(L, 0)])
    lens = None if B < 5 else [(S, 3 * W + 1), (S, W // 2), (0, 0), (S // 2, W)]
    own = random_cache(rng, B, Hkv, d, S, W, lens)
    qb, q = normal_bf16(rng, (B, Hq, d))
    check(prefix, own, qb, q, window)


@pytest.mark.parametrize("Hq,Hkv,d,B,L", [(8, 2, 64, 70, 1500), (32, 8, 128, 40, 700), (16, 16, 64, 130, 129),
                                          (4, 1, 64, 3, 20000), (8, 8, 128, 2, 5000), (16, 2, 128, 257, 300)])
def test_larger_batches_and_longer_prefixes(Hq, Hkv, d, B, L):
    rng = philox(10100 + L)
    prefix = random_cache(rng, 1, Hkv, d, L, 0, [(L, 0)])
    own = random_cache(rng, B, Hkv, d, 0, 40)
    qb, q = normal_bf16(rng, (B, Hq, d))
    check(prefix, own, qb, q, 40)


def test_nothing_visible_and_one_side_empty():
    rng = philox(10200)
    Hq, Hkv, d = 8, 2, 64
    qb, q = normal_bf16(rng, (4, Hq, d))
    empty = random_cache(rng, 1, Hkv, d, 100, 4, [(0, 0)])
    some = random_cache(rng, 1, Hkv, d, 100, 4, [(77, 0)])
    none = random_cache(rng, 4, Hkv, d, 2, 8, [(0, 0)])
    own = random_cache(rng, 4, Hkv, d, 2, 8, [(0, 0), (2, 0), (0, 3), (2, 30)])
    for prefix, cache in ((empty, none), (empty, own), (some, none), (some, own)):
        check(prefix, cache, qb, q, 8)


def test_slots_that_are_not_visible_may_hold_anything():
    """Stale codes and non-finite scales behind the prefix, in empty rings and outside the window."""
    rng = philox(10300)
    Hq, Hkv, d, L, W, window = 8, 2, 128, 90, 24, 10
    prefix = random_cache(rng, 1, Hkv, d, 150, 4, [(L, 0)])
    own = random_cache(rng, 6, Hkv, d, 3, W, [(3, 2 * W + 5), (1, 7), (0, 0)])
    clean, cown = prefix.copy(), own.copy()
    for f in ("k_scale", "v_scale"):
        getattr(prefix, f)[:, :, L:] = np.array([np.nan, np.inf, -np.inf, 3e38], np.float32)
        for b in range(6):
            kpos, sink = oracle.slot_positions(own, b)
            keep = oracle.decode_keep(int(own.seq_len[b]) - 1, kpos, sink, window).astype(bool) & (kpos >= 0)
            getattr(own, f)[b][:, ~keep] = np.nan
    qb, _ = normal_bf16(rng, (6, Hq, d))
    got, want = run(prefix, own, qb, window), run(clean, cown, qb, window)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g, w)


def scales_of_any_size(Hq, Hkv, d, kind, B, L):
    rng = philox(10400 + d)
    W = 16
    prefix = random_cache(rng, 1, Hkv, d, L, 0, [(L, 0)])
    own = random_cache(rng, B, Hkv, d, 0, W)
    kmul, vmul = np.ones(L), np.ones(L)
    if kind == "large":
        kmul[:], vmul[:] = 2.0 ** -20, 2.0 ** 40
    elif kind == "tiny":
        kmul[:], vmul[:] = 2.0 ** 12, 2.0 ** -40
    elif kind == "mixed":
        kmul, vmul = 2.0 ** rng.integers(-40, 1, L), 2.0 ** rng.integers(-20, 21, L)
    elif kind == "rising":
        vmul = 2.0 ** (np.arange(L) // 20)
    else:
        vmul[:200] = 0.0
    prefix.k_scale *= kmul[None, None, :, None].astype(np.float32)
    prefix.v_scale *= vmul[None, None, :, None].astype(np.float32)
    qb, q = normal_bf16(rng, (B, Hq, d))
    if kind == "large":
        own.v_scale *= np.float32(2.0 ** 40)
    if kind == "tiny":
        own.v_scale *= np.float32(2.0 ** -40)
        q, qb = q * 2.0 ** -12, (qb & 0x807F) | (((qb & 0x7F80) >> 7) - 12 << 7).astype(np.uint16)
    out, _ = run(prefix, own, qb, W)
    want, _ = oracle.decode(q, joined(prefix, own), W)
    top = np.abs(want).max()
    assert_close_bf16(out / top, want / top, kind)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("B", [3, 20, 70])   # rows of a KV head: up to 64, up to 128, more
@pytest.mark.parametrize("kind", ["large", "tiny", "mixed", "rising", "zero_v"])
def test_scales_of_any_size(Hq, Hkv, d, kind, B):
    """The power-of-two scaling of keys and values follows the data: large and tiny tokens, magnitudes that differ by
    2^40 within the prefix, values that grow along it, all-zero values."""
    scales_of_any_size(Hq, Hkv, d, kind, B, 330)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("B", [3, 20, 70])
@pytest.mark.parametrize("kind", ["large", "tiny", "mixed", "rising", "zero_v"])
def test_scales_of_any_size_along_a_long_prefix(Hq, Hkv, d, kind, B):
    """The same past the lengths that every pair reads for itself."""
    scales_of_any_size(Hq, Hkv, d, kind, B, 830)


@pytest.mark.parametrize("Hq,Hkv,d", LAYOUTS)
@pytest.mark.parametrize("B,L,cap,S,W,window", [
    (2, 576, 576, 0, 16, 16),        # whole tiles
    (5, 639, 700, 3, 20, 11),        # ends inside a tile, a hole behind it, a narrower window
    (9, 1025, 1025, 0, 33, 64),
    (3, 2000, 5000, 2, 600, 590),    # a long ring
    (40, 513, 900, 0, 520, 600)])    # more pairs than SMs, each with a long walk
def test_matches_the_joined_caches_past_short_prefixes(Hq, Hkv, d, B, L, cap, S, W, window):
    rng = philox(10050 + 7 * L + d + B)
    prefix = random_cache(rng, 1, Hkv, d, cap, 4, [(L, 0)])
    lens = None if B < 5 else [(S, 3 * W + 1), (S, W // 2), (0, 0), (S // 2, W)]
    own = random_cache(rng, B, Hkv, d, S, W, lens)
    qb, q = normal_bf16(rng, (B, Hq, d))
    check(prefix, own, qb, q, window)


def test_the_own_part_beside_the_prefix_kernel():
    """Few pairs: the own part's CTAs run while the prefix is multiplied, also with parts of a pair; a captured call
    follows a prefix that grows from nothing to its capacity."""
    rng = philox(10060)
    for Hq, Hkv, d, B, cap, W in ((8, 2, 128, 1, 6000, 24), (16, 8, 64, 2, 9000, 40), (4, 1, 64, 2, 3000, 2048)):
        prefix = random_cache(rng, 1, Hkv, d, cap, 0, [(cap, 0)])
        own = random_cache(rng, B, Hkv, d, 0, W)
        qb, q = normal_bf16(rng, (B, Hq, d))
        p, c, qd = device_cache(prefix), device_cache(own), dev_bf16(qb)
        ws = torch.empty(nd().nd_shared_prefix_decode_workspace_size(B, Hq, Hkv, d, cap, W), dtype=torch.uint8, device="cuda")
        out = torch.empty(B, Hq, d, dtype=torch.bfloat16, device="cuda")
        nd().nd_shared_prefix_decode(qd, p, c, W, out=out, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            nd().nd_shared_prefix_decode(qd, p, c, W, out=out, workspace=ws)
            nd().nd_shared_prefix_decode(qd, p, c, W, out=out, workspace=ws)
        for length in (0, 1, 130, 2500, cap):
            p.sink_len.fill_(length)
            prefix.sink_len[0] = length
            for _ in range(3):
                g.replay()
            want, _ = oracle.decode(q, joined(prefix, own), W)
            assert_close_bf16(host(out), want, f"prefix of {length} of {cap}")


@pytest.mark.parametrize("B", [3, 20, 70])
def test_slots_behind_a_long_prefix_may_hold_anything(B):
    rng = philox(10350 + B)
    Hq, Hkv, d, L, W = 8, 2, 128, 601, 24
    prefix = random_cache(rng, 1, Hkv, d, 900, 4, [(L, 0)])
    own = random_cache(rng, B, Hkv, d, 3, W, [(3, 2 * W + 5), (1, 7), (0, 0)])
    clean = prefix.copy()
    for f in ("k_scale", "v_scale"):
        getattr(prefix, f)[:, :, L:] = np.array([np.nan, np.inf, -np.inf, 3e38], np.float32)
    qb, q = normal_bf16(rng, (B, Hq, d))
    got, want = run(prefix, own, qb, W), run(clean, own, qb, W)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g, w)
    check(prefix, own, qb, q, W)


@pytest.mark.parametrize("d,W", [(128, 40), (64, 41)])
def test_more_pairs_than_warps(d, W):
    """Several units to a warp one after the other, and a last round that a CTA's warps share."""
    rng = philox(10360 + d)
    Hq, Hkv, B, L = 16, 8, 480, 70
    prefix = random_cache(rng, 1, Hkv, d, L, 0, [(L, 0)])
    own = random_cache(rng, B, Hkv, d, 1, W, [(1, 2 * W), (0, 5), (0, 0), (1, W), (0, W + 1)])
    qb, q = normal_bf16(rng, (B, Hq, d))
    check(prefix, own, qb, q, W - 3)


def test_scores_that_grow_along_the_prefix():
    """The running maximum moves by far more than a lazy rescale allows, in both directions."""
    rng = philox(10500)
    Hq, Hkv, d, L = 8, 2, 64, 400
    for order, B in ((1, 18), (-1, 18), (1, 4), (-1, 4), (1, 40), (-1, 40)):
        prefix = random_cache(rng, 1, Hkv, d, L, 0, [(L, 0)])
        ramp = np.linspace(0.01, 8.0, L)[::order]
        prefix.k_scale *= ramp[None, None, :, None].astype(np.float32)
        own = random_cache(rng, B, Hkv, d, 0, 8)
        qb, q = normal_bf16(rng, (B, Hq, d))
        out, _ = run(prefix, own, qb, 8)
        want, _ = oracle.decode(q, joined(prefix, own), 8)
        # a key's score is off by 2^-10 sum|q_i k_i| / sqrt(d) <= 2^-10 * 8 * 8 = 2^-4 at the largest keys, its weight
        # by as much, and the output by twice that of the largest value
        err = np.abs(out - want)
        assert err.max() <= 2 * 2.0 ** -4 * 4 and err.mean() <= 2e-2


def test_bad_metadata_is_flagged_and_skipped():
    rng = philox(10600)
    Hq, Hkv, d = 8, 2, 64
    prefix = random_cache(rng, 1, Hkv, d, 80, 4, [(80, 0)])
    own = random_cache(rng, 3, Hkv, d, 0, 8)
    qb, q = normal_bf16(rng, (3, Hq, d))
    own.ring_len[1] = 9                     # the sequence's own slots are skipped, the prefix is not
    out, _ = run(prefix, own, qb, 8)
    torch.cuda.synchronize()
    assert nd().nd_device_errors(clear=True) == 2
    own.ring_len[1] = own.ring_start[1] = 0
    want, _ = oracle.decode(q, joined(prefix, own), 8)
    assert_close_bf16(out, want)
    own = random_cache(rng, 3, Hkv, d, 0, 8)
    prefix.sink_len[0] = 81                 # the prefix is skipped, the sequences are not
    out, _ = run(prefix, own, qb, 8)
    torch.cuda.synchronize()
    assert nd().nd_device_errors(clear=True) == 2
    prefix.sink_len[0] = 0
    want, _ = oracle.decode(q, joined(prefix, own), 8)
    assert_close_bf16(out, want)


def test_captured_replayed_and_on_two_streams():
    """A captured call follows the metadata (the prefix and the rings grow between replays); two calls at once with
    their own workspaces do not disturb each other; the same call twice gives the same bits."""
    rng = philox(10700)
    Hq, Hkv, d, B, L = 32, 8, 128, 20, 900
    prefix = random_cache(rng, 1, Hkv, d, L, 0, [(L, 0)])
    own = random_cache(rng, B, Hkv, d, 0, 32)
    qb, q = normal_bf16(rng, (B, Hq, d))
    p, c, qd = device_cache(prefix), device_cache(own), dev_bf16(qb)
    size = nd().nd_shared_prefix_decode_workspace_size(B, Hq, Hkv, d, L, 32)
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = [torch.empty(B, Hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    g = torch.cuda.CUDAGraph()
    nd().nd_shared_prefix_decode(qd, p, c, 32, out=out[0], workspace=ws[0])
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        nd().nd_shared_prefix_decode(qd, p, c, 32, out=out[0], workspace=ws[0])
    for length in (L, 1, 130, 0, L):
        p.sink_len.fill_(length)
        prefix.sink_len[0] = length
        g.replay()
        want, _ = oracle.decode(q, joined(prefix, own), 32)
        assert_close_bf16(host(out[0]), want, f"prefix of {length}")
    first = out[0].clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, w, o in zip(streams, ws, out):
            with torch.cuda.stream(s):
                nd().nd_shared_prefix_decode(qd, p, c, 32, out=o, workspace=w)
    torch.cuda.synchronize()
    for o in out:
        assert torch.equal(o, first)


def test_two_graphs_share_a_workspace():
    """Replayed in turn, as any two users of one workspace have to be."""
    rng = philox(10750)
    Hq, Hkv, d, B = 32, 8, 128, 12
    own = random_cache(rng, B, Hkv, d, 0, 32)
    qb, q = normal_bf16(rng, (B, Hq, d))
    c, qd = device_cache(own), dev_bf16(qb)
    prefixes = [random_cache(rng, 1, Hkv, d, L, 0, [(L, 0)]) for L in (700, 1900)]
    devs = [device_cache(p) for p in prefixes]
    size = max(nd().nd_shared_prefix_decode_workspace_size(B, Hq, Hkv, d, p.sink_cap, 32) for p in prefixes)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    out = [torch.empty(B, Hq, d, dtype=torch.bfloat16, device="cuda") for _ in prefixes]
    graphs = []
    for p, o in zip(devs, out):
        nd().nd_shared_prefix_decode(qd, p, c, 32, out=o, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            nd().nd_shared_prefix_decode(qd, p, c, 32, out=o, workspace=ws)
        graphs.append(g)
    for o in out:
        o.zero_()
    for _ in range(5):
        for g in graphs:
            g.replay()
    for p, o in zip(prefixes, out):
        want, _ = oracle.decode(q, joined(p, own), 32)
        assert_close_bf16(host(o), want)


def test_outputs_and_workspace_stay_inside_their_buffers():
    rng = philox(10800)
    for Hq, Hkv, d, B, L in ((8, 2, 64, 3, 70), (16, 2, 128, 35, 300), (8, 8, 128, 2, 4000)):
        prefix = random_cache(rng, 1, Hkv, d, L, 0, [(L, 0)])
        own = random_cache(rng, B, Hkv, d, 0, 16)
        qb, q = normal_bf16(rng, (B, Hq, d))
        size = nd().nd_shared_prefix_decode_workspace_size(B, Hq, Hkv, d, L, 16)
        pad = 4096
        ws = torch.full((size + 2 * pad,), 0xA5, dtype=torch.uint8, device="cuda")
        o = torch.full((B * Hq * d + 2 * pad,), 3.0, dtype=torch.bfloat16, device="cuda")
        out = o[pad:-pad].view(B, Hq, d)
        nd().nd_shared_prefix_decode(dev_bf16(qb), device_cache(prefix), device_cache(own), 16, out=out,
                                     workspace=ws[pad:pad + size])
        assert (ws[:pad] == 0xA5).all() and (ws[pad + size:] == 0xA5).all()
        assert (o[:pad] == 3.0).all() and (o[-pad:] == 3.0).all()
        want, _ = oracle.decode(q, joined(prefix, own), 16)
        assert_close_bf16(host(out), want)


def test_a_prompt_served_to_many_sessions():
    """The operators together: a prompt's keys are normalised and rotated, put into a one-row cache as its pinned
    prefix, and every session's tokens are appended and decoded over it; the same from per-session caches that were
    given the whole history, and what was appended reads back."""
    rng = philox(10900)
    Hq, Hkv, d, B, L, W, steps, theta = 8, 2, 64, 5, 75, 6, 9, 10000.0
    n = nd()
    wq, wk = (dev(rng.uniform(0.5, 1.5, d).astype(np.float32)) for _ in range(2))
    qkv = dev_bf16(normal_bf16(rng, (1, L, Hq + 2 * Hkv, d))[0])
    _, k = n.nd_qk_norm_rope(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], wq, wk, 1e-6, theta)
    v = qkv[:, :, Hq + Hkv:].contiguous()
    row = torch.zeros(1, dtype=torch.int32, device="cuda")
    ones = torch.ones(1, L, dtype=torch.uint8, device="cuda")
    prefix = n.KVCache.empty(1, Hkv, d, L, 1)
    n.nd_kv_cache_from_prefill(prefix, k, v, row, sink=ones)
    whole = n.KVCache.empty(B, Hkv, d, L, W)
    n.nd_kv_cache_from_prefill(whole, k, v, torch.zeros(B, dtype=torch.int32, device="cuda"), sink=ones.expand(1, L).contiguous())
    own = n.KVCache.empty(B, Hkv, d, 0, W)
    for step in range(steps):
        x = dev_bf16(normal_bf16(rng, (B, Hq + 2 * Hkv, d))[0])
        parts = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        q1 = n.nd_qk_norm_rope_append(parts[0], own, parts[1], parts[2], wq, wk, 1e-6, theta, pos_base=prefix.seq_len)
        q2 = n.nd_qk_norm_rope_append(parts[0], whole, parts[1], parts[2], wq, wk, 1e-6, theta)
        assert torch.equal(q1, q2)
        out = n.nd_shared_prefix_decode(q1, prefix, own, W)
        want = n.nd_swa_sink_decode(q2, whole, W)
        assert_close_bf16(host(out), host(want), f"step {step}")
    a, b = n.nd_kv_cache_read(own, W), n.nd_kv_cache_read(whole, W)
    p = n.nd_kv_cache_read(prefix, 1)
    for i in range(2):
        assert torch.equal(a[i], b[i][:, L:]) and torch.equal(b[i][:, :L], p[i][:, :L].expand(B, -1, -1, -1))
    np.testing.assert_array_equal(host(a[2]) + L, host(b[2])[:, L:])


def test_caches_whose_offsets_pass_32_bits():
    """A prefix region and own rings of more than 2^32 bytes of codes: the last head and sequence lie behind it."""
    rng = philox(10950)
    n, Hq, Hkv, d, B, L, steps = nd(), 8, 2, 128, 2, 600, 5
    far, near = n.KVCache.empty(1, Hkv, d, 34_000_000, 0), n.KVCache.empty(1, Hkv, d, L, 0)
    ref = random_cache(rng, 1, Hkv, d, L, 0, [(L, 0)])
    for f in ("k_codes", "v_codes", "k_scale", "v_scale"):
        getattr(near, f).copy_(dev(getattr(ref, f)))
        getattr(far, f)[:, :, :L].copy_(getattr(near, f))
    own, ring = n.KVCache.empty(B, Hkv, d, 0, 8), n.KVCache.empty(B, Hkv, d, 0, 12_000_000)
    for c, length in ((near, L), (far, L)):
        c.sink_len.fill_(length)
        c.seq_len.fill_(length)
    assert ring.k_codes[0].numel() * (B - 1) + 12_000_000 * d > 1 << 32 and far.k_codes[0, 0].numel() > 1 << 32
    for _ in range(steps):
        x = dev_bf16(normal_bf16(rng, (B, Hq + 2 * Hkv, d))[0])
        parts = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        q = [n.nd_qk_norm_rope_append(parts[0], c, parts[1], parts[2], rope_theta=10000.0, pos_base=near.seq_len)
             for c in (own, ring)]
    assert torch.equal(*q)
    for a, b in zip(n.nd_kv_cache_read(own, 8), n.nd_kv_cache_read(ring, 8)):
        rows = (slice(None), slice(0, steps)) if a.dim() > 1 else slice(None)
        assert torch.equal(a[rows], b[rows])
    want = host(n.nd_shared_prefix_decode(q[0], near, own, 8))
    for prefix, cache in ((far, own), (near, ring), (far, ring)):
        # (two results, each as far from the exact one as any: twice the tolerance, as halves)
        assert_close_bf16(host(n.nd_shared_prefix_decode(q[0], prefix, cache, 8)) / 2, want / 2)
