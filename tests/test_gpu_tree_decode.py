"""Attention of a tree of drafted tokens against the fp64 softmax over each
node's slots and nodes; outputs within the bf16 tolerance of every attention
here (max-abs 2e-2, mean-abs 2e-3).  lse: a score is off by at most 2^-10 sum
|q_i k_i| / sqrt(d) (two fp16 roundings, 2^-11 each, of every key channel) plus
the fp32 sums' roundings; with N(0,1) values the sum stays below 1.5 sqrt(d) for
d >= 64: 2^-10 * 1.5 * sqrt(128) < 2e-2."""
import numpy as np
import pytest
import torch

import oracle
import tree_util as tu
from gpu_util import assert_close_bf16, dev_bf16, host, need_gpu, no_device_errors
from tree_util import i32
from workloads import normal_bf16, philox

pytestmark = pytest.mark.gpu
LSE_TOL = 2e-2


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    no_device_errors()


def nd():
    import sliding_window_kv_swa_gb300 as m
    return m


def nodes(rng, B, n, Hq, Hkv, d):
    bits, x = normal_bf16(rng, (B, n, Hq + 2 * Hkv, d))
    t = dev_bf16(bits)
    return (t[:, :, :Hq].contiguous(), t[:, :, Hq:Hq + Hkv], t[:, :, Hq + Hkv:]), \
        (x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:])


def check(ref, dev_qkv, qkv, depth, see, mask, window, what=""):
    q, k, v = dev_qkv
    B, n, Hq, d = q.shape
    lse = torch.empty((B, Hq, n), dtype=torch.float32, device="cuda")
    out = nd().nd_tree_decode(q, tu.device_cache(ref), k, v, i32(depth), i32(mask), window, lse=lse)
    want, wlse = tu.decode_rows(*qkv[:1], ref, *qkv[1:], depth, see, window)
    got, glse = host(out), host(lse)
    assert_close_bf16(got, want, what)
    seen = np.isfinite(wlse)
    np.testing.assert_array_equal(np.isfinite(glse), seen)
    assert (glse[~seen] == -np.inf).all() and (got.transpose(0, 2, 1, 3)[~seen] == 0).all()
    if seen.any():
        np.testing.assert_allclose(glse[seen], wlse[seen], atol=LSE_TOL, rtol=0)
    return out


LAYOUTS = [(8, 2, 64), (4, 4, 64), (8, 1, 64), (32, 8, 128), (3, 1, 128), (16, 2, 128), (5, 1, 64), (7, 1, 128)]


@pytest.mark.parametrize("Hq,Hkv,d", LAYOUTS)
@pytest.mark.parametrize("B,n,S,W,window", [
    (1, 1, 0, 1, 1),           # one node, nothing of the cache inside its window
    (2, 4, 64, 64, 64),        # whole tiles
    (3, 13, 5, 40, 17),        # ragged, a narrower window
    (2, 33, 63, 65, 500),      # more than a word of nodes, tiles that end inside the sinks and the ring
    (1, 100, 200, 100, 30),    # deeper than the window
    (2, 70, 0, 7, 7)])
def test_matches_the_softmax(Hq, Hkv, d, B, n, S, W, window):
    rng = philox(22000 + 7 * n + d + Hq)
    lens = None if B == 1 else [(S, 3 * W + 1), (S // 2, W // 2), (0, 0)]
    ref = tu.random_cache(rng, B, Hkv, d, S, W, lens)
    parents = tu.random_parents(rng, B, n, reach=3)
    counts = np.maximum(n - np.arange(B) * (n // 3), 0).astype(np.int32)
    depth, _, mask, see = tu.layout(parents, counts, ref.seq_len, 0, window)
    a, b = nodes(rng, B, n, Hq, Hkv, d)
    check(ref, a, b, depth, see, mask, window)


@pytest.mark.parametrize("Hq,Hkv,d,B,n,S,W", [(8, 2, 64, 1, 256, 300, 100), (32, 8, 128, 1, 256, 100, 256), (32, 8, 128, 20, 16, 1024, 256),
                                              (8, 2, 64, 200, 5, 10, 30), (16, 16, 64, 37, 13, 48, 200), (8, 1, 128, 2, 64, 3000, 0),
                                              (4, 1, 64, 1, 8, 20000, 64), (8, 8, 64, 1, 3, 9000, 128)])
def test_larger_ones(Hq, Hkv, d, B, n, S, W):
    rng = philox(22100 + n + S)
    ref = tu.random_cache(rng, B, Hkv, d, S, W)
    depth, _, mask, see = tu.layout(tu.random_parents(rng, B, n), None, ref.seq_len, 0, 64)
    a, b = nodes(rng, B, n, Hq, Hkv, d)
    check(ref, a, b, depth, see, mask, 64)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (32, 8, 128)])
def test_without_a_cache_and_with_arbitrary_masks(Hq, Hkv, d):
    rng = philox(22200)
    B, n = 3, 45
    for S, W in ((0, 8), (9, 0)):
        ref = tu.random_cache(rng, B, Hkv, d, S, W, [(S, W), (0, 0)])
        see = rng.random((B, n, n)) < 0.2
        see[:, 7] = False                          # nothing: empty where the cache is
        see[:, 11] = True
        depth = rng.integers(0, 5, (B, n)).astype(np.int32)
        depth[:, 20] = -1                          # padding in the middle
        depth[0, 3] = -7
        bits = np.zeros((B, n, 64), np.uint64)
        bits[..., :n] = see
        bits[:, 5, n:] = 1                         # bits from n on count nothing
        mask = (bits.reshape(B, n, 2, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
        a, b = nodes(rng, B, n, Hq, Hkv, d)
        check(ref, a, b, depth, see, mask, 6)


def test_metadata_out_of_range_are_flagged_and_give_nothing():
    rng = philox(22240)
    B, n, Hq, Hkv, d, S, W = 4, 10, 8, 2, 64, 300, 40
    ref = tu.random_cache(rng, B, Hkv, d, S, W)
    depth, _, mask, see = tu.layout(tu.random_parents(rng, B, n), None, ref.seq_len, 0, 30)
    (q, k, v), x = nodes(rng, B, n, Hq, Hkv, d)
    want, _ = tu.decode_rows(x[0], ref, x[1], x[2], depth, see, 30)
    cache = tu.device_cache(ref)
    cache.sink_len[0], cache.ring_len[1], cache.ring_start[3] = S + 1, -1, W
    lse = torch.empty((B, Hq, n), dtype=torch.float32, device="cuda")
    out = nd().nd_tree_decode(q, cache, k, v, i32(depth), i32(mask), 30, lse=lse)
    torch.cuda.synchronize()
    assert nd().nd_device_errors(clear=True) == 2
    for b in (0, 1, 3):
        assert (out[b] == 0).all() and (lse[b] == -float("inf")).all()
    assert_close_bf16(host(out)[2], want[2])


def test_depths_far_beyond_the_window():
    rng = philox(22250)
    B, n, Hq, Hkv, d = 1, 6, 8, 2, 64
    ref = tu.random_cache(rng, B, Hkv, d, 0, 20)
    depth = np.array([[0, 19, 20, 2 ** 31 - 1, 1000, 5]], np.int32)
    see = np.eye(n, dtype=bool)[None]
    mask = (1 << np.arange(n, dtype=np.uint32)).astype(np.uint32).reshape(1, n, 1)
    a, b = nodes(rng, B, n, Hq, Hkv, d)
    for window in (1, 20, 2 ** 31 - 1):
        check(ref, a, b, depth, see, mask, window)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (32, 8, 128)])
def test_a_chain_is_a_chunk_and_one_node_a_decode(Hq, Hkv, d):
    """The chunk prefill rounds cached keys to bf16, this to fp16 or not at all: the two are within the sum of their tolerances."""
    rng = philox(22300)
    B, n, S, W, window = 3, 24, 30, 64, 50
    ref = tu.random_cache(rng, B, Hkv, d, S, W, [(S, 2 * W), (S // 2, W // 2), (0, 3)])
    parents = np.tile(np.arange(n, dtype=np.int32) - 1, (B, 1))
    depth, _, mask, _ = tu.layout(parents, None, ref.seq_len, 0, window)
    (q, k, v), _ = nodes(rng, B, n, Hq, Hkv, d)
    out = nd().nd_tree_decode(q, tu.device_cache(ref), k, v, i32(depth), i32(mask), window)
    want = nd().nd_swa_sink_chunk_prefill(q, k.contiguous(), v.contiguous(), tu.device_cache(ref), window)
    err = np.abs(host(out) - host(want))
    assert err.max() <= 4e-2 and err.mean() <= 4e-3


def test_padding_and_masked_keys_may_hold_anything():
    """Keys, values and queries of padding, slots that the metadata hides and nodes that nobody sees reach no output."""
    rng = philox(22400)
    B, n, Hq, Hkv, d, S, W, window = 2, 20, 8, 2, 64, 40, 50, 30
    ref = tu.random_cache(rng, B, Hkv, d, S, W, [(13, 2 * W), (S, W // 3)])
    counts = np.array([12, 7], np.int32)
    depth, _, mask, see = tu.layout(tu.random_parents(rng, B, n), counts, ref.seq_len, 0, window)
    (q, k, v), x = nodes(rng, B, n, Hq, Hkv, d)
    cache = tu.device_cache(ref)
    args = (i32(depth), i32(mask), window)
    want = nd().nd_tree_decode(q, cache, k, v, *args)
    k2, v2, q2 = k.clone(), v.clone(), q.clone()
    for b in range(B):
        for t, bad in ((k2, float("nan")), (v2, float("inf")), (q2, float("nan"))):
            t[b, counts[b]:] = bad
    for scale in (cache.k_scale, cache.v_scale):
        scale[0, :, 13:S] = float("nan")
        scale[1, :, S + W // 3:] = float("inf")
    got = nd().nd_tree_decode(q2, cache, k2, v2, *args)
    assert torch.equal(got, want)


def test_a_row_with_a_nan_or_an_infinity_leaves_the_others():
    rng = philox(22450)
    B, n, Hq, Hkv, d, S, W = 1, 10, 8, 2, 64, 40, 50
    ref = tu.random_cache(rng, B, Hkv, d, S, W)
    depth, _, mask, _ = tu.layout(tu.random_parents(rng, B, n), None, ref.seq_len, 0, 99)
    (q, k, v), _ = nodes(rng, B, n, Hq, Hkv, d)
    cache = tu.device_cache(ref)
    want = nd().nd_tree_decode(q, cache, k, v, i32(depth), i32(mask), 99)
    q2 = q.clone()
    q2[0, 3, 1, 5], q2[0, 4, 6, 0] = float("nan"), float("inf")
    got = nd().nd_tree_decode(q2, cache, k, v, i32(depth), i32(mask), 99)
    same = torch.ones(n, Hq, dtype=torch.bool, device="cuda")
    same[3, 1] = same[4, 6] = False
    assert torch.equal(got[0][same], want[0][same])


def test_a_node_that_is_not_finite_reaches_the_rows_that_see_it_alone():
    """Rows that see such a node are NaN (all channels, and lse); the others' outputs are those without it."""
    rng = philox(22470)
    B, n, Hq, Hkv, d, S, W = 2, 70, 8, 2, 64, 40, 50
    ref = tu.random_cache(rng, B, Hkv, d, S, W)
    depth, _, mask, see = tu.layout(tu.random_parents(rng, B, n, reach=3), None, ref.seq_len, 0, 9)
    (q, k, v), x = nodes(rng, B, n, Hq, Hkv, d)
    k2, v2 = k.clone(), v.clone()
    k2[0, 5, 0, 7], k2[0, 66, 1, 0], v2[1, 9, 1, 63], v2[1, 65, 0, 1] = float("nan"), float("inf"), float("-inf"), float("nan")
    lse = torch.empty((B, Hq, n), dtype=torch.float32, device="cuda")
    out = nd().nd_tree_decode(q, tu.device_cache(ref), k2, v2, i32(depth), i32(mask), 60, lse=lse)
    want, wlse = tu.decode_rows(x[0], ref, x[1], x[2], depth, see, 60)
    got, glse = host(out), host(lse)
    hit = np.zeros((B, n, Hq), bool)
    for b, node, head in ((0, 5, 0), (0, 66, 1), (1, 9, 1), (1, 65, 0)):
        hit[b, :, head * 4:head * 4 + 4] |= see[b, :, node][:, None]
    assert np.isnan(got[hit]).all() and np.isnan(glse.transpose(0, 2, 1)[hit]).all() and hit.any()
    assert_close_bf16(got[~hit], want[~hit])
    np.testing.assert_allclose(glse.transpose(0, 2, 1)[~hit], wlse.transpose(0, 2, 1)[~hit], atol=LSE_TOL, rtol=0)


@pytest.mark.parametrize("d", [64, 128])
def test_values_that_grow_along_the_cache(d):
    """Keys and values whose scales grow (and fall) by tiles: O is rescaled on the way.  A score is off by 2^-10 sum |q k| /
    sqrt(d), so a weight by that of itself and an output by twice that of sum p |v|, plus its rounding."""
    rng = philox(22550 + d)
    B, n, Hq, Hkv, S, W = 1, 40, 4, 2, 900, 300
    for grow in (1.0, -1.0):
        ref = tu.random_cache(rng, B, Hkv, d, S, W)
        steps = np.floor(grow * np.arange(S + W) / 60).astype(np.float32)
        ref.v_scale *= np.exp2(steps)[None, None, :, None]
        ref.k_scale *= np.float32(0.5)
        ref.v_scale[:, :, 128:256] = 0.0
        depth, _, mask, see = tu.layout(tu.random_parents(rng, B, n), None, ref.seq_len, 0, 400)
        (q, k, v), x = nodes(rng, B, n, Hq, Hkv, d)
        out = host(nd().nd_tree_decode(q, tu.device_cache(ref), k, v, i32(depth), i32(mask), 400))
        want, _ = tu.decode_rows(x[0], ref, x[1], x[2], depth, see, 400)
        reach = 2.0 ** -10 * 5.0 * np.abs(x[0]).sum(-1).max() / np.sqrt(d)
        top = np.abs(want).max()
        assert np.abs(out - want).max() <= 2 * reach * max(top, 1.0) * 4 + 2.0 ** -8 * top


def test_large_and_small_values():
    """Keys and values of very different sizes: scores up to a few hundred, values down to 2^-20 of the largest."""
    rng = philox(22500)
    B, n, Hq, Hkv, d, S, W = 1, 18, 8, 2, 128, 150, 60
    ref = tu.random_cache(rng, B, Hkv, d, S, W)
    ref.k_scale *= np.exp2(rng.integers(-6, 3, ref.k_scale.shape)).astype(np.float32)
    ref.v_scale *= np.exp2(rng.integers(-12, 5, ref.v_scale.shape)).astype(np.float32)
    depth, _, mask, see = tu.layout(tu.random_parents(rng, B, n), None, ref.seq_len, 0, 99)
    (q, k, v), x = nodes(rng, B, n, Hq, Hkv, d)
    lse = torch.empty((B, Hq, n), dtype=torch.float32, device="cuda")
    out = host(nd().nd_tree_decode(q, tu.device_cache(ref), k, v, i32(depth), i32(mask), 99, lse=lse))
    want, wlse = tu.decode_rows(x[0], ref, x[1], x[2], depth, see, 99)
    # a score: 2^-10 sum |q_i k_i| / sqrt(d), so a weight is off by that, and an output by twice that of sum p |v|, plus its rounding
    most = max(np.abs(oracle.dequant_g32(ref.k_codes, ref.k_scale)).max(), 5.0)
    reach = 2.0 ** -10 * most * np.abs(x[0]).sum(-1).max() / np.sqrt(d)
    top = max(np.abs(oracle.dequant_g32(ref.v_codes, ref.v_scale)).max(), np.abs(x[2]).max())
    assert np.abs(host(lse) - wlse).max() <= reach
    assert np.abs(out - want).max() <= 2 * reach * top + 2.0 ** -8 * top


def test_repeats_itself_in_a_graph_on_another_stream_and_with_a_workspace():
    rng = philox(22600)
    for B, n, Hq, Hkv, d, S, W in ((2, 20, 8, 2, 64, 700, 64), (1, 64, 32, 8, 128, 2000, 64), (40, 5, 8, 2, 64, 30, 30)):
        ref = tu.random_cache(rng, B, Hkv, d, S, W)
        depth, _, mask, _ = tu.layout(tu.random_parents(rng, B, n), None, ref.seq_len, 0, 99)
        (q, k, v), _ = nodes(rng, B, n, Hq, Hkv, d)
        cache = tu.device_cache(ref)
        size = nd().nd_tree_decode_workspace_size(B, n, Hq, Hkv, d, S + W)
        ws = torch.full((max(size, 16),), 255, dtype=torch.uint8, device="cuda")
        dd, dm = i32(depth), i32(mask)
        want = nd().nd_tree_decode(q, cache, k, v, dd, dm, 99)
        assert torch.equal(nd().nd_tree_decode(q, cache, k, v, dd, dm, 99, workspace=ws), want)
        out = torch.empty_like(q)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            nd().nd_tree_decode(q, cache, k, v, dd, dm, 99, out=out, workspace=ws)
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)


def test_offsets_that_pass_32_bits_in_a_region_mostly_empty():
    """The last KV head's codes lie 5.6 GB into the cache; outputs are those of a small cache with the same slots, whose tiles are
    split otherwise: both within the tolerance of the same fp64 rows."""
    rng = philox(22650)
    B, n, Hq, Hkv, d, S, W = 1, 9, 8, 4, 128, 150, 64
    ref = tu.random_cache(rng, B, Hkv, d, S, W)
    depth, _, mask, see = tu.layout(tu.random_parents(rng, B, n), None, ref.seq_len, 0, 99)
    (q, k, v), x = nodes(rng, B, n, Hq, Hkv, d)
    small, cap = tu.device_cache(ref), (11 << 20) + 5
    big = {}
    for f in ("k_codes", "v_codes", "k_scale", "v_scale"):
        src = getattr(small, f)
        t = torch.empty((B, Hkv, cap + W, src.shape[3]), dtype=src.dtype, device="cuda")
        t[:, :, :S], t[:, :, cap:] = src[:, :, :S], src[:, :, S:]
        big[f] = t
    # (metadata of its own: each cache is appended to below)
    meta = {f: getattr(small, f).clone() for f in ("sink_len", "ring_start", "ring_len", "seq_len")}
    cache = nd().KVCache(**big, **meta, sink_cap=cap, ring_cap=W)
    out = nd().nd_tree_decode(q, cache, k, v, i32(depth), i32(mask), 99)
    want, _ = tu.decode_rows(x[0], ref, x[1], x[2], depth, see, 99)
    assert_close_bf16(host(out), want)
    # and the append: the path's tokens behind the newest ring entry
    path, length = np.array([[0, 3, 8]], np.int32), np.array([3], np.int32)
    nd().nd_tree_commit(cache, k, v, i32(path), i32(length))
    nd().nd_tree_commit(small, k, v, i32(path), i32(length))
    for f in big:
        assert torch.equal(getattr(cache, f)[:, :, cap:], getattr(small, f)[:, :, S:]), f


def test_two_streams_at_once():
    """Calls that share nothing but the cache's slots, on two streams, many times over."""
    rng = philox(22680)
    B, n, Hq, Hkv, d, S, W = 3, 12, 8, 2, 64, 500, 64
    ref = tu.random_cache(rng, B, Hkv, d, S, W)
    cache = tu.device_cache(ref)
    depth, _, mask, _ = tu.layout(tu.random_parents(rng, B, n), None, ref.seq_len, 0, 99)
    dd, dm = i32(depth), i32(mask)
    jobs, want = [nodes(rng, B, n, Hq, Hkv, d)[0] for _ in range(2)], []
    for q, k, v in jobs:
        want.append(nd().nd_tree_decode(q, cache, k, v, dd, dm, 99))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in jobs], [[], []]
    for _ in range(20):
        for i, (q, k, v) in enumerate(jobs):
            with torch.cuda.stream(streams[i]):
                got[i].append(nd().nd_tree_decode(q, cache, k, v, dd, dm, 99))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_the_whole_step():
    """Draft, lay out, rotate, attend, accept, commit, and draft again: the cache after two steps is that of single appends, and
    each step's attention the fp64 one."""
    rng = philox(22700)
    B, n, Hq, Hkv, d, S, W, window, m = 4, 17, 8, 2, 64, 6, 24, 20, 5
    ref = tu.random_cache(rng, B, Hkv, d, S, W, [(S, 2 * W), (S, 3), (0, 0), (S, W)])
    cache = tu.device_cache(ref)
    for step in range(2):
        parents = tu.random_parents(rng, B, n, roots=0)
        counts = rng.integers(1, n + 1, B).astype(np.int32)
        dp, dc = i32(parents), i32(counts)
        depth, pos, mask = nd().nd_tree_layout(dp, cache.seq_len, window, n_nodes=dc)
        (q, k, v), x = nodes(rng, B, n, Hq, Hkv, d)
        qr, kr = nd().nd_rope_positions(q, k, nd().RopeConfig(), positions=pos)
        out = nd().nd_tree_decode(qr, cache, kr, v, depth, mask, window)
        wd, _, _, see = tu.layout(parents, counts, ref.seq_len, 0, window)
        want, _ = tu.decode_rows(host(qr), ref, host(kr), x[2], wd, see, window)
        assert_close_bf16(host(out), want, f"step {step}")
        tokens, target = (rng.integers(0, 2, (B, n)).astype(np.int32) for _ in range(2))
        path, length, _ = nd().nd_tree_accept(dp, i32(tokens), i32(target), m, n_nodes=dc)
        nd().nd_tree_commit(cache, kr, v, path, length)
        wp, wl, _ = tu.accept(parents, counts, tokens, target, None, m)
        np.testing.assert_array_equal(host(path), wp)
        tu.commit(ref, host(kr).astype(np.float32), x[2], wp, wl)
        for f in tu.FIELDS:
            np.testing.assert_array_equal(host(getattr(cache, f)), getattr(ref, f), err_msg=f)


@pytest.mark.parametrize("Hq,Hkv,d,n", [(16, 16, 64, 13), (32, 8, 128, 16), (8, 2, 128, 40)])
def test_a_ctas_many_pairs_are_those_of_calls_of_their_own(Hq, Hkv, d, n):
    """A CTA walks several short (sequence, KV head) pairs, whose queries replace one another while the products before still end;
    a call of few sequences gives each pair a CTA.  Neither splits a pair, so the outputs are equal bit for bit, every time."""
    rng = philox(22800 + d + n)
    ctas = 152 // -(-n * (Hq // Hkv) // 128)      # per block of 128 rows
    B, S, W, window = 4 * ctas // Hkv, 40, 100, 60
    ref = tu.random_cache(rng, B, Hkv, d, S, W)
    depth, _, mask, _ = tu.layout(tu.random_parents(rng, B, n), None, ref.seq_len, 0, window)
    (q, k, v), _ = nodes(rng, B, n, Hq, Hkv, d)
    q[1::2] = -q[::2][:len(q[1::2])]
    cache, dd, dm = tu.device_cache(ref), i32(depth), i32(mask)
    want = torch.empty_like(q)
    few = ctas // Hkv
    for b in range(0, B, few):
        part = slice(b, min(b + few, B))
        one = nd().KVCache(*(getattr(cache, f)[part].contiguous() for f in tu.FIELDS), S, W)
        nd().nd_tree_decode(q[part], one, k[part], v[part], dd[part], dm[part], window, out=want[part])
    for _ in range(20):
        assert torch.equal(nd().nd_tree_decode(q, cache, k, v, dd, dm, window), want)


@pytest.mark.parametrize("Hq,Hkv,d", [(8, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("n,S,W,window", [(5, 40, 50, 6), (12, 5, 200, 150), (70, 60, 300, 290), (40, 200, 9000, 8990)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_slot_that_is_not_finite_reaches_the_rows_that_see_it_alone(Hq, Hkv, d, n, S, W, window, bad):
    """A ring entry that the window leaves behind a few nodes down, and a sink: rows that see one are NaN, channels and lse; the
    others are, bit for bit, what they are where the slots' scales are 0, and within the tolerance of the cache without them."""
    rng = philox(22900 + n + d)
    B, G = 3, Hq // Hkv
    ref = tu.random_cache(rng, B, Hkv, d, S, W, [(S, 2 * W + 7), (S, W), (S, W // 2)])
    parents = tu.random_parents(rng, B, n, reach=2, roots=0)
    parents[:, 0] = -1
    depth, _, mask, see = tu.layout(parents, None, ref.seq_len, 0, window)
    (q, k, v), x = nodes(rng, B, n, Hq, Hkv, d)
    hit, clean, spoilt = np.zeros((B, n, Hq), bool), tu.device_cache(ref), tu.device_cache(ref)
    for b, h, which, group in ((0, 0, "k_scale", 0), (0, 1, "v_scale", 1), (1, 1, "k_scale", 1), (1, 1, "v_scale", 0)):
        rl, rs = int(ref.ring_len[b]), int(ref.ring_start[b])
        e = max(rl - window, 0) + 2                          # at depth 0 among the oldest that the window reaches
        slot = S + (rs + e) % W
        getattr(clean, which)[b, h, slot], getattr(spoilt, which)[b, h, slot] = 0.0, 0.0
        getattr(spoilt, which)[b, h, slot, group] = bad
        hit[b, :, h * G:(h + 1) * G] |= ((depth[b] >= 0) & (depth[b] + rl - e < window))[:, None]
    assert hit[0].any() and (n < 12 or not hit[0].all())
    clean.v_scale[2, 0, S - 1], spoilt.v_scale[2, 0, S - 1] = 0.0, bad    # a sink: all rows of its head
    hit[2, :, :G] = True
    lse, lse0 = (torch.empty((B, Hq, n), dtype=torch.float32, device="cuda") for _ in range(2))
    out = nd().nd_tree_decode(q, spoilt, k, v, i32(depth), i32(mask), window, lse=lse)
    other = nd().nd_tree_decode(q, clean, k, v, i32(depth), i32(mask), window, lse=lse0)
    t = torch.from_numpy(hit).cuda()
    assert torch.isnan(out[t]).all() and torch.isnan(lse.transpose(1, 2)[t]).all()
    assert torch.equal(out[~t], other[~t]) and torch.equal(lse.transpose(1, 2)[~t], lse0.transpose(1, 2)[~t])
    want, _ = tu.decode_rows(x[0], ref, x[1], x[2], depth, see, window)
    assert_close_bf16(host(out)[~hit], want[~hit])


def test_an_appended_infinity_is_left_behind_by_deep_nodes():
    """A token with an infinity goes into the cache as its codec has it; nodes deeper than the window do not see it."""
    rng = philox(22950)
    B, n, Hq, Hkv, d, S, W, window = 1, 12, 8, 2, 64, 20, 40, 6
    ref = tu.random_cache(rng, B, Hkv, d, S, W)
    cache = tu.device_cache(ref)
    bits, x = normal_bf16(rng, (B, 2 * Hkv, d))
    kv = dev_bf16(bits)
    kv[0, 0, 9], kv[0, 3, 40] = float("inf"), float("-inf")              # the key of head 0, the value of head 1
    nd().nd_kv_append_quant(cache, kv[:, :Hkv].contiguous(), kv[:, Hkv:].contiguous())
    oracle.kv_append(ref, x[:, :Hkv], x[:, Hkv:])                        # (finite ones in its place)
    parents = np.arange(n, dtype=np.int32)[None] - 1
    depth, _, mask, see = tu.layout(parents, None, ref.seq_len, 0, window)
    (q, k, v), y = nodes(rng, B, n, Hq, Hkv, d)
    out = host(nd().nd_tree_decode(q, cache, k, v, i32(depth), i32(mask), window))
    want, _ = tu.decode_rows(y[0], ref, y[1], y[2], depth, see, window)
    assert np.isnan(out[0, :window - 1]).all()
    assert_close_bf16(out[0, window - 1:], want[0, window - 1:])


def check_bounds(ref, q, k, v, depth, see, window, zero_seen=0.9):
    """Every channel within its own bound (tree_util.decode_bounds), which a zero output would not be."""
    mask = tu.mask_words(see)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(torch.bfloat16)
    lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32, device="cuda")
    got = host(nd().nd_tree_decode(to(q), tu.device_cache(ref), to(k), to(v), i32(depth), i32(mask), window, lse=lse))
    want, bound, wlse, lse_bound = tu.decode_bounds(q, ref, k, v, depth, see, window)
    assert (np.abs(want) > bound).mean() >= zero_seen
    worst = (np.abs(got - want) / np.maximum(bound, 1e-300)).max()
    assert worst <= 1, worst
    seen = np.isfinite(wlse)
    assert (np.abs(host(lse)[seen] - wlse[seen]) <= lse_bound[seen]).all()
    return got, want, bound


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [8, 24, 80])                       # 4, 2 and 1 copies of the rows
@pytest.mark.parametrize("S,W,grow", [(900, 300, 1 / 300), (900, 300, -1 / 300), (0, 700, 1 / 40), (0, 700, -1 / 40), (0, 700, -1 / 26)])
def test_values_that_grow_or_fall_hold_to_each_channels_bound(d, n, S, W, grow):
    """Value scales by powers of two along the cache, up to 2^26: with S = 0 the nodes' depths reach over the whole ring, so deep
    ones see small values beside large ones that they do not.  Scores are small (keys 2^-6), so that a bound is mostly the
    values': leaving out the first tile's, or a zero output, is far outside it."""
    rng = philox(23000 + d + n)
    B, Hq, Hkv = 1, 4, 2
    ref = tu.random_cache(rng, B, Hkv, d, S, W, [(S, 2 * W + 7)])
    place = np.concatenate([np.arange(S), S + (np.arange(W) - ref.ring_start[0]) % W])   # of a slot, sinks before the ring
    ref.v_scale *= np.exp2(np.floor(grow * place)).astype(np.float32)[None, None, :, None]
    ref.k_scale *= np.float32(2.0 ** -6)
    step, window = (1, 400) if S else (W // n, W)
    depth = step * np.arange(n, dtype=np.int32)[None]
    see = np.eye(n, dtype=bool)[None]
    _, (q, k, v) = nodes(rng, B, n, Hq, Hkv, d)
    v = v if S else v * 2.0 ** np.floor(grow * W)
    got, want, bound = check_bounds(ref, q, k * 2.0 ** -6, v, depth, see, window)
    lost, _, _, _ = tu.decode_bounds(q, ref, k * 2.0 ** -6, v, depth, see, window, drop=range(128))
    if S or grow < 0:
        assert (np.abs(lost - want) > bound)[0, 0].mean() > 0.25


@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_many_sizes_hold_to_each_channels_bound(d):
    """Scales of keys and values that differ from slot to slot; a short cache with as many nodes, whose weights are bf16."""
    rng = philox(23100 + d)
    for S, W, n, spread in ((150, 60, 18, 8), (0, 16, 60, 0), (700, 500, 5, 5)):
        ref = tu.random_cache(rng, 1, 2, d, S, W)
        ref.k_scale *= np.exp2(rng.integers(-6 - spread, -3, ref.k_scale.shape)).astype(np.float32)
        ref.v_scale *= np.exp2(rng.integers(-spread, 3, ref.v_scale.shape)).astype(np.float32)
        depth, _, _, see = tu.layout(tu.random_parents(rng, 1, n), None, ref.seq_len, 0, 99)
        _, (q, k, v) = nodes(rng, 1, n, 8, 2, d)
        check_bounds(ref, q, k * 2.0 ** -3, v, depth, see, 99)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,W", [(40, 30), (5000, 64)])          # whole, split and merged
def test_magnitudes_up_to_2_40(d, S, W):
    """Values up to 2^39.9, alone or behind cached ones that are all 0; queries as large with keys as small."""
    rng = philox(23200 + d)
    n = 7
    for cached, new in ((2.0 ** 37, 2.0 ** 37), (0.0, 2.0 ** 37), (2.0 ** 37, 2.0 ** -60), (2.0 ** -60, 2.0 ** -60)):
        ref = tu.random_cache(rng, 1, 2, d, S, W)
        ref.v_scale *= np.float32(cached)
        ref.k_scale *= np.float32(2.0 ** -43)
        depth, _, _, see = tu.layout(tu.random_parents(rng, 1, n), None, ref.seq_len, 0, 99)
        _, (q, k, v) = nodes(rng, 1, n, 8, 2, d)
        check_bounds(ref, q * 2.0 ** 37, k * 2.0 ** -43, v * new, depth, see, 99, 0.8)
    # scores up to 2^19: a key or two take all the weight
    ref.k_scale *= np.float32(2.0 ** 22)
    ref.v_scale *= np.float32(2.0 ** 60)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(torch.bfloat16)
    got = host(nd().nd_tree_decode(to(q * 2.0 ** 37), tu.device_cache(ref), to(k * 2.0 ** -21), to(v), i32(depth), i32(tu.mask_words(see)), 99))
    top = max(np.abs(oracle.dequant_g32(ref.v_codes, ref.v_scale)).max(), np.abs(v).max())
    assert np.isfinite(got).all() and np.abs(got).max() <= top * (1 + 2.0 ** -7) and (got != 0).mean() > 0.99


@pytest.mark.parametrize("Hq,Hkv,d,n", [(16, 16, 64, 5), (32, 8, 128, 16), (8, 2, 128, 40)])
def test_slots_that_are_not_finite_in_some_of_a_ctas_pairs(Hq, Hkv, d, n):
    """Among many short pairs to a CTA every seventh sequence has such a slot: its head's rows are NaN, all others' outputs are,
    bit for bit, those where the slots' scales are 0."""
    rng = philox(23300 + d + n)
    ctas = 152 // -(-n * (Hq // Hkv) // 128)
    B, S, W, window = 4 * ctas // Hkv, 40, 100, 60
    ref = tu.random_cache(rng, B, Hkv, d, S, W)
    depth, _, mask, _ = tu.layout(tu.random_parents(rng, B, n), None, ref.seq_len, 0, window)
    (q, k, v), _ = nodes(rng, B, n, Hq, Hkv, d)
    clean, spoilt = tu.device_cache(ref), tu.device_cache(ref)
    hit = torch.zeros((B, n, Hq), dtype=torch.bool, device="cuda")
    for b in range(3, B, 7):
        h, slot, which = b % Hkv, (b * 11) % S, ("k_scale", "v_scale")[b % 2]
        getattr(clean, which)[b, h, slot], getattr(spoilt, which)[b, h, slot] = 0.0, float("inf") if b % 3 else float("nan")
        hit[b, :, h * (Hq // Hkv):(h + 1) * (Hq // Hkv)] = True
    dd, dm = i32(depth), i32(mask)
    want = nd().nd_tree_decode(q, clean, k, v, dd, dm, window)
    for _ in range(5):
        got = nd().nd_tree_decode(q, spoilt, k, v, dd, dm, window)
        assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], want[~hit])
