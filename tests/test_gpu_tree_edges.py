"""The tree operators and the rotation at positions at the ends of what they take:
nothing at all, the most rows, many sequences, another stream by argument, threads."""
import threading

import numpy as np
import pytest
import torch

import tree_util as tu
from gpu_util import assert_close_bf16, dev_bf16, host, need_gpu, no_device_errors
from tree_util import i32
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


def nodes(rng, B, n, Hq, Hkv, d):
    bits, x = normal_bf16(rng, (B, n, Hq + 2 * Hkv, d))
    t = dev_bf16(bits)
    return (t[:, :, :Hq].contiguous(), t[:, :, Hq:Hq + Hkv], t[:, :, Hq + Hkv:]), \
        (x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:])


@pytest.mark.parametrize("B,n", [(0, 3), (2, 0), (0, 0)])
def test_nothing_to_do(B, n):
    e = torch.zeros((B, n), dtype=torch.int32, device="cuda")
    x = torch.zeros((B, n, 2, 64), dtype=torch.bfloat16, device="cuda")
    c = nd().KVCache.empty(B, 2, 64, 4, 8)
    depth, pos, mask = nd().nd_tree_layout(e, None, 4)
    assert depth.shape == (B, n) and mask.shape == (B, n, (n + 31) // 32)
    path, length, _ = nd().nd_tree_accept(e, e, e, 2)
    assert path.tolist() == [[-1, -1]] * B and length.tolist() == [0] * B
    assert nd().nd_tree_decode(x, c, x, x, depth, mask, 4).shape == x.shape
    before = [getattr(c, f).clone() for f in tu.FIELDS]
    nd().nd_tree_commit(c, x, x, path, length)
    assert all(torch.equal(getattr(c, f), b) for f, b in zip(tu.FIELDS, before))
    q, k = nd().nd_rope_positions(x, x[:, :, :1], positions=pos)
    assert q.shape == x.shape and k.shape == (B, n, 1, 64)


def test_paths_of_no_tokens_leave_the_cache():
    rng = philox(24000)
    ref = tu.random_cache(rng, 5, 2, 64, 3, 7)
    cache = tu.device_cache(ref)
    (_, k, v), _ = nodes(rng, 5, 4, 2, 2, 64)
    nd().nd_tree_commit(cache, k, v, i32(np.full((5, 3), -1, np.int32)), i32(np.zeros(5, np.int32)))
    for f in tu.FIELDS:
        np.testing.assert_array_equal(host(getattr(cache, f)), getattr(ref, f))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("S,W", [(30, 40), (700, 40)])
def test_the_most_rows(d, S, W):
    """256 nodes of 8 query heads per KV head: 16 row blocks."""
    rng = philox(24100 + d + S)
    ref = tu.random_cache(rng, 2, 2, d, S, W)
    depth, _, mask, see = tu.layout(tu.random_parents(rng, 2, 256), np.array([256, 255], np.int32), ref.seq_len, 0, 50)
    (q, k, v), x = nodes(rng, 2, 256, 16, 2, d)
    want, _ = tu.decode_rows(x[0], ref, x[1], x[2], depth, see, 50)
    assert_close_bf16(host(nd().nd_tree_decode(q, tu.device_cache(ref), k, v, i32(depth), i32(mask), 50)), want)


@pytest.mark.parametrize("Hkv,d", [(1, 64), (3, 128)])
def test_many_sequences(Hkv, d):
    """20 001 sequences of a few slots; every 97th held against the fp64 rows."""
    rng = philox(24200 + d)
    B, n, S, W, window = 20001, 3, 2, 6, 5
    ref = tu.random_cache(rng, B, Hkv, d, S, W, [(S, 2 * W + 1), (0, 0), (1, 3), (S, W)])
    parents = tu.random_parents(rng, B, n)
    counts = rng.integers(0, n + 1, B).astype(np.int32)
    cache, dp, dc = tu.device_cache(ref), i32(parents), i32(counts)
    depth, _, mask = nd().nd_tree_layout(dp, cache.seq_len, window, n_nodes=dc)
    (q, k, v), x = nodes(rng, B, n, 2 * Hkv, Hkv, d)
    out = host(nd().nd_tree_decode(q, cache, k, v, depth, mask, window))
    some = np.arange(0, B, 97)
    part = tu.random_cache(philox(1), len(some), Hkv, d, S, W)
    for f in tu.FIELDS:
        getattr(part, f)[...] = getattr(ref, f)[some]
    wd, _, _, see = tu.layout(parents[some], counts[some], part.seq_len, 0, window)
    want, _ = tu.decode_rows(x[0][some], part, x[1][some], x[2][some], wd, see, window)
    assert_close_bf16(out[some], want)
    tokens, target = (rng.integers(0, 2, (B, n)).astype(np.int32) for _ in range(2))
    path, length, _ = nd().nd_tree_accept(dp, i32(tokens), i32(target), n, n_nodes=dc)
    wp, wl, _ = tu.accept(parents, counts, tokens, target, None, n)
    np.testing.assert_array_equal(host(path), wp)
    nd().nd_tree_commit(cache, k, v, path, length)
    tu.commit(part, x[1][some], x[2][some], wp[some], wl[some])
    for f in tu.FIELDS:
        np.testing.assert_array_equal(host(getattr(cache, f))[some], getattr(part, f), err_msg=f)


def step(rng, seed_cache, stream=None):
    """One step on `stream` (an argument of every call); its outputs."""
    ref, parents, x, tokens, target = seed_cache
    cache = tu.device_cache(ref)
    q, k, v = x
    torch.cuda.current_stream().synchronize()
    depth, pos, mask = nd().nd_tree_layout(parents, cache.seq_len, 30, stream=stream)
    qr, kr = nd().nd_rope_positions(q, k, nd().RopeConfig(), positions=pos, stream=stream)
    out = nd().nd_tree_decode(qr, cache, kr, v, depth, mask, 30, stream=stream)
    path, length, _ = nd().nd_tree_accept(parents, tokens, target, 6, stream=stream)
    nd().nd_tree_commit(cache, kr, v, path, length, stream=stream)
    (stream or torch.cuda.current_stream()).synchronize()
    return [out, path, length] + [getattr(cache, f) for f in tu.FIELDS]


def a_step(rng, B, n, S, W):
    ref = tu.random_cache(rng, B, 2, 64, S, W)
    tokens, target = (i32(rng.integers(0, 2, (B, n)).astype(np.int32)) for _ in range(2))
    return ref, i32(tu.random_parents(rng, B, n)), nodes(rng, B, n, 8, 2, 64)[0], tokens, target


def test_a_stream_given_by_argument():
    rng = philox(24300)
    for B, S in ((3, 20), (1, 4000)):
        job = a_step(rng, B, 19, S, 40)
        want = step(rng, job)
        side = torch.cuda.Stream()
        for got in (step(rng, job, side), step(rng, job, torch.cuda.Stream())):
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_threads():
    """Whole steps from two threads at once, each on a stream of its own and with rotary tables of its own."""
    rng = philox(24400)
    jobs = [a_step(rng, 2, 12, 300, 40), a_step(rng, 5, 33, 10, 64)]
    want = [step(rng, j) for j in jobs]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            side = torch.cuda.Stream()
            for _ in range(20):
                if not all(torch.equal(a, b) for a, b in zip(step(rng, jobs[i], side), want[i])):
                    failed.append(i)
        except Exception as e:  # (an assertion in a thread would be lost)
            failed.append(repr(e))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed


def test_two_rotary_configurations_in_turn():
    """Local and global layers: the table that a thread keeps is that of the configuration it is asked for."""
    rng = philox(24500)
    x = torch.from_numpy(rng.standard_normal((1, 40, 3, 64), dtype=np.float32)).cuda()
    a, b = nd().RopeConfig(), nd().RopeConfig(theta=500000.0, rotary_dim=32, scaling="linear", factor=4.0)
    want = [nd().nd_rope_positions(x, None, c)[0] for c in (a, b)]
    assert not torch.equal(*want)
    for _ in range(3):
        for c, w in zip((a, b), want):
            assert torch.equal(nd().nd_rope_positions(x, None, c)[0], w)


def test_rotary_fields_at_the_end_of_their_range():
    """Frequencies scaled away, or all the same: the rotation is the identity times the magnitude, or plain."""
    rng = philox(24600)
    x = torch.from_numpy(rng.standard_normal((1, 40, 3, 64), dtype=np.float32)).cuda()
    still, _ = nd().nd_rope_positions(x, None, nd().RopeConfig(scaling="linear", factor=3e38))
    assert torch.equal(still, x)
    plain, _ = nd().nd_rope_positions(x, None, nd().RopeConfig())
    # every pair turns more often than `high` over the original length, or less often than `low`
    kept, _ = nd().nd_rope_positions(x, None, nd().RopeConfig(scaling="by_parts", factor=8.0, low=1.0, high=2.0, orig_len=1e38))
    assert torch.equal(kept, plain)
    slow, _ = nd().nd_rope_positions(x, None, nd().RopeConfig(scaling="by_parts", factor=8.0, low=1e38, high=3e38, orig_len=4096.0))
    want, _ = nd().nd_rope_positions(x, None, nd().RopeConfig(scaling="linear", factor=8.0))
    assert torch.equal(slow, want)
