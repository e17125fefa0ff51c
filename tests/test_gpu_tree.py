"""Layout, acceptance and commit of trees of drafted tokens: whole numbers and
codes, equal to the plain forms bit for bit."""
import numpy as np
import pytest
import torch

import tree_util as tu
from gpu_util import dev_bf16, host, need_gpu, no_device_errors
from tree_util import i32
from workloads import normal_bf16, philox

pytestmark = pytest.mark.gpu

CODES = ("k_codes", "v_codes", "k_scale", "v_scale", "sink_len", "ring_start", "ring_len", "seq_len")


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    no_device_errors()


def nd():
    import sliding_window_kv_swa_gb300 as m
    return m


def check_layout(parents, window, n_nodes=None, seq_len=None, base=None):
    opt = lambda a: None if a is None else i32(a)
    b = None if base is None else torch.tensor([base], dtype=torch.int32, device="cuda")
    depth, pos, mask = nd().nd_tree_layout(i32(parents), opt(seq_len), window, n_nodes=opt(n_nodes), pos_base=b)
    want = tu.layout(parents, n_nodes, seq_len, base or 0, window)
    np.testing.assert_array_equal(host(depth), want[0])
    np.testing.assert_array_equal(host(pos), want[1])
    np.testing.assert_array_equal(tu.words(mask), want[2])


@pytest.mark.parametrize("n", [1, 2, 7, 31, 32, 33, 64, 100, 255, 256])
@pytest.mark.parametrize("window", [1, 2, 5, 32, 1000])
def test_layout(n, window):
    rng = philox(20000 + n * 7 + window)
    B = 5
    check_layout(tu.random_parents(rng, B, n), window, rng.integers(0, n + 1, B).astype(np.int32),
                 rng.integers(0, 1 << 20, B).astype(np.int32), 77)


@pytest.mark.parametrize("shape", ["chain", "star", "roots", "binary"])
@pytest.mark.parametrize("n", [1, 33, 256])
def test_layout_of_plain_shapes(shape, n):
    i = np.arange(n)
    parents = {"chain": i - 1, "star": np.where(i > 0, 0, -1), "roots": np.full(n, -1), "binary": (i + 1) // 2 - 1}[shape]
    for window in (1, 31, 256):
        check_layout(np.tile(parents.astype(np.int32), (2, 1)), window)


def test_layout_of_a_large_batch():
    rng = philox(20100)
    check_layout(tu.random_parents(rng, 3001, 9), 4, rng.integers(0, 10, 3001).astype(np.int32))


def test_bad_parents_and_counts_become_padding():
    n = 40
    parents = np.tile(np.arange(n, dtype=np.int32) - 1, (5, 1))
    parents[1, 3] = 3                              # itself
    parents[2, 7] = 2 ** 31 - 1
    parents[3, 39] = -2
    counts = np.array([n, n, n, n, n + 1], np.int32)
    depth, pos, mask = nd().nd_tree_layout(i32(parents), None, 8, n_nodes=i32(counts))
    torch.cuda.synchronize()
    assert nd().nd_device_errors(clear=True) == 2
    want = tu.layout(parents, counts, None, 0, 8)
    np.testing.assert_array_equal(host(depth), want[0])
    np.testing.assert_array_equal(host(pos), want[1])
    np.testing.assert_array_equal(tu.words(mask), want[2])
    assert (host(depth)[1, 3:] == -1).all() and (host(depth)[4] == -1).all()
    target = np.zeros((5, n), np.int32)
    path, length, following = nd().nd_tree_accept(i32(parents), i32(target), i32(target), n, n_nodes=i32(counts))
    torch.cuda.synchronize()
    assert nd().nd_device_errors(clear=True) == 2
    assert host(length).tolist() == [40, 3, 7, 39, 0] and host(following).tolist() == [0, 0, 0, 0, -1]


@pytest.mark.parametrize("n", [1, 2, 13, 32, 65, 256])
@pytest.mark.parametrize("max_path", [1, 3, 40, 300])
@pytest.mark.parametrize("rooted", [False, True])
def test_accept(n, max_path, rooted):
    rng = philox(20200 + n + max_path)
    B = 33
    parents = tu.random_parents(rng, B, n)
    target, tokens = (rng.integers(0, 3, (B, n)).astype(np.int32) for _ in range(2))   # many agree, many ties
    root = rng.integers(0, 3, B).astype(np.int32) if rooted else None
    counts = rng.integers(0, n + 1, B).astype(np.int32)
    got = nd().nd_tree_accept(i32(parents), i32(tokens), i32(target), max_path, n_nodes=i32(counts),
                              root_target=None if root is None else i32(root))
    for g, w in zip(got, tu.accept(parents, counts, tokens, target, root, max_path)):
        np.testing.assert_array_equal(host(g), w)


def test_accept_a_whole_chain_and_ties():
    n = 256
    parents = np.arange(n, dtype=np.int32)[None] - 1
    same = np.full((1, n), -5, np.int32)           # token ids are any int32
    path, length, following = nd().nd_tree_accept(i32(parents), i32(same), i32(same), n)
    assert host(path)[0].tolist() == list(range(n)) and host(length)[0] == n and host(following)[0] == -5
    star = np.full((1, n), -1, np.int32)
    path, length, _ = nd().nd_tree_accept(i32(star), i32(same), i32(same), 2)
    assert host(path)[0].tolist() == [0, -1] and host(length)[0] == 1


def test_accept_without_nodes():
    e = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    root = torch.tensor([4, 9], dtype=torch.int32, device="cuda")
    path, length, following = nd().nd_tree_accept(e, e, e, 3, root_target=root)
    assert host(path).tolist() == [[-1] * 3] * 2 and host(length).tolist() == [0, 0] and host(following).tolist() == [4, 9]


def check_commit(rng, B, n, m, Hkv, d, S, W, lens=None, path=None, length=None, fused=True):
    ref = tu.random_cache(rng, B, Hkv, d, S, W, lens)
    cache = tu.device_cache(ref)
    bits, x = normal_bf16(rng, (B, n, 3 * Hkv, d))
    dx = dev_bf16(bits)
    k, v = dx[:, :, :Hkv], dx[:, :, 2 * Hkv:]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    if path is None:
        path = rng.integers(0, n, (B, m)).astype(np.int32)       # any nodes, the same one twice among them
    if length is None:
        length = rng.integers(0, m + 1, B).astype(np.int32)
    nd().nd_tree_commit(cache, k, v, i32(path), i32(length))
    tu.commit(ref, x[:, :, :Hkv], x[:, :, 2 * Hkv:], path, length)
    for f in CODES:
        np.testing.assert_array_equal(host(getattr(cache, f)), getattr(ref, f), err_msg=f)


@pytest.mark.parametrize("Hkv,d", [(2, 64), (8, 128), (1, 32), (3, 256), (16, 64)])
@pytest.mark.parametrize("B,n,m,S,W", [(1, 1, 1, 0, 1), (3, 16, 6, 4, 9), (5, 64, 16, 0, 16), (2, 8, 40, 3, 7), (70, 5, 3, 1, 64)])
def test_commit(Hkv, d, B, n, m, S, W):
    rng = philox(20300 + B + 10 * n + d)
    check_commit(rng, B, n, m, Hkv, d, S, W, fused=B != 3)
    check_commit(rng, B, n, m, Hkv, d, S, W, lens=[(S, W // 2), (0, 0), (S, 3 * W + 1)])


def test_commit_of_everything_and_nothing():
    rng = philox(20400)
    check_commit(rng, 2, 256, 256, 8, 128, 2, 300, length=np.array([256, 0], np.int32),
                 path=np.tile(np.arange(256, dtype=np.int32), (2, 1)))
    check_commit(rng, 2, 256, 256, 8, 128, 2, 30, length=np.array([256, 31], np.int32))


def test_commit_refuses_bad_paths_and_leaves_the_sequence():
    rng = philox(20500)
    B, n, m, Hkv, d, S, W = 5, 4, 3, 2, 64, 2, 8
    ref = tu.random_cache(rng, B, Hkv, d, S, W)
    ref.ring_start[4] = W                                        # out of range
    cache = tu.device_cache(ref)
    bits, x = normal_bf16(rng, (B, n, 2 * Hkv, d))
    k, v = dev_bf16(bits)[:, :, :Hkv], dev_bf16(bits)[:, :, Hkv:]
    path = np.array([[0, 1, 99], [0, 4, 0], [-1, 0, 0], [0, 1, 2], [0, 0, 0]], np.int32)
    length = np.array([2, 2, 1, 4, 1], np.int32)                 # row 0: the bad node lies behind its end
    nd().nd_tree_commit(cache, k, v, i32(path), i32(length))
    torch.cuda.synchronize()
    assert nd().nd_device_errors(clear=True) == 2
    tu.commit(ref, x[:, :, :Hkv], x[:, :, Hkv:], path, np.array([2, 0, 0, 0, 0]))
    for f in CODES:
        np.testing.assert_array_equal(host(getattr(cache, f)), getattr(ref, f), err_msg=f)


def test_commit_equals_appends_for_any_value():
    """Values beside half-integers, subnormal scales, zeros, infinities and NaN: the codes of nd_kv_append_quant, bit for bit."""
    rng = philox(20450)
    B, n, Hkv, d, W = 2, 12, 3, 128, 16
    bits = rng.integers(0, 1 << 16, (B, n, 2 * Hkv, d)).astype(np.uint16)      # any bf16 at all, one in 256 not finite
    bits[0, 0] = 0
    bits[0, 1] &= 0x803F                                                       # subnormal
    whole = (rng.integers(-127, 128, (n, 2 * Hkv, d)) + 0.5).astype(np.float32)  # quotients on the halves of a scale of 1
    whole[..., ::32] = 127.0
    bits[1] = (whole.view(np.uint32) >> 16).astype(np.uint16)
    x = dev_bf16(bits)
    k, v = x[:, :, :Hkv], x[:, :, Hkv:]
    a, b = (nd().KVCache.empty(B, Hkv, d, 0, W) for _ in range(2))
    path = np.tile(np.arange(n, dtype=np.int32), (B, 1))
    nd().nd_tree_commit(a, k, v, i32(path), i32(np.full(B, n, np.int32)))
    for t in range(n):
        nd().nd_kv_append_quant(b, k[:, t].contiguous(), v[:, t].contiguous())
    for f in CODES:
        x, y = getattr(a, f), getattr(b, f)
        if x.dtype == torch.float32:
            x, y = x.view(torch.int32), y.view(torch.int32)
        assert torch.equal(x, y), f


def test_calls_in_a_graph_and_on_another_stream():
    rng = philox(20600)
    B, n, m, Hkv, d, S, W = 3, 20, 6, 2, 64, 2, 9
    parents = tu.random_parents(rng, B, n)
    ref = tu.random_cache(rng, B, Hkv, d, S, W)
    cache = tu.device_cache(ref)
    bits, x = normal_bf16(rng, (B, n, Hkv, d))
    kv = dev_bf16(bits)
    tokens, target = (rng.integers(0, 2, (B, n)).astype(np.int32) for _ in range(2))
    dp, dt, dg = i32(parents), i32(tokens), i32(target)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        depth, pos, mask = nd().nd_tree_layout(dp, cache.seq_len, 4)
        path, length, following = nd().nd_tree_accept(dp, dt, dg, m)
        nd().nd_tree_commit(cache, kv, kv, path, length)
    for _ in range(3):
        want = tu.layout(parents, None, ref.seq_len, 0, 4)
        graph.replay()
        torch.cuda.synchronize()
        np.testing.assert_array_equal(host(pos), want[1])
        np.testing.assert_array_equal(tu.words(mask), want[2])
        wp, wl, _ = tu.accept(parents, None, tokens, target, None, m)
        np.testing.assert_array_equal(host(path), wp)
        tu.commit(ref, x, x, wp, wl)
        for f in CODES:
            np.testing.assert_array_equal(host(getattr(cache, f)), getattr(ref, f), err_msg=f)
