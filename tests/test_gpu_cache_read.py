"""Reading a cache back: bit for bit the fp32 product code * scale (rounded to
bf16 where asked), in position order, rows behind a sequence left alone."""
import numpy as np
import pytest
import torch

import oracle
from gpu_util import dev, dev_bf16, host, need_gpu, no_device_errors
from workloads import normal_bf16, philox, to_bf16_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()
    yield
    no_device_errors()


def nd():
    import sliding_window_kv_swa_gb300 as m
    return m


def filled(rng, B, Hkv, d, S, W, lens):
    """An oracle cache after lens[b] = (sinks, ring tokens) appends each, and its device twin."""
    ref = oracle.Cache(B, Hkv, d, S, W)
    ns = S + W
    ref.k_codes[...] = rng.integers(-127, 128, (B, Hkv, ns, d))
    ref.v_codes[...] = rng.integers(-127, 128, (B, Hkv, ns, d))
    ref.k_scale[...] = rng.uniform(1e-3, 10, (B, Hkv, ns, d // 32))
    ref.v_scale[...] = rng.uniform(1e-30, 1e20, (B, Hkv, ns, d // 32))
    for b, (sl, n) in enumerate(lens):
        ref.sink_len[b], ref.ring_len[b], ref.seq_len[b] = sl, min(n, W), sl + n
        ref.ring_start[b] = n % W if n > W else 0
    c = nd().KVCache(*(dev(getattr(ref, f)) for f in ("k_codes", "v_codes", "k_scale", "v_scale", "sink_len",
                                                      "ring_start", "ring_len", "seq_len")), S, W)
    return ref, c


def expect(ref, window, n_rows, f32):
    B, Hkv, d = ref.B, ref.Hkv, ref.d
    k = np.full((B, n_rows, Hkv, d), -7.0, np.float32)
    v = np.full((B, n_rows, Hkv, d), -7.0, np.float32)
    pos = np.full((B, n_rows), -1, np.int32)
    length = np.zeros(B, np.int32)
    for b in range(B):
        kpos, sink = oracle.slot_positions(ref, b)
        keep = oracle.decode_keep(int(ref.seq_len[b]) - 1, kpos, sink, window).astype(bool) & (kpos >= 0)
        slots = np.flatnonzero(keep)
        slots = slots[np.argsort(kpos[slots], kind="stable")]
        length[b] = len(slots)
        pos[b, : len(slots)] = kpos[slots]
        for out, codes, scale in ((k, ref.k_codes, ref.k_scale), (v, ref.v_codes, ref.v_scale)):
            x = codes[b][:, slots].astype(np.float32) * np.repeat(scale[b][:, slots], 32, -1)
            out[b, : len(slots)] = x.transpose(1, 0, 2)
    if not f32:
        k, v = to_bf16_bits(k), to_bf16_bits(v)
    return k, v, pos, length


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("d,Hkv,S,W,window,extra", [
    (64, 2, 8, 16, 16, 0), (128, 3, 5, 13, 9, 2), (32, 1, 0, 7, 100, 0), (256, 1, 3, 1, 1, 1), (128, 8, 64, 40, 33, 0)])
def test_read_matches_the_slots(d, Hkv, S, W, window, extra, f32):
    rng = philox(9800 + d + W)
    lens = [(S, 3 * W + 2), (S, W), (S // 2, W // 2), (0, 0), (0, 1), (S, 0)]
    ref, c = filled(rng, len(lens), Hkv, d, S, W, lens)
    n_rows = S + min(W, window) + extra
    dt = torch.float32 if f32 else torch.bfloat16
    k, v = (torch.full((len(lens), n_rows, Hkv, d), -7.0, dtype=dt, device="cuda") for _ in range(2))
    got = nd().nd_kv_cache_read(c, window, k_out=k, v_out=v)
    for g, w, name in zip(got, expect(ref, window, n_rows, f32), ("k", "v", "positions", "lengths")):
        g = g.cpu()
        g = g.view(torch.int16).numpy().view(np.uint16) if g.dtype == torch.bfloat16 else g.numpy()
        if name in "kv":   # a sequence without a key: the rows hold -7 in both
            np.testing.assert_array_equal(g.reshape(-1).view(np.uint16), w.reshape(-1).view(np.uint16), err_msg=name)
        else:
            np.testing.assert_array_equal(g, w, err_msg=name)


def test_bad_metadata_is_flagged_and_skipped():
    rng = philox(9900)
    _, c = filled(rng, 3, 1, 64, 4, 8, [(4, 8)] * 3)
    c.ring_len[0] = 9
    c.ring_start[1] = -1
    k, v = (torch.full((3, 12, 1, 64), -7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _, _, pos, n = nd().nd_kv_cache_read(c, 8, k_out=k, v_out=v)
    torch.cuda.synchronize()
    assert nd().nd_device_errors(clear=True) == 2
    np.testing.assert_array_equal(host(n), [0, 0, 12])
    assert (k[:2] == -7).all() and (v[:2] == -7).all() and (pos[:2] == -1).all()


def test_read_back_and_handed_over_again_is_the_same_cache():
    """Codec values survive the round trip: a prefill's segment into a cache, out of it, into another."""
    B, T, Hkv, d, S, W = 1, 50, 2, 64, 8, 16
    rng = philox(9950)
    kb, _ = normal_bf16(rng, (B, T, Hkv, d))
    vb, _ = normal_bf16(rng, (B, T, Hkv, d))
    sink = np.zeros((B, T), np.uint8)
    sink[:, :S] = 1
    row = torch.zeros(1, dtype=torch.int32, device="cuda")
    one = nd().KVCache.empty(1, Hkv, d, S, W)
    nd().nd_kv_cache_from_prefill(one, dev_bf16(kb), dev_bf16(vb), row, sink=dev(sink))
    k, v, pos, n = nd().nd_kv_cache_read(one, W, dtype=torch.float32)
    assert host(n)[0] == S + W
    np.testing.assert_array_equal(host(pos)[0], list(range(S)) + list(range(T - W, T)))
    # the largest code of a group is 127 exactly, so the same scale comes back out of the fp32 values
    # only where amax / 127 * 127 rounds back to amax; bf16 keeps the comparison to the stored values
    two = nd().KVCache.empty(1, Hkv, d, S, W)
    nd().nd_kv_cache_from_prefill(two, k.bfloat16(), v.bfloat16(), row, sink=dev(np.r_[np.ones(S), np.zeros(W)].astype(np.uint8)[None]))
    k2, v2, pos2, n2 = nd().nd_kv_cache_read(two, W, dtype=torch.float32)
    assert host(n2)[0] == S + W
    # a value is rounded to bf16 (2^-8 of it) and quantised again (half a step of amax / 127)
    for a, b in ((k, k2), (v, v2)):
        amax = a.unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True)
        tol = 2.0 ** -8 * a.unflatten(-1, (-1, 32)).abs() + (1 + 2.0 ** -8) * amax / 254 * (1 + 2.0 ** -8)
        assert ((a - b).unflatten(-1, (-1, 32)).abs() <= tol).all()
