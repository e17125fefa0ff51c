"""The operators at sizes and in uses that stand apart from the rest: caches
without a ring, a very large batch, two threads.  Against plain torch in 64
bits; attention outputs within max-abs 2e-2 and mean-abs 2e-3 as everywhere."""
import threading

import pytest
import torch

from gpu_util import assert_close_bf16, dev_bf16, host, need_gpu, no_device_errors
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


def fill(cache, seed, lens=None):
    """Random codes and scales of tokens of size 1; every sink and ring slot filled, or lens = (sinks, ring)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for codes, scale in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
        codes.copy_(torch.randint(-127, 128, codes.shape, generator=g, device="cuda", dtype=torch.int8))
        scale.copy_(torch.rand(scale.shape, generator=g, device="cuda") * 0.01 + 0.005)
    s, r = (cache.sink_cap, cache.ring_cap) if lens is None else lens
    cache.sink_len.fill_(s)
    cache.ring_len.fill_(r)
    cache.seq_len.fill_(s + r)
    return cache


def values(codes, scale):
    return (codes.double().unflatten(-1, (-1, 32)) * scale.double().unsqueeze(-1)).flatten(-2)


def attention(q, prefix, cache, L, chunk=4096):
    """[B, Hq, d] in 64 bits: the prefix's first L slots and every slot of the cache (all filled)."""
    B, Hq, d = q.shape
    Hkv = cache.k_codes.shape[1]
    kp, vp = (values(c, s)[0, :, :L] for c, s in ((prefix.k_codes, prefix.k_scale), (prefix.v_codes, prefix.v_scale)))
    out = []
    for b in range(0, B, chunk):
        x = q[b:b + chunk].double().unflatten(1, (Hkv, -1))
        ko, vo = (values(c[b:b + chunk], s[b:b + chunk]) for c, s in ((cache.k_codes, cache.k_scale),
                                                                      (cache.v_codes, cache.v_scale)))
        s = torch.cat([torch.einsum("bhgc,hjc->bhgj", x, kp), torch.einsum("bhgc,bhjc->bhgj", x, ko)], -1) / d ** 0.5
        p = s.softmax(-1)
        o = torch.einsum("bhgj,hjc->bhgc", p[..., :L], vp) + torch.einsum("bhgj,bhjc->bhgc", p[..., L:], vo)
        out.append(o.flatten(1, 2))
    return torch.cat(out)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,sinks", [(2, 1), (5, 40), (40, 33)])
@pytest.mark.parametrize("L", [70, 700])
def test_caches_without_a_ring(d, B, sinks, L):
    """Sink appends into a cache of sinks alone, its decode over a shared prefix, and its read-back."""
    rng = philox(12000 + d + sinks + L)
    Hq, Hkv = 8, 2
    prefix, own = fill(nd().KVCache.empty(1, Hkv, d, L, 0), 1), nd().KVCache.empty(B, Hkv, d, sinks, 0)
    for i in range(sinks):
        x = dev_bf16(normal_bf16(rng, (B, Hq + 2 * Hkv, d))[0])
        q = nd().nd_qk_norm_rope_append(x[:, :Hq], own, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], rope_theta=10000.0, to_sink=True)
    assert (own.sink_len == sinks).all() and (own.seq_len == sinks).all()
    out = nd().nd_shared_prefix_decode(q, prefix, own, 1)
    assert_close_bf16(host(out), attention(q, prefix, own, L).cpu().numpy())
    k, v, pos, n = nd().nd_kv_cache_read(own, 1, dtype=torch.float32)
    assert (n == sinks).all() and torch.equal(pos, torch.arange(sinks, device="cuda", dtype=torch.int32).expand(B, -1))
    assert torch.equal(k, values(own.k_codes, own.k_scale).float().transpose(1, 2).contiguous())
    assert torch.equal(v, values(own.v_codes, own.v_scale).float().transpose(1, 2).contiguous())


@pytest.mark.parametrize("d,Hq,L", [(64, 1, 600), (128, 3, 5), (64, 8, 130)])
def test_very_many_sequences(d, Hq, L):
    """More sequences than a 16-bit grid dimension holds, each with a handful of slots."""
    B, W = 70001, 5
    prefix, own = fill(nd().KVCache.empty(1, 1, d, L, 0), 2), fill(nd().KVCache.empty(B, 1, d, 0, W), 3, (0, W - 1))
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(B, Hq + 2, d, generator=g, device="cuda").bfloat16()
    q = nd().nd_qk_norm_rope_append(x[:, :Hq], own, x[:, Hq:Hq + 1], x[:, Hq + 1:], rope_theta=10000.0)
    assert (own.ring_len == W).all()
    want, _ = nd().nd_qk_norm_rope(x[:, None, :Hq], None, rope_theta=10000.0,
                                   positions=torch.full((B, 1), W - 1, dtype=torch.int32, device="cuda"))
    assert torch.equal(q, want[:, 0])
    out = nd().nd_shared_prefix_decode(q, prefix, own, W)
    err = (out.double() - attention(q, prefix, own, L)).abs()
    assert err.max() <= 2e-2 and err.mean() <= 2e-3
    with pytest.raises(nd().NDError):
        nd().nd_kv_cache_read(own, W)


def test_two_threads_with_streams_of_their_own():
    """The same prefix and calls of other shapes at once, without an output or a workspace given."""
    prefix = fill(nd().KVCache.empty(1, 8, 128, 900, 0), 5)
    jobs, wants = [], []
    for i, (B, Hq) in enumerate(((20, 32), (3, 64))):
        own = fill(nd().KVCache.empty(B, 8, 128, 0, 48), 6 + i)
        q = torch.randn(B, Hq, 128, device="cuda").bfloat16()
        jobs.append((q, own, torch.cuda.Stream()))
        wants.append((nd().nd_shared_prefix_decode(q, prefix, own, 48), nd().nd_qk_norm_rope(q[:, None], None, eps=1e-6)[0]))
    torch.cuda.synchronize()
    bad = []

    def work(i):
        q, own, stream = jobs[i]
        for _ in range(30):
            if i:   # the stream as an argument
                out = nd().nd_shared_prefix_decode(q, prefix, own, 48, stream=stream)
                y = nd().nd_qk_norm_rope(q[:, None], None, eps=1e-6, stream=stream)[0]
            else:
                with torch.cuda.stream(stream):
                    out = nd().nd_shared_prefix_decode(q, prefix, own, 48)
                    y = nd().nd_qk_norm_rope(q[:, None], None, eps=1e-6)[0]
            stream.synchronize()
            with torch.cuda.stream(stream):
                if not (torch.equal(out, wants[i][0]) and torch.equal(y, wants[i][1])):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
