"""Plain forms of the tree operators (numpy, 64 bits), and trees to try them on."""
import numpy as np
import torch

import oracle
from gpu_util import dev
from workloads import normal_bf16, philox

FIELDS = ("k_codes", "v_codes", "k_scale", "v_scale", "sink_len", "ring_start", "ring_len", "seq_len")


def device_cache(ref):
    import sliding_window_kv_swa_gb300 as m
    return m.KVCache(*(dev(getattr(ref, f)) for f in FIELDS), ref.sink_cap, ref.ring_cap)


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


def random_parents(rng, B, n, reach=4, roots=0.1):
    """Node i continues one of the `reach` nodes before it, or (a share of `roots`) the cache."""
    i = np.arange(n)[None]
    p = np.maximum(i - rng.integers(1, reach + 1, (B, n)), -1)
    return np.where(rng.random((B, n)) < roots, -1, p).astype(np.int32)


def layout(parents, n_nodes=None, seq_len=None, base=0, window=1 << 30):
    B, n = parents.shape
    words = (n + 31) // 32
    depth, pos = np.full((B, n), -1, np.int32), np.full((B, n), -1, np.int32)
    see = np.zeros((B, n, n), bool)
    for b in range(B):
        lines = {}
        for i in range(n if n_nodes is None else (n_nodes[b] if 0 <= n_nodes[b] <= n else 0)):
            up = int(parents[b, i])
            if up == -1:
                lines[i] = [i]
            elif up in lines:                      # an earlier node that is one
                lines[i] = lines[up] + [i]
            if i in lines:
                depth[b, i] = len(lines[i]) - 1
                pos[b, i] = (0 if seq_len is None else seq_len[b]) + base + depth[b, i]
                see[b, i, lines[i][-window:]] = True
    bits = np.zeros((B, n, words * 32), np.uint64)
    bits[..., :n] = see
    mask = (bits.reshape(B, n, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return depth, pos, mask, see


def decode_rows(q, ref, k, v, depth, see, window):
    """fp64 attention of every node: out [B, n, Hq, d], lse [B, Hq, n]."""
    B, n, Hq, d = q.shape
    Hkv = ref.Hkv
    G = Hq // Hkv
    out, lse = np.zeros((B, n, Hq, d)), np.full((B, Hq, n), -np.inf)
    for b in range(B):
        kc = oracle.dequant_g32(ref.k_codes[b], ref.k_scale[b]).astype(np.float64)
        vc = oracle.dequant_g32(ref.v_codes[b], ref.v_scale[b]).astype(np.float64)
        sl, rs, rl, sq = (int(getattr(ref, f)[b]) for f in ("sink_len", "ring_start", "ring_len", "seq_len"))
        cap = max(ref.ring_cap, 1)
        ring = np.array([ref.sink_cap + (rs + e) % cap for e in range(rl)], int)
        at = np.array([sq - rl + e for e in range(rl)], int)
        for i in range(n):
            if depth[b, i] < 0:
                continue
            p = sq + int(depth[b, i])
            slots = np.concatenate([np.arange(sl), ring[p - at < window]]).astype(int)
            nodes = np.array([j for j in range(n) if see[b, i, j] and depth[b, j] >= 0], int)
            if not len(slots) and not len(nodes):
                continue
            for h in range(Hkv):
                kk = np.concatenate([kc[h, slots], k[b, nodes, h]])
                vv = np.concatenate([vc[h, slots], v[b, nodes, h]])
                s = q[b, i, h * G:(h + 1) * G] @ kk.T / np.sqrt(d)
                m = s.max(-1, keepdims=True)
                e = np.exp(s - m)
                z = e.sum(-1, keepdims=True)
                out[b, i, h * G:(h + 1) * G] = e @ vv / z
                lse[b, h * G:(h + 1) * G, i] = (m + np.log(z))[:, 0]
    return out, lse


def mask_words(see):
    """The layout's mask of a truth table [B, n, n]."""
    B, n, _ = see.shape
    bits = np.zeros((B, n, (n + 31) // 32 * 32), np.uint64)
    bits[..., :n] = see
    return (bits.reshape(B, n, -1, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)


def floor_log2(x):
    return np.frexp(x)[1] - 1


def decode_bounds(q, ref, k, v, depth, see, window, drop=()):
    """decode_rows with a bound for every output channel and lse, from the precision that nd_tree_decode states:
      a key of the cache is off by 2^-10 of itself or 2^-21 of the largest of its 32 slots, a value likewise;
      a cached slot's weight is off by 2^-11 of itself or 2^(k-32) of the row's largest, 2^k the power of two by which the largest
      value scale up to its tile exceeds the largest of its 32; a node's by 2^-8 of itself; the sums by what fp32 loses.
    A weight is off by its score's error s besides (a factor of e^s).  With w the weights over their sum Z, numerator N = sum w v:
    |out - N| <= sum |dw| |v| + w |dv| + |N| |dZ|, over 1 - |dZ|, plus the rounding to bf16, 2^-8.
    `drop`: slots (sinks, then ring entries from the oldest that is seen at depth 0) whose values are left out, as a mistake would."""
    B, n, Hq, d = q.shape
    G = Hq // ref.Hkv
    out, bound = np.zeros((B, n, Hq, d)), np.zeros((B, n, Hq, d))
    lse, lse_bound = np.full((B, Hq, n), -np.inf), np.zeros((B, Hq, n))
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    for b in range(B):
        sl, rs, rl = (int(getattr(ref, f)[b]) for f in ("sink_len", "ring_start", "ring_len"))
        nv = min(rl, window - 1)
        slots = np.concatenate([np.arange(sl), ref.sink_cap + (rs + rl - nv + np.arange(nv)) % max(ref.ring_cap, 1)]).astype(int)
        order = np.concatenate([np.arange(sl), np.arange(nv)]).astype(int)     # place in its region
        region = np.concatenate([np.zeros(sl, int), np.ones(nv, int)])
        tile = region * (ref.sink_cap // 128 + 2) + order // 128
        group = region * (ref.sink_cap // 32 + 8) + order // 32
        for h in range(ref.Hkv):
            kc = oracle.dequant_g32(ref.k_codes[b, h, slots], ref.k_scale[b, h, slots]).astype(np.float64)
            vc = oracle.dequant_g32(ref.v_codes[b, h, slots], ref.v_scale[b, h, slots]).astype(np.float64)
            most = lambda a, g: np.array([a[g == x].max() for x in g]) if len(a) else a
            vs = ref.v_scale[b, h, slots].astype(np.float64).max(-1) if len(slots) else np.zeros(0)
            top = np.array([vs[tile <= t].max() for t in tile]) if len(slots) else vs
            mine = most(vs, group)
            ratio = np.where(mine > 0, 2.0 ** (floor_log2(np.maximum(top, 1e-300)) - floor_log2(np.maximum(mine, 1e-300))), 1.0)
            dk = np.maximum(2.0 ** -10 * np.abs(kc), 2.0 ** -21 * most(np.abs(kc).max(-1), group)[:, None]) if len(slots) else kc
            dv = np.maximum(2.0 ** -10 * np.abs(vc), 2.0 ** -21 * most(np.abs(vc).max(-1), group)[:, None]) if len(slots) else vc
            alive = np.nonzero(depth[b] >= 0)[0]
            kk, vv = np.concatenate([kc, k[b, alive, h]]), np.concatenate([vc, v[b, alive, h]])
            dk, dv = np.concatenate([dk, 0 * k[b, alive, h]]), np.concatenate([dv, 0 * v[b, alive, h]])
            cached = np.arange(len(kk)) < len(slots)
            ratio = np.concatenate([ratio, np.ones(len(alive))])
            for i in alive:
                sees = np.concatenate([(region == 0) | (int(depth[b, i]) + nv - order < window), see[b, i, alive]])
                if not sees.any():
                    continue
                x = q[b, i, h * G:(h + 1) * G]
                s = np.where(sees, x @ kk.T / np.sqrt(d), -np.inf)
                # fp32: d products and sums, the factor, the exponent's argument
                ds = (np.abs(x) @ dk.T + d * 2.0 ** -23 * (np.abs(x) @ np.abs(kk).T)) / np.sqrt(d)
                m = s.max(-1, keepdims=True)
                ds = np.where(sees, ds + 2.0 ** -22 * (1 + np.abs(np.where(sees, s, 0)) + np.abs(m)), 0)
                w = np.exp(s - m)
                z = w.sum(-1, keepdims=True)
                big = np.expm1(ds)
                dw = w * big + w * (1 + big) * np.where(cached, 2.0 ** -11, 2.0 ** -8) + \
                    np.where(sees & cached, 2.0 ** -32 * ratio * np.exp(ds.max(-1, keepdims=True)), 0)
                fp32 = len(kk) * 2.0 ** -23
                dz = (w * big).sum(-1, keepdims=True) / z + fp32
                assert dz.max() < 0.5
                left = np.ones(len(kk))
                left[list(drop)] = 0
                o = (w * left) @ vv / z
                num = (dw @ (np.abs(vv) + dv) + w @ (dv + fp32 * np.abs(vv))) / z
                err = (num + np.abs(o) * dz) / (1 - dz)
                at = slice(h * G, (h + 1) * G)
                out[b, i, at], bound[b, i, at] = o, err + 2.0 ** -8 * (np.abs(o) + err)
                lse[b, at, i], lse_bound[b, at, i] = (m + np.log(z))[:, 0], (dz / (1 - dz))[:, 0] + 2.0 ** -20
    return out, bound, lse, lse_bound


def accept(parents, n_nodes, tokens, target, root_target, max_path):
    B, n = parents.shape
    path, length, following = np.full((B, max_path), -1, np.int32), np.zeros(B, np.int32), np.full(B, -1, np.int32)
    for b in range(B):
        best, lines = [], {}
        for i in range(n if n_nodes is None else (n_nodes[b] if 0 <= n_nodes[b] <= n else 0)):
            up = int(parents[b, i])
            if up == -1:
                if root_target is None or tokens[b, i] == root_target[b]:
                    lines[i] = [i]
            elif up in lines and tokens[b, i] == target[b, up]:
                lines[i] = lines[up] + [i]
            if i in lines and len(best) < len(lines[i]) <= max_path:
                best = lines[i]
        path[b, :len(best)], length[b] = best, len(best)
        following[b] = target[b, best[-1]] if best else -1 if root_target is None else root_target[b]
    return path, length, following


def commit(ref, k, v, path, length):
    """`length` single appends of the path's nodes, sequence by sequence (k, v fp32 [B, n, Hkv, d])."""
    for b in range(ref.B):
        one = oracle.Cache(1, ref.Hkv, ref.d, ref.sink_cap, ref.ring_cap)
        for f in FIELDS:
            getattr(one, f)[...] = getattr(ref, f)[b:b + 1]
        for j in path[b, :length[b]]:
            oracle.kv_append(one, k[b:b + 1, j], v[b:b + 1, j])
        for f in FIELDS:
            getattr(ref, f)[b] = getattr(one, f)[0]


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int32)).cuda()


def words(t):
    return t.cpu().numpy().view(np.uint32)


__all__ = ["philox", "normal_bf16"]
