"""Measured cases of the operators around a step that verifies a tree of drafted tokens.

A session's next tokens are drafted as a tree: node i continues its parent's
path, the roots continue the cache.  From the parents come each node's depth,
position and mask of ancestors; queries and keys are rotated at the nodes'
positions; one pass attends from every node to the session's int8 cache (pinned
slots, and the ring entries its window reaches) and to its ancestors; the
longest path that the model's own choices agree with is found, and its keys and
values are quantised into the ring.

Each case names one operator (`op`) and its sizes; `run` computes it in plain
torch operations, or with `own` set through the library's entry points.
"""
import math

import torch

own = False

GROUP = 32                        # channels per scale of the cache
KV_FIELDS = ("k_codes", "v_codes", "k_scale", "v_scale", "sink_len", "ring_start", "ring_len", "seq_len")


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def listed():
    def decode(name, B, n, Hq, Hkv, d, sinks, ring, window, full):
        return dict(name=name, op="tree_decode", B=B, n=n, Hq=Hq, Hkv=Hkv, d=d, sinks=sinks, ring=ring, window=window, full=full)

    def rope(name, B, T, Hq, Hkv, d, dtype, r, interleaved, inverse, scaling, fused, positions):
        return dict(name=name, op="rope", B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, r=r, interleaved=interleaved, inverse=inverse,
                    scaling=scaling, fused=fused, positions=positions)

    def layout(name, B, n, window, full):
        return dict(name=name, op="tree_layout", B=B, n=n, window=window, full=full)

    def accept(name, B, n, path, rooted):
        return dict(name=name, op="tree_accept", B=B, n=n, path=path, rooted=rooted)

    def commit(name, B, n, path, Hkv, d, ring):
        return dict(name=name, op="tree_commit", B=B, n=n, path=path, Hkv=Hkv, d=d, ring=ring)

    return [
        # two sessions with a handful of drafted tokens each over a short context: the latency of a call
        decode("tree_b2_n8", 2, 8, 8, 2, 64, 64, 256, 256, True),
        # ragged: an odd batch of trees of up to 13 nodes, own sinks, part-filled rings, a narrower window, one query head per KV head
        decode("tree_b37_n13_mha", 37, 13, 16, 16, 64, 48, 200, 160, False),
        # the large batch over 1024 pinned slots and a full ring, 16 drafted tokens a session: the caches' bytes
        decode("tree_b128_n16", 128, 16, 32, 8, 128, 1024, 256, 256, True),
        # few sessions over a very long document with large trees: a dense contraction
        decode("tree_b8_n64_s32768", 8, 64, 32, 8, 128, 32768, 256, 256, True),
        # the gradient of a short fp32 prompt's rotation, frequencies scaled by parts
        rope("rope_f32_t512_inverse", 1, 512, 4, 1, 64, "f32", 64, False, True, "by_parts", False, False),
        # a packed batch of prompts, neighbouring channels paired, half of each head, positions of their own, inside one fused projection
        rope("rope_packed_fused", 8, 4096, 32, 8, 128, "bf16", 64, True, False, "linear", True, True),
        # one session's small tree
        layout("layout_b1_n8", 1, 8, 256, True),
        # a large batch of the largest trees, deeper than the window
        layout("layout_b512_n256", 512, 256, 32, False),
        # one session's small tree
        accept("accept_b1_n8", 1, 8, 8, False),
        # a large batch of the largest trees; whether a root holds is up to the model too
        accept("accept_b512_n256", 512, 256, 32, True),
        # 64 small sessions take up to 6 of 16 drafted tokens
        commit("commit_b64_n16", 64, 16, 6, 2, 64, 256),
        # 512 sessions take up to 16 of 64
        commit("commit_b512_n64", 512, 64, 16, 8, 128, 256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree_decode", "tree_decode", "tree_decode", "rope", "rope", "tree_layout", "tree_accept", "tree_commit"])
    Hq, Hkv, d = rng.choice([(8, 2, 64), (16, 16, 64), (4, 1, 64), (32, 8, 128), (8, 8, 128), (16, 2, 128), (12, 4, 64)])
    if op == "tree_decode":
        for _ in range(100):
            B, n, sinks = _log(rng, 1, 128), _log(rng, 1, 128), rng.choice([0, 5, 64, _log(rng, 1, 32768)])
            ring = _log(rng, 1, 384)
            if B * n * Hq * d * (sinks + ring) <= 8 * 64 * 32 * 128 * 33024 and B * Hkv * d * (sinks + ring) <= 128 * 8 * 128 * 2048:
                break
        else:
            B, n, sinks = 4, 16, 64
        return dict(op=op, B=B, n=n, Hq=Hq, Hkv=Hkv, d=d, sinks=sinks, ring=ring, window=_log(rng, 1, 512), full=rng.random() < 0.5)
    if op == "rope":
        T = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(64, 8 * 4096 // T)))
        r = rng.choice([d, d, d // 2, d // 4])
        return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, dtype=rng.choice(["bf16", "f32"]) if B * T * Hq * d <= 4 * 4096 * 32 * 128 else "bf16",
                    r=r, interleaved=rng.random() < 0.5, inverse=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "by_parts"]),
                    fused=rng.random() < 0.5, positions=rng.random() < 0.7)
    B, n = _log(rng, 1, 512), _log(rng, 1, 256)
    if op == "tree_layout":
        return dict(op=op, B=B, n=n, window=_log(rng, 1, 512), full=rng.random() < 0.5)
    if op == "tree_accept":
        return dict(op=op, B=B, n=n, path=_log(rng, 1, 32), rooted=rng.random() < 0.5)
    ring = _log(rng, 1, 384)
    return dict(op=op, B=B, n=min(n, 64), path=min(_log(rng, 1, 16), n, ring), Hkv=Hkv, d=d, ring=ring)


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(g, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int32)


def _quantise(x):
    """The cache codec: per group of 32 channels scale = amax / 127, code = rint(x / scale)."""
    y = x.float().unflatten(-1, (-1, GROUP))
    amax = y.abs().amax(-1)
    scale = amax / 127.0
    code = torch.round(y / torch.where(scale > 0, scale, torch.ones_like(scale)).unsqueeze(-1)).clamp(-127, 127)
    return code.flatten(-2).to(torch.int8), scale


def _cache(g, B, Hkv, d, sinks, ring, full):
    """A cache as appends leave it: N(0,1) tokens through the codec, every ring rotated by its own history."""
    ns = sinks + ring
    kc, ks = _quantise(_normal(g, B, Hkv, ns, d).bfloat16())
    vc, vs = _quantise(_normal(g, B, Hkv, ns, d).bfloat16())
    sink_len = torch.full((B,), sinks, dtype=torch.int32, device="cuda")
    ring_len = torch.full((B,), ring, dtype=torch.int32, device="cuda")
    ring_start = _ints(g, 0, max(ring - 1, 0), B)
    if not full:
        ring_len = _ints(g, 0, ring, B)
        ring_start = torch.where(ring_len < ring, torch.zeros_like(ring_start), ring_start)
        sink_len = _ints(g, 0, sinks, B)
    return dict(k_codes=kc, v_codes=vc, k_scale=ks, v_scale=vs, sink_len=sink_len, ring_start=ring_start,
                ring_len=ring_len, seq_len=sink_len + ring_len + ring_start, sink_cap=sinks, ring_cap=ring)


def _parents(g, B, n):
    """Trees as a drafter grows them: a node continues one of the six nodes before it, now and then the cache itself."""
    i = torch.arange(n, device="cuda", dtype=torch.int32)[None]
    p = (i - _ints(g, 1, 6, B, n)).clamp(min=-1)
    return torch.where(_ints(g, 0, 63, B, n) == 0, torch.full_like(p, -1), p).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    op, B = c["op"], c["B"]
    if op == "rope":
        Hq, Hkv, d, T = c["Hq"], c["Hkv"], c["d"], c["T"]
        dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
        x = _normal(g, B, T, Hq + 2 * Hkv, d).to(dt)
        q, k = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv]
        if not c["fused"]:
            q, k = q.contiguous(), k.contiguous()
        s = dict(case=c, q=q, k=k, positions=None)
        if c["positions"]:  # each row: two packed prompts, the second at an offset of a long session
            cut = torch.randint(0, T + 1, (B, 1), generator=g, device="cuda")
            off = torch.randint(0, 100000, (B, 1), generator=g, device="cuda")
            t = torch.arange(T, device="cuda")[None]
            s["positions"] = torch.where(t < cut, t, t - cut + off).to(torch.int32)
        return s
    n = c["n"]
    if op == "tree_commit":
        Hkv, d, m = c["Hkv"], c["d"], c["path"]
        x = _normal(g, B, n, 3 * Hkv, d).bfloat16()
        # a path: rising node numbers, the first len of them taken
        path = torch.rand(B, n, generator=g, device="cuda").argsort(1)[:, :m].sort(1).values.to(torch.int32).contiguous()
        return dict(case=c, cache=_cache(g, B, Hkv, d, 0, c["ring"], False), k=x[:, :, Hkv:2 * Hkv].contiguous(), v=x[:, :, 2 * Hkv:],
                    path=path, path_len=_ints(g, 0, m, B))
    s = dict(case=c, parents=_parents(g, B, n))
    if op == "tree_layout":
        s["n_nodes"] = None if c["full"] else _ints(g, 0, n, B)
        s["seq_len"] = _ints(g, 0, 100000, B)
        s["base"] = torch.tensor([1024], dtype=torch.int32, device="cuda")
        return s
    if op == "tree_accept":
        s["target"] = _ints(g, 0, 31999, B, n)
        s["root_target"] = _ints(g, 0, 31999, B) if c["rooted"] else None
        of_parent = s["target"].gather(1, s["parents"].clamp(min=0).long())
        if c["rooted"]:
            of_parent = torch.where(s["parents"] < 0, s["root_target"][:, None], of_parent)
        s["tokens"] = torch.where(torch.rand(B, n, generator=g, device="cuda") < 0.8, of_parent, _ints(g, 0, 31999, B, n))
        s["n_nodes"] = _ints(g, max(1, n // 2), n, B)
        return s
    Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
    x = _normal(g, B, n, Hq + 2 * Hkv, d).bfloat16()
    s["n_nodes"] = torch.full((B,), n, dtype=torch.int32, device="cuda") if c["full"] else _ints(g, max(1, n // 2), n, B)
    s["cache"] = _cache(g, B, Hkv, d, c["sinks"], c["ring"], c["full"])
    s["q"], s["k"], s["v"] = x[:, :, :Hq].contiguous(), x[:, :, Hq:Hq + Hkv].contiguous(), x[:, :, Hq + Hkv:]
    s["depth"], _, s["mask"] = _plain_layout(s["parents"], s["n_nodes"], s["cache"]["seq_len"], None, c["window"])
    return s


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------

ROPE = dict(theta=10000.0, factor=4.0, low=1.0, high=32.0, orig_len=4096)


def _dequant(codes, scale):
    return (codes.float().unflatten(-1, (-1, GROUP)) * scale.unsqueeze(-1)).flatten(-2)


def _frequencies(c, dtype=torch.float64):
    r = c["r"]
    f = ROPE["theta"] ** (-2.0 * torch.arange(r // 2, dtype=dtype, device="cuda") / r)
    if c["scaling"] == "linear":
        return f / ROPE["factor"]
    if c["scaling"] == "by_parts":
        turns = ROPE["orig_len"] * f / (2 * math.pi)
        keep = ((turns - ROPE["low"]) / (ROPE["high"] - ROPE["low"])).clamp(0, 1)
        return (1 - keep) * f / ROPE["factor"] + keep * f
    return f


def _magnitude(c):
    return 0.1 * math.log(ROPE["factor"]) + 1.0 if c["scaling"] == "by_parts" else 1.0


def _plain_rope(s):
    c = s["case"]
    r = c["r"]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(c["T"], device="cuda")[None].expand(c["B"], -1)
    angle = pos.double()[..., None, None] * _frequencies(c)
    cos, sin = (angle.cos() * _magnitude(c)).float(), (angle.sin() * _magnitude(c)).float()
    if c["inverse"]:
        sin = -sin

    def turn(x):
        y = x.float().clone()
        if c["interleaved"]:
            a, b = x[..., 0:r:2].float(), x[..., 1:r:2].float()
            y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :r // 2].float(), x[..., r // 2:r].float()
            y[..., :r // 2], y[..., r // 2:r] = a * cos - b * sin, b * cos + a * sin
        return y.to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _ancestors(parents, live):
    """[B, n, n] of 0 and 1: j is i or an ancestor of i (rows and columns of nodes that are not live are 0)."""
    B, n = parents.shape
    j = torch.arange(n, device=parents.device)
    up = ((parents[..., None] == j) & live[:, :, None]).float()
    seen = torch.eye(n, device=parents.device) * live[:, :, None] + up
    for _ in range(max(n - 1, 1).bit_length()):     # paths of up to 2, 4, 8 ... steps
        seen = ((seen @ seen) > 0).float()
    return seen


def _pack(bits):
    """[.., n] of truth values -> int32 words, bit j of word w is element 32 w + j."""
    n = bits.shape[-1]
    words = (n + 31) // 32
    b = torch.nn.functional.pad(bits.long(), (0, 32 * words - n)).unflatten(-1, (words, 32))
    w = (b << torch.arange(32, device=bits.device)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _plain_layout(parents, n_nodes, seq_len, base, window):
    B, n = parents.shape
    i = torch.arange(n, device=parents.device)[None]
    live = (i < n_nodes[:, None]) if n_nodes is not None else torch.ones_like(parents, dtype=torch.bool)
    seen = _ancestors(parents, live)
    depth = torch.where(live, seen.sum(-1).to(torch.int32) - 1, -1)
    near = (seen > 0) & (depth[:, :, None] - depth[:, None] < window)
    start = seq_len + (base if base is not None else 0)
    positions = torch.where(live, start[:, None] + depth, -1).to(torch.int32)
    return depth.to(torch.int32), positions, _pack(near)


def _plain_accept(s):
    c, parents, target, tokens = s["case"], s["parents"].long(), s["target"], s["tokens"]
    B, n, m = c["B"], c["n"], c["path"]
    i = torch.arange(n, device="cuda")[None]
    live = i < s["n_nodes"][:, None]
    root = parents < 0
    if s["root_target"] is None:
        right = root
    else:
        right = root & (tokens == s["root_target"][:, None])
    right = live & (right | (~root & (tokens == target.gather(1, parents.clamp(min=0)))))
    seen = _ancestors(s["parents"], live)
    depth = seen.sum(-1).long() - 1
    agreed = right & ((seen * (~right)[:, None]).sum(-1) == 0) & (depth < m)
    rank = torch.where(agreed, (depth + 1) * n - i, 0)      # deepest first, then the lowest number
    best, at = rank.max(1)
    found = best > 0
    length = torch.where(found, depth.gather(1, at[:, None])[:, 0] + 1, 0)
    on_path = (seen.gather(1, at[:, None, None].expand(-1, -1, n))[:, 0] > 0) & found[:, None]
    # the nodes of the path in order of depth; -1 behind its end
    order = torch.where(on_path, i, n).sort(1).values
    order = torch.nn.functional.pad(order, (0, max(0, m - n)), value=n)[:, :m]
    path = torch.where(order < n, order, -1).to(torch.int32)
    none = s["root_target"] if s["root_target"] is not None else torch.full_like(length, -1)
    following = torch.where(found, target.gather(1, at[:, None])[:, 0], none)
    return dict(path=path, path_len=length.to(torch.int32), next=following.to(torch.int32))


def _plain_commit(s):
    c, cache, path, length = s["case"], s["cache"], s["path"].long(), s["path_len"]
    cap, m = c["ring"], c["path"]
    rs, rl = cache["ring_start"], cache["ring_len"]
    row = torch.arange(c["B"], device="cuda")[:, None]
    t = torch.arange(m, device="cuda")[None]
    slot = torch.remainder(rs[:, None] + rl[:, None] + t, cap).long()
    take = (t < length[:, None])[..., None, None]
    for name, x in (("k", s["k"]), ("v", s["v"])):
        code, scale = _quantise(x[row, path])
        for field, new in ((name + "_codes", code), (name + "_scale", scale)):
            cache[field][row, :, slot] = torch.where(take, new, cache[field][row, :, slot])
    more = rl + length
    rs.copy_(torch.where(more > cap, torch.remainder(rs + more - cap, cap), rs))
    rl.copy_(more.clamp(max=cap))
    cache["seq_len"] += length
    # the newest `path` entries, oldest first; rows behind a short session stay 0
    n = rl.clamp(max=m)
    slot = torch.remainder(rs[:, None] + (rl - n)[:, None] + t, cap).long()
    live = (t < n[:, None])[..., None, None]
    newest = {x: torch.where(live, _dequant(cache[x + "_codes"][row, :, slot], cache[x + "_scale"][row, :, slot]), 0.0).bfloat16()
              for x in ("k", "v")}
    return dict(k=newest["k"], v=newest["v"], ring_start=rs, ring_len=rl, seq_len=cache["seq_len"])


def _unpack(mask, n):
    return ((mask[..., None] >> torch.arange(32, device=mask.device)) & 1).flatten(-2)[..., :n] > 0


def _plain_decode(s):
    c, cache = s["case"], s["cache"]
    B, n, Hq, Hkv, d = c["B"], c["n"], c["Hq"], c["Hkv"], c["d"]
    G, S, W = Hq // Hkv, c["sinks"], c["ring"]
    # [B, n, slots]: the filled sinks, and the ring entries within the window of each node's position
    seen = (torch.arange(S, device="cuda")[None] < cache["sink_len"][:, None])[:, None].expand(-1, n, -1)
    age = torch.remainder(torch.arange(W, device="cuda")[None] - cache["ring_start"][:, None], W)
    rl = cache["ring_len"][:, None]
    back = (rl - age)[:, None] + s["depth"][..., None]      # how far behind the node the entry is
    ring = (age < rl)[:, None] & (back < c["window"])
    live = s["depth"] >= 0
    seen = torch.cat([seen, ring, _unpack(s["mask"], n)], 2) & live[..., None]
    used = torch.cat([torch.arange(S, device="cuda")[None] < cache["sink_len"][:, None], age < rl, live], 1)[:, None, :, None]
    k = torch.cat([_dequant(cache["k_codes"], cache["k_scale"]), s["k"].float().transpose(1, 2)], 2)
    v = torch.cat([_dequant(cache["v_codes"], cache["v_scale"]), s["v"].float().transpose(1, 2)], 2)
    k, v = torch.where(used, k, 0.0), torch.where(used, v, 0.0)
    q = (s["q"].float() * d ** -0.5).view(B, n, Hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, d)
    p = (q @ k.transpose(2, 3)).view(B, Hkv, n, G, -1).masked_fill(~seen[:, None, :, None], -math.inf)
    p = (p - p.amax(-1, keepdim=True).clamp(min=-3e38)).exp()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, n * G, -1) @ v).view(B, Hkv, n, G, d)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 2, 1, 3, 4).reshape(B, n, Hq, d).bfloat16()


# --------------------------------------------------------------------------
# The library's calls
# --------------------------------------------------------------------------

def _kv(s):
    """The library's handle on the cache's tensors, made once per state as a user's program keeps it."""
    import sliding_window_kv_swa_gb300 as nd
    if "kv" not in s:
        c = s["cache"]
        s["kv"] = nd.KVCache(*(c[f] for f in KV_FIELDS), c["sink_cap"], c["ring_cap"])
    return s["kv"]


def _own(s):
    import sliding_window_kv_swa_gb300 as nd
    c, op = s["case"], s["case"]["op"]
    if op == "rope":
        if "rope" not in s:
            s["rope"] = nd.RopeConfig(theta=ROPE["theta"], rotary_dim=c["r"], interleaved=c["interleaved"], inverse=c["inverse"],
                                      scaling=c["scaling"], factor=ROPE["factor"], low=ROPE["low"], high=ROPE["high"],
                                      orig_len=ROPE["orig_len"], magnitude=_magnitude(c))
        return nd.nd_rope_positions(s["q"], s["k"], s["rope"], positions=s["positions"])
    if op == "tree_layout":
        return nd.nd_tree_layout(s["parents"], s["seq_len"], c["window"], n_nodes=s["n_nodes"], pos_base=s["base"])
    if op == "tree_accept":
        path, length, following = nd.nd_tree_accept(s["parents"], s["tokens"], s["target"], c["path"], n_nodes=s["n_nodes"],
                                                    root_target=s["root_target"])
        return dict(path=path, path_len=length, next=following)
    cache = _kv(s)
    if op == "tree_commit":
        nd.nd_tree_commit(cache, s["k"], s["v"], s["path"], s["path_len"])
        if "k_out" not in s:  # the rows behind a short session stay what they were: zeros here, as a padded batch wants them
            s["k_out"], s["v_out"] = (torch.zeros(c["B"], c["path"], c["Hkv"], c["d"], dtype=torch.bfloat16, device="cuda") for _ in range(2))
        k, v, _, _ = nd.nd_kv_cache_read(cache, c["path"], k_out=s["k_out"], v_out=s["v_out"])
        return dict(k=k, v=v, ring_start=cache.ring_start, ring_len=cache.ring_len, seq_len=cache.seq_len)
    if "ws" not in s:
        size = nd.nd_tree_decode_workspace_size(c["B"], c["n"], c["Hq"], c["Hkv"], c["d"], c["sinks"] + c["ring"])
        s["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return nd.nd_tree_decode(s["q"], cache, s["k"], s["v"], s["depth"], s["mask"], c["window"], workspace=s["ws"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "tree_layout":
        return _plain_layout(state["parents"], state["n_nodes"], state["seq_len"], state["base"], state["case"]["window"])
    return {"rope": _plain_rope, "tree_accept": _plain_accept, "tree_commit": _plain_commit, "tree_decode": _plain_decode}[op](state)


def work(case):
    c, op, B = case, case["op"], case["B"]
    if op == "rope":
        channels = B * c["T"] * (c["Hq"] + c["Hkv"]) * c["d"]
        return dict(bytes=channels * 2 * (4 if c["dtype"] == "f32" else 2) + (4 * B * c["T"] if c["positions"] else 0),
                    flops=3 * channels * c["r"] // c["d"])
    n, words = c["n"], (c["n"] + 31) // 32
    if op == "tree_layout":
        return dict(bytes=B * n * (4 + 8 + 4 * words), flops=B * n * words)
    if op == "tree_accept":
        return dict(bytes=B * (12 * n + 4 * c["path"] + 12), flops=B * n)
    Hkv, d = c["Hkv"], c["d"]
    slot = 2 * (d + d // 8)                       # K and V codes and scales of one (slot, KV head)
    if op == "tree_commit":
        taken = B * c["path"] * 0.5
        # each taken token read and stored; the newest `path` rows read back: codes once more, two bf16 rows out
        return dict(bytes=Hkv * (taken * (4 * d + slot) + B * c["path"] * (slot + 4 * d)), flops=4 * taken * Hkv * d)
    fill = 1.0 if c["full"] else 0.5
    nodes = n * (1.0 if c["full"] else 0.75)
    seen = fill * c["sinks"] + min(fill * c["ring"], c["window"])
    return dict(bytes=B * (Hkv * slot * seen + nodes * Hkv * 4 * d + 4 * n * c["Hq"] * d + 4 * n * (1 + words)),
                flops=4 * B * nodes * c["Hq"] * d * (seen + nodes / 2))


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_slots(cache, b, window, depth):
    """The slots of sequence b that a node at this depth sees."""
    sl, rs, rl, sq = (int(cache[f][b]) for f in ("sink_len", "ring_start", "ring_len", "seq_len"))
    here = sq + depth
    return list(range(sl)) + [cache["sink_cap"] + (rs + e) % cache["ring_cap"] for e in range(rl) if here - (sq - rl + e) < window]


def _exact_turn(c, x, pos):
    """The first r channels of each head as complex numbers, turned by pos * f and stretched."""
    r = c["r"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    f = torch.pow(torch.tensor(ROPE["theta"], dtype=torch.float64, device="cuda"), -2 * i / r)
    if c["scaling"] == "linear":
        f = f * (1.0 / ROPE["factor"])
    elif c["scaling"] == "by_parts":
        ramp = torch.clamp((ROPE["orig_len"] * f / (2 * math.pi) - ROPE["low"]) / (ROPE["high"] - ROPE["low"]), 0.0, 1.0)
        f = torch.lerp(f / ROPE["factor"], f, ramp)
    angle = pos.double()[..., None, None] * f * (-1.0 if c["inverse"] else 1.0)
    z = torch.polar(torch.full_like(angle, _magnitude(c)), angle)
    head, tail = x.double()[..., :r], x.double()[..., r:]
    if c["interleaved"]:
        head = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
    else:
        w = torch.complex(head[..., :r // 2].contiguous(), head[..., r // 2:].contiguous()) * z
        head = torch.cat([w.real, w.imag], -1)
    return torch.cat([head, tail], -1)


def exact(case, seed):
    op = case["op"]
    if op in ("tree_layout", "tree_accept"):
        return None                                # whole numbers alone
    s = prepare(case, seed)
    c = s["case"]
    if op == "rope":
        pos = s["positions"]
        if pos is None:
            pos = torch.arange(c["T"], device="cuda").repeat(c["B"], 1)
        return _exact_turn(c, s["q"], pos), _exact_turn(c, s["k"], pos)
    cache = s["cache"]
    if op == "tree_commit":
        m, cap = c["path"], c["ring"]
        out = {x: torch.zeros(c["B"], m, c["Hkv"], c["d"], dtype=torch.float64) for x in ("k", "v")}
        host = {f: cache[f].cpu() for f in KV_FIELDS}
        kv = {x: s[x].cpu().double() for x in ("k", "v")}
        path, length = s["path"].tolist(), s["path_len"].tolist()
        for b in range(c["B"]):
            rs, rl = int(host["ring_start"][b]), int(host["ring_len"][b])
            line = [("slot", (rs + e) % cap) for e in range(rl)] + [("node", j) for j in path[b][:length[b]]]
            for at, (what, j) in enumerate(line[-cap:][-m:]):
                for x in ("k", "v"):
                    if what == "slot":
                        value = host[x + "_codes"][b, :, j].double().unflatten(-1, (-1, GROUP)) * host[x + "_scale"][b, :, j].double()[..., None]
                    else:                          # the stored scale has 32 bits
                        y = kv[x][b, j].unflatten(-1, (-1, GROUP))
                        scale = (y.abs().amax(-1, keepdim=True).float() / 127.0).double()
                        value = torch.round(y / scale.clamp(min=1e-300)).clamp(-127, 127) * scale
                    out[x][b, at] = value.flatten(-2)
        return dict(k=out["k"].cuda(), v=out["v"].cuda(), ring_start=None, ring_len=None, seq_len=None)
    B, n, Hq, Hkv, d = c["B"], c["n"], c["Hq"], c["Hkv"], c["d"]
    G = Hq // Hkv
    parents, count = s["parents"].tolist(), s["n_nodes"].tolist()
    got = torch.zeros(B, n, Hq, d, dtype=torch.float64, device="cuda")
    for b in range(B):                             # one session at a time; nodes of one depth see the same slots
        keys = {x: cache[x + "_codes"][b].double() * cache[x + "_scale"][b].double().repeat_interleave(GROUP, dim=-1) for x in ("k", "v")}
        lines, by_depth = [], {}
        for i in range(count[b]):
            lines.append((lines[parents[b][i]] if parents[b][i] >= 0 else []) + [i])
            by_depth.setdefault(len(lines[i]) - 1, []).append(i)
        for depth, nodes in by_depth.items():
            slots = torch.tensor(_exact_slots(cache, b, c["window"], depth), dtype=torch.long, device="cuda")
            up = torch.tensor([lines[i][-c["window"]:] for i in nodes], device="cuda")       # [nodes, ancestors]
            q = s["q"][b, nodes].double().view(len(nodes), Hkv, G, d) / math.sqrt(d)
            k0, v0 = keys["k"][:, slots], keys["v"][:, slots]
            k1, v1 = s["k"][b].double()[up].transpose(1, 2), s["v"][b].double()[up].transpose(1, 2)  # [nodes, Hkv, ancestors, d]
            a = torch.einsum("nhgd,hsd->nhgs", q, k0)
            p = torch.softmax(torch.cat([a, q @ k1.transpose(2, 3)], -1), -1)
            o = torch.einsum("nhgs,hsd->nhgd", p[..., :len(slots)], v0) + p[..., len(slots):] @ v1
            got[b, nodes] = o.reshape(len(nodes), Hq, d)
    return got
