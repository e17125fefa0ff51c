"""Measured cases of the operators around a batch that shares one pinned prefix.

Many sessions that carry the same tool definitions keep them once, in an int8
cache of one row, and each session keeps its own ring of recent tokens.  One
decode step normalises and rotates each head's query and key, quantises the
key and value into the session's ring, and attends to the shared prefix (once
for the whole batch) and to the session's own slots.  Before it stands the
same normalisation and rotation over a prefill; beside it, reading a cache
back into the layout a prefill uses.

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
    def decode(name, B, Hq, Hkv, d, prefix, prefix_cap, sinks, ring, window, full):
        return dict(name=name, op="shared_decode", B=B, Hq=Hq, Hkv=Hkv, d=d, prefix=prefix, prefix_cap=prefix_cap,
                    sinks=sinks, ring=ring, window=window, full=full)

    def norm(name, B, T, Hq, Hkv, d, dtype, fused, positions, theta):
        return dict(name=name, op="norm_rope", B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, fused=fused,
                    positions=positions, theta=theta)

    def append(name, B, Hq, Hkv, d, ring, base, fused):
        return dict(name=name, op="norm_append", B=B, Hq=Hq, Hkv=Hkv, d=d, ring=ring, base=base, fused=fused, theta=10000.0)

    def read(name, B, Hkv, d, sinks, ring, window, dtype, full):
        return dict(name=name, op="cache_read", B=B, Hkv=Hkv, d=d, sinks=sinks, ring=ring, window=window, dtype=dtype, full=full)

    return [
        # two sessions over a short tool list: the latency of a call
        decode("shared_b2_p64", 2, 8, 2, 64, 64, 64, 0, 256, 256, True),
        # a node serving 64 small sessions over a prompt of a few thousand tokens
        decode("shared_b64_d64_p4096", 64, 8, 2, 64, 4096, 4096, 0, 256, 256, True),
        # ragged: odd batch, a prefix that ends inside a tile of a larger region, own sinks, part-filled rings, a narrower window
        decode("shared_b37_mha_p4097", 37, 16, 16, 64, 4097, 4200, 48, 200, 160, False),
        # few sessions over a very long document: the prefix is read from memory once
        decode("shared_b4_p65536", 4, 32, 8, 128, 65536, 65536, 0, 256, 256, True),
        # the large batch whose 1024 pinned slots are the same for every session
        decode("shared_b512_p1024", 512, 32, 8, 128, 1024, 1024, 0, 256, 256, True),
        # many sessions over a long document: a dense contraction
        decode("shared_b128_p32768", 128, 32, 8, 128, 32768, 32768, 0, 256, 256, True),
        # a short fp32 prompt
        norm("norm_rope_f32_t512", 1, 512, 4, 1, 64, "f32", False, False, 10000.0),
        # a packed batch of prompts, each position its own, q and k inside one fused projection
        norm("norm_rope_packed_fused", 8, 4096, 32, 8, 128, "bf16", True, True, 10000.0),
        # one token of each of 64 sessions
        append("norm_append_b64", 64, 8, 2, 64, 256, 1000, False),
        # one token of each of 512 sessions behind a long prefix, straight from a fused projection
        append("norm_append_b512", 512, 32, 8, 128, 256, 100000, True),
        # one evicted session comes back as bf16
        read("cache_read_b1", 1, 2, 64, 64, 256, 256, "bf16", True),
        # all rows of a packed prefill's handoff, part of them short
        read("cache_read_b36", 36, 8, 128, 512, 256, 256, "bf16", False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["shared_decode", "shared_decode", "shared_decode", "norm_rope", "norm_append", "cache_read"])
    Hq, Hkv, d = rng.choice([(8, 2, 64), (16, 16, 64), (4, 1, 64), (32, 8, 128), (8, 8, 128), (16, 2, 128), (12, 4, 64)])
    if op == "shared_decode":
        for _ in range(100):
            B, prefix = _log(rng, 1, 512), _log(rng, 1, 65536)
            if B * Hq * prefix * d <= 128 * 32 * 32768 * 128:
                break
        else:
            B, prefix = 16, 1024
        ring = _log(rng, 1, 384)
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, d=d, prefix=prefix, prefix_cap=prefix + rng.choice([0, 0, 1, 37, 128]),
                    sinks=rng.choice([0, 0, 7, 64]), ring=ring, window=_log(rng, 1, 512), full=rng.random() < 0.5)
    if op == "norm_rope":
        T = _log(rng, 1, 4096)
        B = _log(rng, 1, max(1, min(64, 8 * 4096 // T)))
        return dict(op=op, B=B, T=T, Hq=Hq, Hkv=Hkv, d=d, dtype=rng.choice(["bf16", "f32"]) if B * T * Hq * d <= 4 * 4096 * 32 * 128 else "bf16",
                    fused=rng.random() < 0.5, positions=rng.random() < 0.5, theta=rng.choice([10000.0, 500000.0]))
    if op == "norm_append":
        return dict(op=op, B=_log(rng, 1, 512), Hq=Hq, Hkv=Hkv, d=d, ring=_log(rng, 1, 384), base=_log(rng, 1, 1 << 20),
                    fused=rng.random() < 0.5, theta=rng.choice([10000.0, 500000.0]))
    sinks, ring = rng.choice([0, 5, 64, 512]), _log(rng, 1, 384)
    return dict(op=op, B=_log(rng, 1, 36), Hkv=Hkv if Hkv < 16 else 8, d=d, sinks=sinks, ring=ring, window=_log(rng, 1, 512),
                dtype=rng.choice(["bf16", "f32"]), full=rng.random() < 0.5)


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _quantise(x):
    """The cache codec: per group of 32 channels scale = amax / 127, code = rint(x / scale)."""
    y = x.float().unflatten(-1, (-1, GROUP))
    amax = y.abs().amax(-1)
    scale = amax / 127.0
    code = torch.round(y / torch.where(scale > 0, scale, torch.ones_like(scale)).unsqueeze(-1)).clamp(-127, 127)
    return code.flatten(-2).to(torch.int8), scale


def _cache(g, B, Hkv, d, sinks, ring, full, prefix=None):
    """A cache as appends leave it: N(0,1) tokens through the codec, every ring rotated by its own history."""
    ns = sinks + ring
    kc, ks = _quantise(_normal(g, B, Hkv, ns, d).bfloat16())
    vc, vs = _quantise(_normal(g, B, Hkv, ns, d).bfloat16())
    i32 = dict(dtype=torch.int32, device="cuda")

    def ints(lo, hi):
        return torch.randint(lo, hi + 1, (B,), generator=g, **i32)

    sink_len = torch.full((B,), sinks if prefix is None else prefix, **i32)
    ring_len = torch.full((B,), ring, **i32)
    ring_start = ints(0, max(ring - 1, 0)) if ring else torch.zeros(B, **i32)
    if not full:
        ring_len = ints(0, ring)
        ring_start = torch.where(ring_len < ring, torch.zeros_like(ring_start), ring_start)
        if prefix is None:
            sink_len = ints(0, sinks)
    return dict(k_codes=kc, v_codes=vc, k_scale=ks, v_scale=vs, sink_len=sink_len, ring_start=ring_start,
                ring_len=ring_len, seq_len=sink_len + ring_len + ring_start, sink_cap=sinks, ring_cap=ring)


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    op, Hkv, d = c["op"], c["Hkv"], c["d"]
    if op == "shared_decode":
        return dict(case=c, q=_normal(g, c["B"], c["Hq"], d).bfloat16(),
                    prefix=_cache(g, 1, Hkv, d, c["prefix_cap"], 0, True, c["prefix"]),
                    cache=_cache(g, c["B"], Hkv, d, c["sinks"], c["ring"], c["full"]))
    if op == "cache_read":
        return dict(case=c, cache=_cache(g, c["B"], Hkv, d, c["sinks"], c["ring"], c["full"]))
    Hq, B = c["Hq"], c["B"]
    lead = (B, c["T"]) if op == "norm_rope" else (B,)
    dt = torch.float32 if c.get("dtype") == "f32" else torch.bfloat16
    heads = Hq + 2 * Hkv
    x = (_normal(g, *lead, heads, d) * 1.5 + 0.1).to(dt)
    q, k, v = x[..., :Hq, :], x[..., Hq:Hq + Hkv, :], x[..., Hq + Hkv:, :]
    if not c["fused"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    s = dict(case=c, q=q, k=k, v=v, wq=1.0 + 0.2 * _normal(g, d), wk=1.0 + 0.2 * _normal(g, d))
    if op == "norm_rope":
        s["positions"] = None
        if c["positions"]:  # each row: two packed prompts, the second at an offset of a long session
            T = c["T"]
            cut = torch.randint(0, T + 1, (B, 1), generator=g, device="cuda")
            off = torch.randint(0, 100000, (B, 1), generator=g, device="cuda")
            t = torch.arange(T, device="cuda")[None]
            s["positions"] = torch.where(t < cut, t, t - cut + off).to(torch.int32)
        return s
    s["cache"] = _cache(g, B, Hkv, d, 0, c["ring"], False)
    s["base"] = torch.tensor([c["base"]], dtype=torch.int32, device="cuda")
    return s


# --------------------------------------------------------------------------
# Plain forms
# --------------------------------------------------------------------------

EPS = 1e-6


def _dequant(codes, scale):
    return (codes.float().unflatten(-1, (-1, GROUP)) * scale.unsqueeze(-1)).flatten(-2)


def _visible(cache, window):
    """[B, slots]: the filled sinks, and the ring entries that the window reaches."""
    S, W = cache["sink_cap"], cache["ring_cap"]
    dev = cache["sink_len"].device
    seen = torch.arange(S, device=dev)[None] < cache["sink_len"][:, None]
    if not W:
        return seen
    age = torch.remainder(torch.arange(W, device=dev)[None] - cache["ring_start"][:, None], W)
    n = cache["ring_len"].clamp(max=window)
    first = (cache["ring_len"] - n)[:, None]
    return torch.cat([seen, (age >= first) & (age < cache["ring_len"][:, None])], 1)


def _norm_rope(x, w, pos, theta):
    """x [..., heads, d] at positions pos [...]: RMS norm of each head with weights, then the rotation."""
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    half = x.shape[-1] // 2
    freq = theta ** (-torch.arange(half, dtype=torch.float64, device=x.device) / half)
    a = pos.double()[..., None, None] * freq
    c, s = a.cos().float(), a.sin().float()
    lo, hi = y[..., :half], y[..., half:]
    return torch.cat([lo * c - hi * s, hi * c + lo * s], -1)


def _plain_shared_decode(s):
    c, q, pre, own_c = s["case"], s["q"].float(), s["prefix"], s["cache"]
    B, Hq, d = q.shape
    Hkv = c["Hkv"]
    G = Hq // Hkv
    q = q.view(B, Hkv, G, d) * d ** -0.5
    # the prefix: one product for the rows of all sessions
    seen_p = torch.arange(pre["sink_cap"], device=q.device) < pre["sink_len"][0]
    kp = torch.where(seen_p[None, :, None], _dequant(pre["k_codes"][0], pre["k_scale"][0]), 0.0)
    vp = torch.where(seen_p[None, :, None], _dequant(pre["v_codes"][0], pre["v_scale"][0]), 0.0)
    rows = q.transpose(0, 1).reshape(Hkv, B * G, d)
    sp = (rows @ kp.transpose(1, 2)).masked_fill(~seen_p, -math.inf)
    # each session's own slots
    seen = _visible(own_c, c["window"])
    keep = seen[:, None, :, None]
    ko = torch.where(keep, _dequant(own_c["k_codes"], own_c["k_scale"]), 0.0)
    vo = torch.where(keep, _dequant(own_c["v_codes"], own_c["v_scale"]), 0.0)
    so = (q @ ko.transpose(2, 3)).masked_fill(~seen[:, None, None], -math.inf)
    so = so.transpose(0, 1).reshape(Hkv, B * G, -1)
    m = torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True)).clamp(min=-3e38)
    sp, so = (sp - m).exp(), (so - m).exp()
    total = sp.sum(-1, keepdim=True) + so.sum(-1, keepdim=True)
    o = sp @ vp + (so.view(Hkv, B, G, -1).transpose(0, 1) @ vo).transpose(0, 1).reshape(Hkv, B * G, d)
    o = torch.where(total > 0, o / total, 0.0)
    return o.view(Hkv, B, G, d).transpose(0, 1).reshape(B, Hq, d).bfloat16()


def _plain_norm_rope(s):
    c, q, k = s["case"], s["q"], s["k"]
    pos = s["positions"]
    if pos is None:
        pos = torch.arange(c["T"], device=q.device)[None].expand(c["B"], -1)
    return _norm_rope(q, s["wq"], pos, c["theta"]).to(q.dtype), _norm_rope(k, s["wk"], pos, c["theta"]).to(k.dtype)


def _plain_norm_append(s):
    c, cache = s["case"], s["cache"]
    pos = cache["seq_len"] + s["base"]
    q = _norm_rope(s["q"], s["wq"], pos, c["theta"]).bfloat16()
    k = _norm_rope(s["k"], s["wk"], pos, c["theta"]).bfloat16()
    cap, rs, rl = cache["ring_cap"], cache["ring_start"], cache["ring_len"]
    row = torch.arange(c["B"], device=q.device)
    slot = torch.remainder(rs + rl, cap).long()
    for name, x in (("k", k), ("v", s["v"])):
        code, scale = _quantise(x)
        cache[name + "_codes"][row, :, slot] = code
        cache[name + "_scale"][row, :, slot] = scale
    full = rl == cap
    rs.copy_(torch.where(full, torch.remainder(rs + 1, cap), rs))
    rl.copy_(torch.where(full, rl, rl + 1))
    cache["seq_len"] += 1
    newest = {n: _dequant(cache[n + "_codes"][row, :, slot], cache[n + "_scale"][row, :, slot]).bfloat16()[:, None]
              for n in ("k", "v")}
    return dict(q=q, k=newest["k"], v=newest["v"], ring_start=rs, ring_len=rl, seq_len=cache["seq_len"])


def _plain_cache_read(s):
    """Row r of a session: its sinks, then the ring entries the window reaches, oldest first; rows behind them stay 0."""
    c, cache = s["case"], s["cache"]
    S, W = cache["sink_cap"], cache["ring_cap"]
    n_rows = S + min(W, c["window"])
    dev = cache["k_codes"].device
    sl, rs, rl, sq = (cache[f][:, None].long() for f in ("sink_len", "ring_start", "ring_len", "seq_len"))
    r = torch.arange(n_rows, device=dev)[None]
    n = rl.clamp(max=c["window"])
    entry = rl - n + (r - sl)                     # ring entry, oldest first
    slot = torch.where(r < sl, r, S + torch.remainder(rs + entry, max(W, 1)))
    live = r < sl + n
    pos = torch.where(live, torch.where(r < sl, r, sq - rl + entry), -1)
    slot = torch.where(live, slot, 0)
    dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
    take = slot[:, None, :, None]
    out = []
    for name in ("k", "v"):
        codes, scale = cache[name + "_codes"], cache[name + "_scale"]
        codes = codes.gather(2, take.expand(-1, codes.shape[1], -1, codes.shape[3]))
        scale = scale.gather(2, take.expand(-1, scale.shape[1], -1, scale.shape[3]))
        x = torch.where(live[:, None, :, None], _dequant(codes, scale), 0.0)
        out.append(x.transpose(1, 2).to(dt).contiguous())
    return dict(k=out[0], v=out[1], positions=pos.to(torch.int32), lengths=(sl + n)[:, 0].to(torch.int32))


# --------------------------------------------------------------------------
# The library's calls
# --------------------------------------------------------------------------

def _kv(s, name):
    """The library's handle on a cache's tensors, made once per state as a user's program keeps it."""
    import sliding_window_kv_swa_gb300 as nd
    key = "kv_" + name
    if key not in s:
        c = s[name]
        s[key] = nd.KVCache(*(c[f] for f in KV_FIELDS), c["sink_cap"], c["ring_cap"])
    return s[key]


def _own(s):
    import sliding_window_kv_swa_gb300 as nd
    c, op = s["case"], s["case"]["op"]
    if op == "shared_decode":
        cache, prefix, q = _kv(s, "cache"), _kv(s, "prefix"), s["q"]
        if "ws" not in s:
            size = nd.nd_shared_prefix_decode_workspace_size(c["B"], c["Hq"], c["Hkv"], c["d"], c["prefix_cap"],
                                                             c["sinks"] + c["ring"])
            s["ws"] = torch.empty(max(size, 16), dtype=torch.uint8, device=q.device)
        return nd.nd_shared_prefix_decode(q, prefix, cache, c["window"], workspace=s["ws"])
    if op == "norm_rope":
        return nd.nd_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], EPS, c["theta"], positions=s["positions"])
    cache = _kv(s, "cache")
    if op == "norm_append":
        q = nd.nd_qk_norm_rope_append(s["q"], cache, s["k"], s["v"], s["wq"], s["wk"], EPS, c["theta"], pos_base=s["base"])
        k, v, _, _ = nd.nd_kv_cache_read(cache, 1)
        return dict(q=q, k=k, v=v, ring_start=cache.ring_start, ring_len=cache.ring_len, seq_len=cache.seq_len)
    if "k_out" not in s:  # the rows behind a short session stay what they were: zeros here, as a padded batch wants them
        dt = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
        shape = (c["B"], c["sinks"] + min(c["ring"], c["window"]), c["Hkv"], c["d"])
        s["k_out"], s["v_out"] = (torch.zeros(shape, dtype=dt, device="cuda") for _ in range(2))
    k, v, pos, n = nd.nd_kv_cache_read(cache, c["window"], k_out=s["k_out"], v_out=s["v_out"])
    return dict(k=k, v=v, positions=pos, lengths=n)


def run(state):
    if own:
        return _own(state)
    return {"shared_decode": _plain_shared_decode, "norm_rope": _plain_norm_rope, "norm_append": _plain_norm_append,
            "cache_read": _plain_cache_read}[state["case"]["op"]](state)


def work(case):
    c, op, d, Hkv = case, case["op"], case["d"], case["Hkv"]
    slot = 2 * (d + d // 8)                       # K and V codes and scales of one (slot, KV head)
    if op == "shared_decode":
        fill = 1.0 if c["full"] else 0.5
        seen = fill * c["sinks"] + min(fill * c["ring"], c["window"])
        return dict(bytes=Hkv * slot * (c["prefix"] + c["B"] * seen) + 4 * c["B"] * c["Hq"] * d,
                    flops=4 * c["B"] * c["Hq"] * d * (c["prefix"] + seen))
    if op == "norm_rope":
        rows = c["B"] * c["T"] * (c["Hq"] + Hkv)
        return dict(bytes=rows * d * 2 * (4 if c["dtype"] == "f32" else 2) + (4 * c["B"] * c["T"] if c["positions"] else 0),
                    flops=rows * d * 7)
    if op == "norm_append":
        rows = c["B"] * (c["Hq"] + Hkv)
        # the row written by the step is read back: codes once more, two bf16 rows out
        return dict(bytes=c["B"] * (4 * c["Hq"] * d + 4 * Hkv * d + 2 * Hkv * slot + 4 * Hkv * d), flops=rows * d * 7 + 4 * c["B"] * Hkv * d)
    fill = 1.0 if c["full"] else 0.5
    seen = c["B"] * (fill * c["sinks"] + min(fill * c["ring"], c["window"]))
    return dict(bytes=seen * Hkv * (slot + 2 * d * (4 if c["dtype"] == "f32" else 2)), flops=2 * seen * Hkv * d)


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_tokens(cache, b, window):
    """Sequence b's visible slots in position order, and their positions."""
    sl, rs, rl, sq = (int(cache[f][b]) for f in ("sink_len", "ring_start", "ring_len", "seq_len"))
    n = min(rl, window)
    slots = list(range(sl)) + [cache["sink_cap"] + (rs + i) % cache["ring_cap"] for i in range(rl - n, rl)]
    return slots, list(range(sl)) + [sq - rl + i for i in range(rl - n, rl)]


def _exact_rows(cache, which, b, slots):
    codes = cache[which + "_codes"][b][:, slots].double()
    return codes * cache[which + "_scale"][b][:, slots].double().repeat_interleave(GROUP, dim=-1)


def _exact_turn(x, w, pos, theta):
    """One head-rows tensor [..., heads, d] in 64 bits, as complex numbers turned by pos * theta^(-2i/d)."""
    x, d = x.double(), x.shape[-1]
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS) * w.double()
    i = torch.arange(d // 2, dtype=torch.float64, device=x.device)
    angle = pos.double()[..., None, None] * torch.pow(torch.tensor(theta, dtype=torch.float64, device=x.device), -2 * i / d)
    z = torch.complex(y[..., : d // 2], y[..., d // 2:]) * torch.polar(torch.ones_like(angle), angle)
    return torch.cat([z.real, z.imag], -1)


def _exact_code(x):
    """What the int8 codec stores for x, as values."""
    y = x.double().unflatten(-1, (-1, GROUP))
    amax = y.abs().amax(-1, keepdim=True)
    scale = (amax.float() / 127.0).double()       # the stored scale has 32 bits
    return (torch.round(y / scale.clamp(min=1e-300)).clamp(-127, 127) * scale).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], s["case"]["op"]
    if op == "norm_rope":
        pos = s["positions"]
        if pos is None:
            pos = torch.arange(c["T"], device="cuda").repeat(c["B"], 1)
        return _exact_turn(s["q"], s["wq"], pos, c["theta"]), _exact_turn(s["k"], s["wk"], pos, c["theta"])
    cache = s["cache"]
    if op == "norm_append":
        pos = cache["seq_len"] + s["base"]
        k = _exact_turn(s["k"], s["wk"], pos, c["theta"]).bfloat16()  # the key is rounded to bf16, then stored
        return dict(q=_exact_turn(s["q"], s["wq"], pos, c["theta"]), k=_exact_code(k)[:, None], v=_exact_code(s["v"])[:, None],
                    ring_start=None, ring_len=None, seq_len=None)
    if op == "cache_read":
        n_rows = c["sinks"] + min(c["ring"], c["window"])
        out = {n: torch.zeros(c["B"], n_rows, c["Hkv"], c["d"], dtype=torch.float64, device="cuda") for n in ("k", "v")}
        for b in range(c["B"]):
            slots, _ = _exact_tokens(cache, b, c["window"])
            for n in ("k", "v"):
                out[n][b, : len(slots)] = _exact_rows(cache, n, b, slots).transpose(0, 1)
        return dict(k=out["k"], v=out["v"], positions=None, lengths=None)
    G, L = c["Hq"] // c["Hkv"], c["prefix"]
    kp, vp = (_exact_rows(s["prefix"], n, 0, list(range(L))) for n in ("k", "v"))
    got = []
    for b in range(c["B"]):                       # one session at a time: prefix and own slots in one row
        slots, _ = _exact_tokens(cache, b, c["window"])
        k = torch.cat([kp, _exact_rows(cache, "k", b, slots)], 1)
        v = torch.cat([vp, _exact_rows(cache, "v", b, slots)], 1)
        q = s["q"][b].double().view(c["Hkv"], G, -1)
        p = torch.softmax(q @ k.transpose(1, 2) / math.sqrt(c["d"]), -1)
        got.append((p @ v).reshape(c["Hq"], -1))
    return torch.stack(got)
