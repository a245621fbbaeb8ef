"""Measured calls of a ragged serving step over bf16 paged caches.

Four operators, in the order a step makes them:

  rope     rotary positions: q and k of a packed batch of tokens rotated by each token's own position,
           the whole head or the first part of it, pairs half a head apart or neighbours, frequencies
           scaled for long contexts (``DuoRope.rotate``)
  append   the tokens' keys and values into a paged cache (retrieval heads) and into the sink + ring
           caches (streaming heads), keys and queries rotated on the way (``DuoPagedLayer.append_ragged``)
  prefill  attention of a packed batch of chunks, each sequence with its own cached length and number of
           new tokens, over the paged cache and the chunk's own keys (``DuoPagedLayer.prefill_ragged``)
  decode   the same for one token a sequence, appended before, with the lengths on the device
           (``DuoPagedLayer.decode_varlen``)

``own = False`` computes them with elementary torch operations in 32 bits (angles in 64: a position of a
million times a frequency leaves 32 bits no fraction to speak of), ``own = True`` calls the package.
"""

import math

import torch

own = False

# frequencies as this framework's users set them: plain, and scaled for contexts past the trained length
ROPES = {
    "plain": dict(theta=10000.0, scaling=None),
    "linear": dict(theta=10000.0, scaling=dict(kind="linear", factor=4.0)),
    "ntk": dict(theta=10000.0, scaling=dict(kind="ntk", factor=8.0)),
    "yarn": dict(theta=1000000.0, scaling=dict(kind="yarn", factor=4.0, original=32768)),
    "wavelength": dict(theta=500000.0, scaling=dict(kind="wavelength", factor=8.0, low=1.0, high=4.0, original=8192)),
}


# --------------------------------------------------------------------------- the cases
def listed():
    gqa = dict(Hq=32, Hkv=8, D=128, S=64, R=256)
    return [
        # the rotation of a decode step: 64 tokens far into long contexts; latency counts
        dict(name="rope_step_b64", op="rope", N=64, far=1 << 20, Hq=32, Hkv=8, D=128, rd=128, layout="half", rope="yarn",
             fused=False),
        # a packed batch of prompts, q and k slices of a fused projection
        dict(name="rope_prompts_24k", op="rope", N=24001, far=32768, Hq=32, Hkv=8, D=128, rd=128, layout="half",
             rope="wavelength", fused=True),
        # half of a 64-dim head, neighbouring pairs
        dict(name="rope_part_d64", op="rope", N=5003, far=8192, Hq=16, Hkv=16, D=64, rd=32, layout="interleaved",
             rope="plain", fused=False),
        # the append of a decode step: one token each for 64 sequences, q rotated along
        dict(name="append_step_b64", op="append", B=64, T=1, n=16384, n_ret=2, page=128, rd=128, layout="half", rope="yarn",
             **gqa),
        # ragged chunks of prompts, 64-dim heads, slices of a fused projection
        dict(name="append_ragged_d64", op="append", B=12, T=4096, n=4096, Hq=16, Hkv=4, n_ret=2, D=64, S=4, R=32, page=128,
             rd=64, layout="interleaved", rope="plain"),
        # fresh prompts of very different lengths in one packed batch
        dict(name="prefill_prompts", op="prefill", B=5, T=12000, n=0, n_ret=4, page=256, kind="chunks", **gqa),
        # a mixed step: most sequences take one token over long contexts, two take a chunk
        dict(name="prefill_mixed_b32", op="prefill", B=32, T=1500, n=32000, n_ret=2, page=128, kind="mixed", **gqa),
        # follow-up questions of a few hundred tokens to long conversations, odd lengths
        dict(name="prefill_turns", op="prefill", B=3, T=333, n=9001, n_ret=4, page=256, kind="chunks", **gqa),
        # the last chunk of a 32K prompt, multi-head attention, a quarter of the heads retrieval
        dict(name="prefill_chunk_28k", op="prefill", B=1, T=4096, n=28672, Hq=32, Hkv=32, n_ret=8, D=128, S=64, R=256,
             page=256, kind="chunks"),
        # a few hundred tokens, small heads: latency counts
        dict(name="decode_tiny", op="decode", B=2, n=272, Hq=4, Hkv=4, n_ret=2, D=64, S=4, R=32, page=128),
        # one sequence of a million tokens
        dict(name="decode_1m", op="decode", B=1, n=(1 << 20) - 27, n_ret=2, page=256, **gqa),
        # a serving batch of ragged lengths, an empty one among them
        dict(name="decode_ragged_b48", op="decode", B=48, n=32000, n_ret=2, page=128, **gqa),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "prefill", "prefill", "decode", "decode"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([2, 4, 8])
    heads = dict(Hkv=Hkv, Hq=Hkv * rng.choice([1, 2, 4, 8]), D=D)
    rope = dict(rd=rng.choice([D, D, D // 2, D // 4, 3 * D // 4]), layout=rng.choice(["half", "interleaved"]),
                rope=rng.choice(sorted(ROPES)))
    if op == "rope":
        return dict(op=op, N=_log_int(rng, 1, 400000 // (heads["Hq"] + Hkv)), far=_log_int(rng, 100, 1 << 22),
                    fused=rng.random() < 0.5, **heads, **rope)
    S, R = rng.choice([(64, 256), (4, 32), (0, rng.randint(1, 300)), (rng.randint(1, 130), rng.randint(1, 300))])
    heads.update(n_ret=rng.randint(1, Hkv), S=S, R=R, page=128 * rng.randint(1, 4))
    n_ret, per = heads["n_ret"], heads["Hq"] // Hkv
    if op == "append":
        T = rng.choice([1, _log_int(rng, 2, 8192)])
        B = _log_int(rng, 1, max(1, min(128, 400000 // (heads["Hq"] + 2 * Hkv) // T)))
        return dict(op=op, B=B, T=T, n=_log_int(rng, 1, 8192), **heads, **rope)
    if op == "decode":
        n = _log_int(rng, 1, 400000 if n_ret < 5 else 250000)
        return dict(op=op, B=_log_int(rng, 1, max(1, min(64, 2000000 // (n * n_ret)))), n=n, **heads)
    kind = rng.choice(["chunks", "chunks", "mixed"])
    T = _log_int(rng, 1, 4000)
    pairs = 10 ** 9 // (n_ret * per)  # query-key pairs a head that cost what the listed chunk costs
    n = rng.choice([0, _log_int(rng, 1, max(1, min(24000, pairs // T - T)))])
    most = max(1, min(16, pairs // (T * (n + T))))
    return dict(op=op, B=rng.randint(4, 24) if kind == "mixed" and n * 24 < 300000 else rng.randint(1, most),
                T=T, n=n, kind=kind, **heads)


# --------------------------------------------------------------------------- inputs
def _retrieval(c):
    """Which KV heads are retrieval heads: n_ret of them, spread over the heads."""
    return [1 if (h * c["n_ret"]) // c["Hkv"] != ((h + 1) * c["n_ret"]) // c["Hkv"] else 0 for h in range(c["Hkv"])]


def _heads(c):
    m = _retrieval(c)
    return (torch.tensor([h for h in range(c["Hkv"]) if m[h]], device="cuda", dtype=torch.long),
            torch.tensor([h for h in range(c["Hkv"]) if not m[h]], device="cuda", dtype=torch.long))


def _keys(g, *shape):
    """Rows with a few strong channels, as keys have."""
    x = torch.randn(*shape, generator=g, device="cuda")
    gain = torch.ones(shape[-1], device="cuda")
    gain[3::29] = 3.0
    return (x * gain).to(torch.bfloat16)


def _values(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def _projection(g, c, N):
    """q, k, v [N, heads, D] as slices of one fused projection's output."""
    x = torch.cat([_values(g, N, c["Hq"], c["D"]), _keys(g, N, c["Hkv"], c["D"]), _values(g, N, c["Hkv"], c["D"])], 1)
    return x.split([c["Hq"], c["Hkv"], c["Hkv"]], 1)


def _frequencies(c):
    """Angle per position of each pair, in radians, and the factor of the rotated pairs."""
    spec = ROPES[c["rope"]]
    theta, sc, rd = spec["theta"], spec["scaling"], c["rd"]
    half = rd // 2
    f = [theta ** (-2.0 * i / rd) for i in range(half)]
    if sc is None:
        return f, 1.0
    s = sc["factor"]
    if sc["kind"] == "linear":
        return [x / s for x in f], 1.0
    if sc["kind"] == "ntk":
        base = theta * s ** (rd / (rd - 2.0))
        return [base ** (-2.0 * i / rd) for i in range(half)], 1.0
    if sc["kind"] == "wavelength":
        out = []
        for x in f:
            turns = sc["original"] * x / (2 * math.pi)  # over the trained length
            keep = min(1.0, max(0.0, (turns - sc["low"]) / (sc["high"] - sc["low"])))
            out.append(x * keep + x / s * (1 - keep))
        return out, 1.0
    at = lambda turns: rd * math.log(sc["original"] / (turns * 2 * math.pi)) / (2 * math.log(theta))
    lo, hi = max(0, math.floor(at(32.0))), min(rd - 1, math.ceil(at(1.0)))
    out = []
    for i, x in enumerate(f):
        past = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
        out.append(x * (1 - past) + x / s * past)
    return out, 0.1 * math.log(s) + 1.0


def _rope(c):
    """The package's frequencies of the same."""
    import streaming_kv_cache_duo_gb300 as duo
    spec = ROPES[c["rope"]]
    return duo.DuoRope(c["D"], theta=spec["theta"], rotary_dim=c["rd"], layout=c["layout"], scaling=spec["scaling"])


def _ring_positions(lens, S, R):
    """Token position held by each sink + ring slot after len tokens, -1 if empty: [B, S + R] int32."""
    slot = torch.arange(S + R, device="cuda")[None, :]
    n = lens[:, None].long()
    last = n - 1 - (n - 1 - slot) % R  # the last position below n that is congruent to the slot
    # (slot S + (t - S) mod R holds t: slots and positions are congruent modulo R)
    pos = torch.where(slot < S, slot, last)
    ok = torch.where(slot < S, slot < n, (pos >= S) & (n > 0))
    return torch.where(ok, pos, torch.full_like(pos, -1)).to(torch.int32)


def _lengths(c, g):
    """Cached tokens of each sequence, and its new ones."""
    B, n = c["B"], c["n"]
    share = torch.rand(B, generator=g, device="cuda")
    lens = (share * (n + 1)).long().clamp(max=n)
    lens[0] = n
    T = c.get("T", 1)
    if c["op"] == "decode":
        if B >= 4:
            lens[1], lens[2] = 0, min(n, 41)
        new = torch.ones(B, dtype=torch.long, device="cuda")
    else:
        new = torch.ones(B, dtype=torch.long, device="cuda")
        some = 2 if c["op"] == "prefill" and c["kind"] == "mixed" else B  # sequences with more than one token
        if some > 1:  # they share out what is left of the step at random
            spare = _packed(c) - T - (B - 1)
            share = torch.rand(some - 1, generator=g, device="cuda", dtype=torch.float64) + 0.3
            more = (share / share.sum() * spare).long()
            more[-1] += spare - more.sum()
            new[1:some] += more
        new[0] = T
    return lens.to(torch.int32), new.to(torch.int32)


def _packed(c):
    """Tokens of the packed batch: T of the first sequence, half as many of each other one with a chunk."""
    B, T = c["B"], c["T"]
    if c["op"] == "prefill" and c["kind"] == "mixed":
        return T + (B > 1) * ((T + 1) // 2) + max(0, B - 2)
    return T + (B - 1) * ((T + 1) // 2)


def _cache(c, g, lens, cap):
    """A paged cache of sequences of `lens` tokens, with blocks for `cap` tokens each in a random order."""
    B, D, S, R, n_ret, page = c["B"], c["D"], c["S"], c["R"], c["n_ret"], c["page"]
    per = -(-cap.long() // page)  # [B]
    most = max(1, int(per.max()))
    total = int(per.sum()) * n_ret
    size = total + 3
    if c["op"] == "append":  # (the pool is given back: of one size for every batch of these sizes)
        size = n_ret * (B * (c["n"] // page + 2) + _packed(c) // page) + 3
    ids = torch.randperm(size, generator=g, device="cuda")
    have = (torch.arange(most, device="cuda")[None, None, :] < per[:, None, None]).expand(B, n_ret, most)
    table = torch.full(have.shape, -1, dtype=torch.int32, device="cuda")
    table[have] = ids[:total].to(torch.int32)
    s = {"lens": lens, "table": table, "num_blocks": size, "pos": _ring_positions(lens, S, R)}
    for name, make in (("k", _keys), ("v", _values)):
        pool = torch.empty(size, page, D, dtype=torch.bfloat16, device="cuda")
        for i in range(0, size, 1024):  # (a pool of a million rows at a time)
            pool[i:i + 1024] = make(g, min(1024, size - i), page, D)
        s[name + "_full"] = pool
        s[name + "_sr"] = make(g, B, c["Hkv"] - n_ret, S + R, D)
    return s


BUFFERS = ("k_full", "v_full", "k_sr", "v_sr", "pos")


def _layer(c, s):
    """The package's owner of that cache."""
    import streaming_kv_cache_duo_gb300 as duo
    layer = duo.DuoPagedLayer(c["B"], c["Hq"], c["Hkv"], c["D"], c["S"], c["R"], c["page"], s["table"].shape[2],
                              s["num_blocks"], s["table"], _retrieval(c))
    for name in BUFFERS:
        getattr(layer, name).copy_(s[name])
        s[name] = getattr(layer, name)
    return layer


def _slots(c, s, lens, new):
    """Where each packed token goes: cu_new, token_seq, token_pos, slots."""
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), new.long().cumsum(0)])
    seq = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), new.long())
    at = lens.long()[seq] + torch.arange(seq.numel(), device="cuda") - cu[seq]
    ids = s["table"][seq, :, at // c["page"]].long()
    s["cu_new"], s["token_seq"], s["token_pos"] = cu.int(), seq.int(), at.int()
    s["slots"] = ids * c["page"] + (at % c["page"])[:, None]
    if own:
        import streaming_kv_cache_duo_gb300 as duo
        s["map"] = duo.DuoSlotMap(s["cu_new"], s["token_seq"], s["token_pos"], s["slots"])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] == "rope":
        N = c["N"]
        s = {"token_pos": (torch.rand(N, generator=g, device="cuda", dtype=torch.float64) * c["far"]).int()}
        if c["fused"]:
            s["q"], s["k"], _ = _projection(g, c, N)
        else:
            s["q"], s["k"] = _values(g, N, c["Hq"], c["D"]), _keys(g, N, c["Hkv"], c["D"])
    else:
        lens, new = _lengths(c, g)
        s = _cache(c, g, lens, lens + new)
        s["new"] = new
        if c["op"] == "decode":
            s["q"] = _values(g, c["B"], c["Hq"], c["D"])
        else:
            _slots(c, s, lens, new)
            N = s["token_seq"].numel()
            s["q"], s["k"], s["v"] = _projection(g, c, N)
            if c["op"] == "prefill":  # q and k come out of the rotation, v is still a slice
                s["q"], s["k"] = s["q"].contiguous(), s["k"].contiguous()
        if own:
            s["layer"] = _layer(c, s)
    if "rope" in c:
        f, scale = _frequencies(c)
        s["freq"], s["scale"] = torch.tensor(f, dtype=torch.float64, device="cuda"), scale
        if own:
            s["rope"] = _rope(c)
    s["case"] = c
    if c["op"] != "rope":
        s["heads"] = _heads(c)
    return s


# --------------------------------------------------------------------------- one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    c = s["case"]
    if c["op"] == "rope":
        return s["rope"].rotate(s["q"], s["k"], s["token_pos"])
    layer = s["layer"]
    if c["op"] == "append":
        q = layer.append_ragged(s["k"], s["v"], s["map"], rope=s["rope"], q=s["q"])
        return {"q": q, **_buffers(s)}
    if c["op"] == "prefill":
        return layer.prefill_ragged(s["q"], s["k"], s["v"], s["map"])
    return layer.decode_varlen(s["q"], s["lens"], c["n"])


def _buffers(s):
    """The cache after an append."""
    return {name: s[name] for name in BUFFERS}


def _run_plain(s):
    op = s["case"]["op"]
    return {"rope": _plain_rope, "append": _plain_append, "prefill": _plain_prefill, "decode": _plain_decode}[op](s)


def _rotated(s, x):
    """Rows [N, heads, D] turned by their tokens' angles, in 32 bits; rounded once."""
    c = s["case"]
    rd = c["rd"]
    angle = s["token_pos"].double()[:, None] * s["freq"]
    cos, sin = ((f(angle) * s["scale"]).float()[:, None, :] for f in (torch.cos, torch.sin))
    y = x.float()
    turned = y[..., :rd]
    if c["layout"] == "half":
        a, b = turned[..., : rd // 2], turned[..., rd // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned.to(torch.bfloat16), x[..., rd:]], -1)


def _plain_rope(s):
    return _rotated(s, s["q"]), _rotated(s, s["k"])


def _plain_append(s):
    c, (ret, stream) = s["case"], s["heads"]
    S, R, D = c["S"], c["R"], c["D"]
    q, k = _rotated(s, s["q"]), _rotated(s, s["k"])
    seq, at = s["token_seq"].long(), s["token_pos"].long()
    end = (s["lens"] + s["new"]).long()
    keep = ((at < S) | (at >= end[seq] - R)).nonzero()[:, 0]
    slot = torch.where(at[keep] < S, at[keep], S + (at[keep] - S) % R)
    for name, x in (("k", k), ("v", s["v"])):
        s[name + "_full"].view(-1, D)[s["slots"].reshape(-1)] = x[:, ret].reshape(-1, D)
        if stream.numel():
            s[name + "_sr"][seq[keep], :, slot] = x[keep][:, stream]
    if stream.numel():
        s["pos"][seq[keep], slot] = at[keep].int()
    return {"q": q, **_buffers(s)}


def _softmax_rows(sc, vis, v):
    """softmax over the last axis of the visible scores times v; 0 for a row that sees nothing."""
    sc = torch.where(vis, sc, torch.full_like(sc, -math.inf))
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    den = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(den > 0, den, torch.ones_like(den))


def _plain_prefill(s):
    c, kinds = s["case"], _retrieval(s["case"])
    Hkv, D, S, R, page = c["Hkv"], c["D"], c["S"], c["R"], c["page"]
    g = c["Hq"] // Hkv
    lens, cu = s["lens"].tolist(), s["cu_new"].tolist()
    out = torch.empty_like(s["q"])
    order = [sum(kinds[:h]) if kinds[h] else h - sum(kinds[:h]) for h in range(Hkv)]
    for b in range(c["B"]):
        n, T = lens[b], cu[b + 1] - cu[b]
        if T == 0:
            continue
        rows = slice(cu[b], cu[b + 1])
        i = n + torch.arange(T, device="cuda")
        for h in range(Hkv):
            q = s["q"][rows, h * g:(h + 1) * g].float().transpose(0, 1) / math.sqrt(D)  # [g, T, D]
            if kinds[h]:
                ids = s["table"][b, order[h], : -(-n // page)].long()
                held = torch.arange(n, device="cuda")
                old = [s[x + "_full"][ids].reshape(-1, D)[:n] for x in "kv"]
            else:
                held = s["pos"][b].long()
                old = [s[x + "_sr"][b, order[h]] for x in "kv"]
            pos = torch.cat([held, i])
            k, v = (torch.cat([o, s[x][rows, h]]).float() for o, x in zip(old, "kv"))
            step = max(1, (1 << 28) // (g * pos.numel()))
            for t in range(0, T, step):
                row = i[t:t + step, None]
                vis = (pos >= 0) & (pos <= row)
                if not kinds[h]:
                    vis &= (pos < S) | (row - pos < R)
                o = _softmax_rows(torch.matmul(q[:, t:t + step], k.T), vis, v)
                out[cu[b] + t:cu[b] + t + row.shape[0], h * g:(h + 1) * g] = o.transpose(0, 1).to(torch.bfloat16)
    return out


def _plain_decode(s):
    c, (ret, stream) = s["case"], s["heads"]
    B, Hkv, D, page = c["B"], c["Hkv"], c["D"], c["page"]
    lens = s["lens"].long()
    q = s["q"].float().reshape(B, Hkv, c["Hq"] // Hkv, D) / math.sqrt(D)
    o = torch.zeros_like(q)
    ids = s["table"][:, :, : -(-c["n"] // page)].long().clamp(min=0)
    k, v = (s[x + "_full"][ids].reshape(B, c["n_ret"], -1, D).float() for x in "kv")
    vis = torch.arange(k.shape[2], device="cuda") < lens[:, None, None, None]
    o[:, ret] = _softmax_rows(torch.matmul(q[:, ret], k.transpose(-1, -2)), vis, v)
    pos, i = s["pos"].long(), lens[:, None] - 1
    vis = (pos >= 0) & (pos <= i) & ((pos < c["S"]) | (i - pos < c["R"]))
    k, v = s["k_sr"].float(), s["v_sr"].float()
    o[:, stream] = _softmax_rows(torch.matmul(q[:, stream], k.transpose(-1, -2)), vis[:, None, None, :], v)
    return o.reshape(B, c["Hq"], D).to(torch.bfloat16)


# --------------------------------------------------------------------------- cost and truth
def _expected(c):
    """Sequences' (cached, new) tokens, the cached ones on average, for the count of work."""
    B, n, T = c["B"], c["n"], c.get("T", 1)
    out = []
    for b in range(B):
        chunk = T if b == 0 else (T + 1) // 2
        if c["op"] == "decode" or (c["op"] == "prefill" and c["kind"] == "mixed" and b >= 2):
            chunk = 1
        out.append((n if b == 0 else n / 2, chunk))
    return out


def work(case):
    c = case
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if c["op"] == "rope":
        return {"bytes": c["N"] * ((Hq + Hkv) * D * 4 + 4), "flops": c["N"] * (Hq + Hkv) * c["rd"] * 3}
    S, R, n_ret, g = c["S"], c["R"], c["n_ret"], Hq // Hkv
    n_str = Hkv - n_ret
    lens = _expected(c)
    new = sum(t for _, t in lens)
    if c["op"] == "append":
        # q in and out; k and v in (a streaming head's where it keeps the token) and into the caches
        kept = sum(min(t, S + R) for _, t in lens)
        rows = n_ret * new + n_str * kept
        return {"bytes": new * (Hq * D * 4 + 8 + 8 * n_ret) + rows * D * 8, "flops": 3 * c["rd"] * (new * Hq + rows)}
    cached = sum(n_ret * n + n_str * min(n, S + R) for n, _ in lens) * D * 4
    if c["op"] == "decode":
        keys = sum(n_ret * n + n_str * min(n, S + R) for n, _ in lens)
        return {"bytes": cached + 4 * c["B"] * Hq * D, "flops": 4 * D * g * keys}
    pairs = sum(n_ret * (t * n + t * (t + 1) / 2) + n_str * (min(t * n + t * (t + 1) / 2, t * (S + R)))
                for n, t in lens)
    return {"bytes": cached + new * D * (4 * Hq + 4 * Hkv), "flops": 4 * D * g * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope", "append"):
        return _exact_rotation(case, s)
    return _exact_attention(case, s)


def _turn64(c, s, x):
    """Pair after pair as complex numbers times e^(i angle), in 64 bits."""
    half = c["rd"] // 2
    w = torch.polar(torch.full((1,), s["scale"], dtype=torch.float64, device="cuda"),
                    s["token_pos"].double()[:, None] * s["freq"][None, :])[:, None, :]
    y = x.double().clone()
    first = torch.arange(half, device="cuda") * (1 if c["layout"] == "half" else 2)
    second = first + (half if c["layout"] == "half" else 1)
    z = torch.complex(y[..., first], y[..., second]) * w
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rotation(c, s):
    q, k = _turn64(c, s, s["q"]), _turn64(c, s, s["k"])
    if c["op"] == "rope":
        return q, k
    ret, stream = (h.tolist() for h in s["heads"])
    out = {name: s[name].double() for name in BUFFERS if name != "pos"}
    at, seq = s["token_pos"].tolist(), s["token_seq"].tolist()
    last = (s["lens"] + s["new"]).tolist()
    for r, h in enumerate(ret):
        row = s["slots"][:, r]
        out["k_full"][row // c["page"], row % c["page"]] = k[:, h]
        out["v_full"][row // c["page"], row % c["page"]] = s["v"][:, h].double()
    if stream:
        # token by token, in the order they come
        where = {}
        for i, (b, p) in enumerate(zip(seq, at)):
            if p < c["S"] or p >= last[b] - c["R"]:
                where[(b, p if p < c["S"] else c["S"] + (p - c["S"]) % c["R"])] = i
        b = torch.tensor([key[0] for key in where], device="cuda")
        slot = torch.tensor([key[1] for key in where], device="cuda")
        i = torch.tensor(list(where.values()), device="cuda")
        for e, h in enumerate(stream):
            out["k_sr"][b, e, slot] = k[i, h]
            out["v_sr"][b, e, slot] = s["v"][i, h].double()
    return {"q": q, **{name: out.get(name) for name in BUFFERS}}  # (positions are whole numbers)


def _exact_attention(c, s):
    """Head by head over the keys a block of queries can see, in 64 bits."""
    ret, stream = (h.tolist() for h in s["heads"])
    Hq, Hkv, D, S, R, page = (c[x] for x in ("Hq", "Hkv", "D", "S", "R", "page"))
    g = Hq // Hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    begin = 0
    for b in range(c["B"]):
        n = int(s["lens"][b])
        T = int(s["new"][b])
        first = n if c["op"] == "prefill" else n - 1
        rows = range(begin, begin + T)
        begin += T
        if c["op"] == "decode" and n == 0:
            continue
        at = torch.arange(first, first + T, device="cuda")
        for h in range(Hkv):
            parts = {}
            for name in ("k", "v"):
                if h in ret:
                    blocks = s["table"][b, ret.index(h), : -(-n // page)].long()
                    old = s[name + "_full"][blocks].reshape(-1, D)[:n]
                    held = torch.arange(n, device="cuda")
                else:
                    held = s["pos"][b].long()
                    old = s[name + "_sr"][b, stream.index(h)][held >= 0]
                    held = held[held >= 0]
                if c["op"] == "prefill":
                    old = torch.cat([old, s[name][rows.start:rows.stop, h]])
                    held = torch.cat([held, at])
                parts[name] = old.double()
            for t in range(0, T, 512):
                i = at[t:t + 512]
                near = held <= i[-1]  # keys any query of the block sees
                if h in stream:
                    near &= (held < S) | (held > i[0] - R)
                j = held[near]
                sees = j[None, :] <= i[:, None]
                if h in stream:
                    sees &= (j[None, :] < S) | (i[:, None] - j[None, :] < R)
                qb = s["q"][rows.start + t:rows.start + t + i.numel(), h * g:(h + 1) * g].double()
                sc = torch.einsum("thd,kd->htk", qb, parts["k"][near]) / math.sqrt(D)
                p = torch.softmax(sc.masked_fill(~sees, -math.inf), -1)
                out[rows.start + t:rows.start + t + i.numel(), h * g:(h + 1) * g] = \
                    torch.einsum("htk,kd->thd", p, parts["v"][near])
    return out
