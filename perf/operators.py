"""Measured calls of the 8-bit KV cache operators and of the block tables that feed them.

Four operators of a serving step over mixed retrieval / streaming heads:

  tables   block tables, slot maps and the free list, brought up to date on the GPU from the
           requests' lengths (``DuoBlockPool.update``)
  append   new K and V rows into an 8-bit cache: blocks of 64 tokens of one head, one fp32
           scale each, codes int8 or e4m3; the block being filled stays bf16 in a tail
  decode   one query token per sequence over that cache (retrieval heads) and over the bf16
           sink + ring cache (streaming heads)
  prefill  a chunk of T query tokens over that cache and the chunk's own keys

``own = False`` computes them with elementary torch operations in 32 bits, ``own = True``
calls the package.
"""

import math

import torch

own = False

BLOCK = 64  # tokens that share a scale
CODE_MAX = {"int8": 127.0, "e4m3": 448.0}
CODE_TYPE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


# --------------------------------------------------------------------------- the cases
def listed():
    gqa = dict(Hq=32, Hkv=8, D=128, S=64, R=256)
    return [
        # a decode step of a running batch: one token each, a few requests finish; latency counts
        dict(name="tables_step_b256", op="tables", B=256, planes=2, page=128, max_len=16384, new=1, releases=5),
        # prompts of very different lengths admitted at once
        dict(name="tables_prompts_131k", op="tables", B=40, planes=4, page=256, max_len=32768, new=6000, releases=0),
        # the append of that step: one row per sequence and head, one sequence in 64 completes a block
        dict(name="append_step_b64", op="append", B=64, T=1, n=16384, Hkv=8, n_ret=2, D=128, S=64, R=256, page=128,
             ragged=True, code="int8"),
        # ragged prompts' chunks into a paged cache, 64-dim heads
        dict(name="append_ragged_d64", op="append", B=12, T=2048, n=4096, Hkv=4, n_ret=2, D=64, S=4, R=32, page=128,
             ragged=True, code="e4m3"),
        # a whole 32K prompt
        dict(name="append_prompt_32k", op="append", B=1, T=32768, n=0, Hkv=8, n_ret=4, D=128, S=64, R=256, page=0,
             ragged=False, code="e4m3"),
        # a few hundred tokens, small heads: launch latency
        dict(name="decode_tiny", op="decode", B=1, n=272, Hq=4, Hkv=4, n_ret=2, D=64, S=4, R=32, page=0, ragged=False,
             code="int8"),
        # one sequence of a million tokens (and a tail)
        dict(name="decode_1m", op="decode", B=1, n=(1 << 20) - 27, n_ret=2, page=0, ragged=False, code="int8", **gqa),
        # eight sequences of 128K
        dict(name="decode_b8_128k", op="decode", B=8, n=131072, n_ret=2, page=0, ragged=False, code="e4m3", **gqa),
        # a serving batch of ragged lengths (an empty one among them), pages of 128 tokens, lengths on the device
        dict(name="decode_ragged_b48", op="decode", B=48, n=32000, n_ret=2, page=128, ragged=True, code="int8", **gqa),
        # the last chunk of a 32K prompt, multi-head attention, a quarter of the heads retrieval
        dict(name="prefill_chunk_28k", op="prefill", B=1, T=4096, n=28672, Hq=32, Hkv=32, n_ret=8, D=128, S=64, R=256,
             page=0, code="int8"),
        # a follow-up question of a few hundred tokens to a long conversation, paged, odd lengths
        dict(name="prefill_turn_paged", op="prefill", B=2, T=333, n=9001, n_ret=4, page=256, code="e4m3", **gqa),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "decode", "decode", "prefill"])
    code = rng.choice(["int8", "e4m3"])
    if op == "tables":
        B = _log_int(rng, 1, 512)
        new = rng.choice([1, 1, _log_int(rng, 2, 4000)])
        new = min(new, max(1, 200000 // B))
        return dict(op=op, B=B, planes=rng.choice([1, 2, 3, 4, 8]), page=128 * rng.randint(1, 4),
                    max_len=_log_int(rng, 1000, 32768), new=new, releases=rng.randint(0, B // 8))
    D = rng.choice([64, 128])
    Hkv = rng.choice([2, 4, 8])
    n_ret = rng.randint(1, Hkv)
    S, R = rng.choice([(64, 256), (4, 32), (0, rng.randint(1, 300)), (rng.randint(1, 130), rng.randint(1, 300))])
    page = rng.choice([0, 128, 256, 384])
    heads = dict(Hkv=Hkv, n_ret=n_ret, D=D, S=S, R=R)
    if op == "append":
        ragged = page > 0 and rng.random() < 0.7
        T = rng.choice([1, _log_int(rng, 2, 8192)])
        B = _log_int(rng, 1, max(1, min(128, 32768 // (T * n_ret))))
        n = _log_int(rng, 64, 8192)
        return dict(op=op, B=B, T=T, n=n if T == 1 else n // BLOCK * BLOCK, page=page, ragged=ragged, code=code, **heads)
    heads["Hq"] = Hkv * rng.choice([1, 2, 4, 8])
    if op == "decode":
        ragged = rng.random() < 0.5
        n = _log_int(rng, 1, 400000)
        B = _log_int(rng, 1, max(1, min(64, 2000000 // (n * n_ret))))
        return dict(op=op, B=B, n=n, page=page, ragged=ragged, code=code, **heads)
    T = _log_int(rng, 1, 3000)
    per_head = 10 ** 9 * Hkv // (n_ret * heads["Hq"])  # query-key pairs that cost what the listed chunk costs
    n = _log_int(rng, 1, max(1, min(20000, per_head // T - T)))
    B = rng.randint(1, max(1, min(4, per_head // (T * (n + T)))))
    return dict(op=op, B=B, T=T, n=n, page=page, code=code, **heads)


# --------------------------------------------------------------------------- inputs
def _retrieval(c):
    """Which KV heads are retrieval heads: n_ret of them, spread over the heads."""
    return [1 if (h * c["n_ret"]) // c["Hkv"] != ((h + 1) * c["n_ret"]) // c["Hkv"] else 0 for h in range(c["Hkv"])]


def _heads(c):
    m = _retrieval(c)
    dev = "cuda"
    return (torch.tensor([h for h in range(c["Hkv"]) if m[h]], device=dev, dtype=torch.long),
            torch.tensor([h for h in range(c["Hkv"]) if not m[h]], device=dev, dtype=torch.long))


def _keys(g, *shape):
    """Rows with a few strong channels, as keys after the rotary layer have."""
    x = torch.randn(*shape, generator=g, device="cuda")
    gain = torch.ones(shape[-1], device="cuda")
    gain[3::29] = 3.0
    return (x * gain).to(torch.bfloat16)


def _values(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def _quantise(x, code):
    """[..., 64, D] -> codes of the same shape, fp32 scales [...]: scale = amax / 127 (448),
    code = x / scale rounded to nearest even, 0 where the scale is 0."""
    x = x.float()
    top = x.abs().amax(dim=(-1, -2))
    scale = top / torch.full_like(top, CODE_MAX[code])  # (a Python divisor would become a product)
    s = scale[..., None, None]
    y = torch.where(s > 0, x / s, torch.zeros_like(x)).clamp(-CODE_MAX[code], CODE_MAX[code])
    return (y.round() if code == "int8" else y).to(CODE_TYPE[code]), scale


def _stored(g, make, rows, D, code):
    codes, scale = _quantise(make(g, rows // BLOCK, BLOCK, D), code)
    return codes.reshape(rows, D), scale


def _ring_positions(lens, S, R):
    """Token position held by each sink + ring slot after len tokens, -1 if empty: [B, S + R] int32."""
    slot = torch.arange(S + R, device="cuda")[None, :]
    n = lens[:, None].long()
    last = n - 1 - (n - 1 - slot) % R  # the last position below n that is congruent to the slot
    pos = torch.where(slot < S, slot, last)
    ok = torch.where(slot < S, slot < n, (pos >= S) & (n > 0))
    return torch.where(ok, pos, torch.full_like(pos, -1)).to(torch.int32)


def _lengths(c, g):
    B, n = c["B"], c["n"]
    if not c.get("ragged"):
        return torch.full((B,), n, dtype=torch.int32, device="cuda")
    lens = (torch.rand(B, generator=g, device="cuda") * (n + 1)).long().clamp(max=n)
    lens[0] = n
    if B >= 4 and c["op"] == "decode":
        lens[1] = 0
        lens[2] = min(n, 41)
    if c["op"] == "append" and c["T"] > 1:
        lens = lens // BLOCK * BLOCK
    return lens.to(torch.int32)


def _pages(c, g, rows):
    """A pool's table for `rows` rows a sequence and head: ids in a random order."""
    per = -(-rows.long() // c["page"])  # [B]
    most = max(1, int(per.max()))
    total = int(per.sum()) * c["n_ret"]
    size = max(total, int(c["B"] * -(-(c["n"] + c.get("T", 0)) // c["page"]) * c["n_ret"]) if c["op"] == "append" else 0) + 3
    ids = torch.randperm(size, generator=g, device="cuda")
    have = (torch.arange(most, device="cuda")[None, None, :] < per[:, None, None]).expand(c["B"], c["n_ret"], most)
    table = torch.full(have.shape, -1, dtype=torch.int32, device="cuda")
    table[have] = ids[:total].to(torch.int32)
    return table, size


def _cache(c, g, lens, cap):
    """The 8-bit cache of sequences of `lens` tokens, with room for `cap` tokens each."""
    B, D, S, R = c["B"], c["D"], c["S"], c["R"]
    n_ret, n_str = c["n_ret"], c["Hkv"] - c["n_ret"]
    s = {"lens": lens}
    if c["page"]:
        s["table"], s["num_blocks"] = _pages(c, g, torch.as_tensor(cap, device="cuda").expand(B).clamp(min=1))
        rows, lead, slead = s["num_blocks"] * c["page"], (s["num_blocks"], c["page"]), (s["num_blocks"], c["page"] // BLOCK)
    else:
        cap64 = -(-max(int(torch.as_tensor(cap).max()), 1) // BLOCK) * BLOCK
        s["cap"] = cap64
        rows, lead, slead = B * n_ret * cap64, (B, n_ret, cap64), (B, n_ret, cap64 // BLOCK)
    for name, make in (("k", _keys), ("v", _values)):
        codes, scale = _stored(g, make, rows, D, c["code"])
        s[name + "_codes"] = codes.reshape(*lead, D)
        s[name + "_scale"] = scale.reshape(slead)
        s[name + "_tail"] = make(g, B, n_ret, BLOCK, D)
        s[name + "_sr"] = make(g, B, n_str, S + R, D)
    s["pos"] = _ring_positions(lens, S, R)
    return s


def _layer(c, s, Hq):
    """The package's owner of that cache."""
    import streaming_kv_cache_duo_gb300 as duo
    if c["page"]:
        table = s["table"]
        layer = duo.DuoKv8PagedLayer(c["B"], Hq, c["Hkv"], c["D"], c["S"], c["R"], c["page"], table.shape[2],
                                     s["num_blocks"], table, _retrieval(c), code=c["code"])
    else:
        layer = duo.DuoKv8Layer(c["B"], Hq, c["Hkv"], c["D"], c["S"], c["R"], s["cap"], _retrieval(c), code=c["code"])
    for name in BUFFERS:
        getattr(layer, name).copy_(s[name].reshape(getattr(layer, name).shape))
        s[name] = getattr(layer, name)
    return layer


BUFFERS = ("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail", "k_sr", "v_sr", "pos")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] == "tables":
        return _prepare_tables(c, g)
    lens = _lengths(c, g)
    if c["op"] == "append":
        new = torch.full((c["B"],), c["T"], dtype=torch.int32, device="cuda")
        if c["ragged"] and c["T"] > 1:
            new = (1 + torch.rand(c["B"], generator=g, device="cuda") * c["T"]).int().clamp(max=c["T"])
        s = _cache(c, g, lens, lens.long() + new.long())
        s["new"] = new
        if c["ragged"]:
            N = int(new.sum())
            s["cu_new"] = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), new.cumsum(0).int()])
            s["token_seq"] = torch.repeat_interleave(torch.arange(c["B"], device="cuda"), new.long()).int()
            k = torch.arange(N, device="cuda").int() - s["cu_new"][s["token_seq"].long()]
            s["token_pos"] = lens[s["token_seq"].long()] + k
            at = s["token_pos"].long()
            ids = s["table"][s["token_seq"].long(), :, at // c["page"]].long()
            s["slots"] = ids * c["page"] + (at % c["page"])[:, None]
            lead = (N,)
        else:
            lead = (c["B"], c["T"])
        s["k_new"], s["v_new"] = _keys(g, *lead, c["Hkv"], c["D"]), _values(g, *lead, c["Hkv"], c["D"])
        if own:
            import streaming_kv_cache_duo_gb300 as duo
            s["layer"] = _layer(c, s, c["Hkv"])
            if c["ragged"]:
                s["map"] = duo.DuoSlotMap(s["cu_new"], s["token_seq"], s["token_pos"], s["slots"])
    else:
        s = _cache(c, g, lens, lens)
        T = (c["T"],) if c["op"] == "prefill" else ()
        s["q"] = _values(g, c["B"], *T, c["Hq"], c["D"])
        if c["op"] == "prefill":
            s["k"], s["v"] = _keys(g, c["B"], *T, c["Hkv"], c["D"]), _values(g, c["B"], *T, c["Hkv"], c["D"])
        if own:
            s["layer"] = _layer(c, s, c["Hq"])
    s["case"] = c
    s["heads"] = _heads(c)
    return s


def _packed(c):
    """Tokens of a step's packed batch."""
    return c["B"] if c["new"] == 1 else c["B"] * c["new"] // 2 + 1


def _prepare_tables(c, g):
    B, planes, page = c["B"], c["planes"], c["page"]
    dev = dict(device="cuda")
    lens = (torch.rand(B, generator=g, **dev) * (c["max_len"] + 1)).int()
    gone = torch.randperm(B, generator=g, **dev)[: c["releases"]]
    new = torch.ones(B, dtype=torch.int32, **dev)
    N = _packed(c)
    if c["new"] > 1:  # a packed batch of N tokens, shared out at random
        share = torch.rand(B, generator=g, **dev) + 0.01
        share[gone] = 0
        new = (share / share.sum() * (N - 1)).int()
        lens = torch.where(torch.rand(B, generator=g, **dev) < 0.7, torch.zeros_like(lens), lens)
    new[gone] = -1
    most = -(-(c["max_len"] + N) // page)
    per = -(-lens.long() // page)
    held = int(per.sum()) * planes
    total = planes * (B * (c["max_len"] // page + 2) + N // page) + 17  # the pool
    ids = torch.randperm(total, generator=g, **dev).int()
    have = (torch.arange(most, **dev)[None, None, :] < per[:, None, None]).expand(B, planes, most)
    table = torch.full((B, planes, most), -1, dtype=torch.int32, **dev)
    table[have] = ids[:held]
    free = torch.full((total,), -1, dtype=torch.int32, **dev)
    free[: total - held] = ids[held:]
    s = dict(case=c, lens=lens, new=new, block_table=table, free_list=free, N=N, num_blocks=total,
             free_count=torch.tensor([total - held], dtype=torch.int32, **dev), seq_lens_out=torch.empty_like(lens),
             free_count_out=torch.empty(1, dtype=torch.int32, **dev))
    if own:
        import streaming_kv_cache_duo_gb300 as duo
        pool = duo.DuoBlockPool(B, planes, page, most, total, N)
        for name, t in (("block_table", table), ("free_list", free), ("free_count", s["free_count"]), ("seq_lens", lens)):
            getattr(pool, name).copy_(t)
        s["pool"] = pool
    return s


# --------------------------------------------------------------------------- one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    c = s["case"]
    if c["op"] == "tables":
        pool = s["pool"]
        m = pool.update(s["new"], seq_lens_out=s["seq_lens_out"], free_count_out=s["free_count_out"])
        return (pool.block_table, s["seq_lens_out"], pool.free_list, s["free_count_out"], m.cu_new, m.token_seq,
                m.token_pos, m.slots)
    layer = s["layer"]
    if c["op"] == "append":
        if c["ragged"]:
            layer.append_ragged(s["k_new"], s["v_new"], s["map"])
        else:
            layer.cache.n = c["n"]
            layer.append(s["k_new"], s["v_new"])
        return _buffers(s)
    layer.cache.n = c["n"]
    if c["op"] == "prefill":
        return layer.prefill(s["q"], s["k"], s["v"])
    return layer.decode_varlen(s["q"], s["lens"], c["n"]) if c["ragged"] else layer.decode(s["q"])


def _buffers(s):
    """The cache after an append."""
    return {name: s[name] for name in BUFFERS}


def _run_plain(s):
    op = s["case"]["op"]
    return {"tables": _plain_tables, "append": _plain_append, "decode": _plain_decode, "prefill": _plain_prefill}[op](s)


def _plain_tables(s):
    c, lens, new = s["case"], s["lens"].long(), s["new"].long()
    page, planes, N = c["page"], c["planes"], s["N"]
    dev = lens.device
    table, free = s["block_table"], s["free_list"]
    j = torch.arange(table.shape[2], device=dev)
    old = -(-lens // page)
    # finished requests give their blocks back, in the order (request, plane, block)
    gone = new < 0
    back = table[(gone[:, None, None] & (j < old[:, None, None])).expand_as(table)]
    count = s["free_count"].long()
    place = count + torch.arange(back.shape[0], device=dev)
    free[place] = back
    avail = count + back.shape[0]
    # new blocks, in the same order, from the end of the list
    add = new.clamp(min=0)
    grown = -(-(lens + add) // page)
    more = (grown - old) * planes
    upto = more.cumsum(0)
    served = (~gone) & ((more == 0) | (upto <= avail))
    base = upto - more
    fresh = (served[:, None, None] & (j >= old[:, None, None]) & (j < grown[:, None, None])).expand_as(table)
    order = base[:, None, None] + torch.arange(planes, device=dev)[None, :, None] * (grown - old)[:, None, None] \
        + (j - old[:, None, None])
    table[fresh] = free[(avail - 1 - order)[fresh]]
    lens_out = torch.where(gone, torch.zeros_like(lens), torch.where(served, lens + add, lens)).int()
    count_out = (avail - torch.where(served & (more > 0), upto, torch.zeros_like(upto)).max()).int()
    # the packed new tokens
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), add.cumsum(0)])
    i = torch.arange(N, device=dev)
    seq = (torch.searchsorted(cu, i, right=True) - 1).clamp(max=c["B"] - 1)
    real = i < cu[-1]
    at = lens[seq] + i - cu[seq]
    at = torch.where(real & served[seq], at, torch.full_like(at, -1))
    ids = table[seq, :, at.clamp(min=0) // page].long()
    slots = torch.where((at >= 0)[:, None], ids * page + (at.clamp(min=0) % page)[:, None], torch.full_like(ids, -1))
    seq = torch.where(real, seq, torch.full_like(seq, -1))
    return (table, lens_out, free, count_out, cu.int(), seq.int(), at.int(), slots)


def _plain_append(s):
    c, (ret, stream) = s["case"], s["heads"]
    B, S, R, D, n_ret = c["B"], c["S"], c["R"], c["D"], c["n_ret"]
    dev = ret.device
    if c["ragged"]:
        seq, at, start = s["token_seq"].long(), s["token_pos"].long(), s["cu_new"].long()
        end = s["lens"].long() + s["new"].long()
    else:
        i = torch.arange(B * c["T"], device=dev)
        seq, at = i // c["T"], c["n"] + i % c["T"]
        start = torch.arange(B + 1, device=dev) * c["T"]
        end = torch.full((B,), c["n"] + c["T"], device=dev)
    full = (at % BLOCK == BLOCK - 1).nonzero()[:, 0]  # the tokens that complete a block
    part = (at // BLOCK == end[seq] // BLOCK).nonzero()[:, 0]  # the tokens of the block that stays open
    if c["ragged"]:
        block = s["slots"][full] // BLOCK  # [M, n_ret]
    elif c["page"]:
        ids = s["table"][seq[full], :, at[full] // c["page"]].long()
        block = ids * (c["page"] // BLOCK) + (at[full] % c["page"] // BLOCK)[:, None]
    else:
        plane = seq[full][:, None] * n_ret + torch.arange(n_ret, device=dev)
        block = plane * (s["cap"] // BLOCK) + (at[full] // BLOCK)[:, None]
    back = torch.arange(BLOCK, device=dev) - (BLOCK - 1)
    src = full[:, None] + back  # [M, 64] packed rows of each block; those before the call are in the tail
    held = src < start[seq[full]][:, None]
    keep = (at >= 0) & ((at < S) | (at >= end[seq] - R))
    keep = keep.nonzero()[:, 0] if stream.numel() else keep.nonzero()[:0, 0]
    slot = torch.where(at[keep] < S, at[keep], S + (at[keep] - S) % R)
    s["pos"][seq[keep], slot] = at[keep].int()
    for name in ("k", "v"):
        x = s[name + "_new"].reshape(-1, c["Hkv"], D)
        rows = x[src.clamp(min=0)][:, :, ret]  # [M, 64, n_ret, D]
        tail = s[name + "_tail"][seq[full]].transpose(1, 2)
        rows = torch.where(held[:, :, None, None], tail, rows).transpose(1, 2)
        codes, scale = _quantise(rows, c["code"])
        whole = s[name + "_codes"].view(-1, BLOCK, D).view(torch.uint8)
        whole[block.reshape(-1)] = codes.reshape(-1, BLOCK, D).view(torch.uint8)
        s[name + "_scale"].view(-1)[block.reshape(-1)] = scale.reshape(-1)
        s[name + "_tail"][seq[part], :, at[part] % BLOCK] = x[part][:, ret]
        s[name + "_sr"][seq[keep], :, slot] = x[keep][:, stream]
    return _buffers(s)


def _dequantised(s, name, n):
    """fp32 rows [B, n_ret, blocks * 64, D] of the cache, the open block from the tail."""
    c = s["case"]
    B, n_ret, D = c["B"], c["n_ret"], c["D"]
    lens = s["lens"].long()
    codes, scale = s[name + "_codes"], s[name + "_scale"]
    nb = -(-max(n, 1) // BLOCK)
    if c["page"]:
        per = c["page"] // BLOCK
        ids = s["table"][:, :, : -(-nb // per)].long().clamp(min=0)
        x = codes[ids].reshape(B, n_ret, -1, BLOCK, D)[:, :, :nb].float()
        f = scale[ids].reshape(B, n_ret, -1)[:, :, :nb]
    else:
        x = codes.view(B, n_ret, -1, BLOCK, D)[:, :, :nb].float()
        f = scale[:, :, :nb]
    x = x * f[..., None, None]
    open_at = lens // BLOCK
    has = (lens % BLOCK > 0)[:, None, None, None]
    b = torch.arange(B, device=x.device)
    at = open_at.clamp(max=nb - 1)
    x[b, :, at] = torch.where(has, s[name + "_tail"].float(), x[b, :, at])
    return x.reshape(B, n_ret, nb * BLOCK, D)


def _softmax_rows(sc, vis, v, equation):
    """softmax over the last axis of the visible scores times v; 0 for a row that sees nothing."""
    sc = torch.where(vis, sc, torch.full_like(sc, -math.inf))
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    den = p.sum(-1, keepdim=True)
    return torch.einsum(equation, p, v) / torch.where(den > 0, den, torch.ones_like(den))


def _plain_decode(s):
    c, (ret, stream) = s["case"], s["heads"]
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    g = c["Hq"] // Hkv
    lens = s["lens"].long()
    q = s["q"].float().reshape(B, Hkv, g, D) / math.sqrt(D)
    o = torch.zeros_like(q)
    k = _dequantised(s, "k", c["n"])
    sc = torch.einsum("bhgd,bhkd->bhgk", q[:, ret], k)
    del k
    vis = torch.arange(sc.shape[-1], device=sc.device) < lens[:, None, None, None]
    v = _dequantised(s, "v", c["n"])
    o[:, ret] = _softmax_rows(sc, vis, v, "bhgk,bhkd->bhgd")
    pos = s["pos"].long()
    i = lens[:, None] - 1
    vis = (pos >= 0) & (pos <= i) & ((pos < c["S"]) | (i - pos < c["R"]))
    sc = torch.einsum("bhgd,bhkd->bhgk", q[:, stream], s["k_sr"].float())
    o[:, stream] = _softmax_rows(sc, vis[:, None, None, :], s["v_sr"].float(), "bhgk,bhkd->bhgd")
    return o.reshape(B, c["Hq"], D).to(torch.bfloat16)


def _plain_prefill(s):
    c, (ret, stream) = s["case"], s["heads"]
    B, T, n, Hkv, D = c["B"], c["T"], c["n"], c["Hkv"], c["D"]
    g = c["Hq"] // Hkv
    q = s["q"].float().reshape(B, T, Hkv, g, D).permute(0, 2, 3, 1, 4) / math.sqrt(D)
    kn, vn = (s[x].float().transpose(1, 2) for x in ("k", "v"))  # [B, Hkv, T, D]
    i = n + torch.arange(T, device=q.device)
    o = torch.zeros_like(q)
    k = torch.cat([_dequantised(s, "k", n)[:, :, :n], kn[:, ret]], 2)
    v = torch.cat([_dequantised(s, "v", n)[:, :, :n], vn[:, ret]], 2)
    vis = torch.arange(n + T, device=q.device) <= i[:, None]
    o[:, ret] = _softmax_rows(torch.einsum("bhgtd,bhkd->bhgtk", q[:, ret], k), vis, v, "bhgtk,bhkd->bhgtd")
    pos = torch.cat([s["pos"].long(), i.expand(B, T)], 1)[:, None, :]  # [B, 1, keys]
    row = i[:, None]
    vis = (pos >= 0) & (pos <= row) & ((pos < c["S"]) | (row - pos < c["R"]))
    k = torch.cat([s["k_sr"].float(), kn[:, stream]], 2)
    v = torch.cat([s["v_sr"].float(), vn[:, stream]], 2)
    sc = torch.einsum("bhgtd,bhkd->bhgtk", q[:, stream], k)
    o[:, stream] = _softmax_rows(sc, vis[:, None, None], v, "bhgtk,bhkd->bhgtd")
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, c["Hq"], D).to(torch.bfloat16)


# --------------------------------------------------------------------------- cost and truth
def _streaming_pairs(c):
    """Visible (query, key) pairs of a streaming head in a prefill chunk."""
    rows = range(c["n"], c["n"] + c["T"])
    K = c["S"] + c["R"]
    return sum(min(i + 1, K) for i in rows)


def work(case):
    c = case
    if c["op"] == "tables":
        # lengths twice, the free list's and the table's new entries, the maps of every new token
        B, planes = c["B"], c["planes"]
        tokens = _packed(c)
        blocks = B * planes / c["page"] if c["new"] == 1 else planes * (tokens // c["page"] + B // 2)
        freed = c["releases"] * planes * c["max_len"] / 2 / c["page"]
        return {"bytes": 16 * B + 8 * blocks + 8 * freed + tokens * (8 + planes * 8 + (4 * planes if c["new"] == 1 else 0)),
                "flops": 0}
    B, Hkv, D, S, R, n_ret = (c[k] for k in ("B", "Hkv", "D", "S", "R", "n_ret"))
    n_str = Hkv - n_ret
    if c["op"] == "append":
        # a row is read in bf16; it goes to the tail in bf16 or, with its block, to 8-bit codes
        T = c["T"]
        tokens = B * T if not c["ragged"] or T == 1 else B * (T + 1) // 2
        ring = B * min(T, S + R) * n_str * D * 2 * 2 * 2
        if T == 1:  # one step in 64 reads the tail and writes a block of codes
            return {"bytes": 2 * B * n_ret * D * (2 + 2 + (63 * 2 + 64) / 64) + ring, "flops": 4 * tokens * n_ret * D}
        return {"bytes": 2 * tokens * n_ret * D * (2 + 1) + 8 * tokens * n_ret / BLOCK + ring,
                "flops": 6 * tokens * n_ret * D}
    Hq = c["Hq"]
    mean = (c["n"] + 1) / 2 if c.get("ragged") and B > 1 else c["n"]
    cache = B * n_ret * (mean * D * 2 + mean / BLOCK * 8) + B * n_str * min(c["n"], S + R) * D * 4
    if c["op"] == "decode":
        return {"bytes": cache + 4 * B * Hq * D,
                "flops": 4 * D * B * (Hq // Hkv) * (n_ret * mean + n_str * min(c["n"], S + R))}
    T, n = c["T"], c["n"]
    pairs = n_ret * (T * n + T * (T + 1) // 2) + n_str * _streaming_pairs(c)
    return {"bytes": cache + B * T * D * (4 * Hq + 4 * Hkv), "flops": 4 * D * B * (Hq // Hkv) * pairs}


def exact(case, seed):
    c = case
    if c["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_attention, "prefill": _exact_attention}[c["op"]](c, s)


def _exact_append(c, s):
    """Sequence by sequence: the rows of every block that is full after the call, put together
    from the tail and the new tokens and divided by their scale in 64 bits. The rest of the
    buffers is as it was."""
    ret, stream = s["heads"]
    out = {name: s[name].double() if s[name].dtype != torch.int8 else None for name in BUFFERS}
    out["pos"] = None
    S, R, D = c["S"], c["R"], c["D"]
    top = CODE_MAX[c["code"]]
    begin = 0
    for b in range(c["B"]):
        n, t = int(s["lens"][b]), int(s["new"][b])
        for name in ("k", "v"):
            x = s[name + "_new"].reshape(-1, c["Hkv"], D)[begin:begin + t].double()
            for r in range(c["n_ret"]):
                first = n // BLOCK * BLOCK
                rows = torch.cat([s[name + "_tail"][b, r, : n - first].double(), x[:, ret[r]]])
                for j in range(rows.shape[0] // BLOCK):
                    w = rows[j * BLOCK:(j + 1) * BLOCK]
                    scale = w.abs().max() / top
                    blk = first // BLOCK + j
                    if c["page"]:
                        per = c["page"] // BLOCK
                        where = (int(s["table"][b, r, blk // per]), blk % per)
                        at = (where[0], slice(where[1] * BLOCK, where[1] * BLOCK + BLOCK))
                    else:
                        where, at = (b, r, blk), (b, r, slice(blk * BLOCK, blk * BLOCK + BLOCK))
                    out[name + "_scale"][where] = scale
                    if c["code"] == "e4m3":
                        y = w / scale
                        e = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
                        step = torch.exp2(e - 3)
                        out[name + "_codes"][at] = (torch.round(y / step) * step).clamp(-top, top)
                left = rows.shape[0] % BLOCK
                done = rows.shape[0] - left
                if left:
                    fresh = max(done, n - first)
                    out[name + "_tail"][b, r, fresh - done:left] = rows[fresh:]
            for p in range(n, n + t):
                if p < S or p >= n + t - R:
                    slot = p if p < S else S + (p - S) % R
                    out[name + "_sr"][b, :, slot] = x[p - n][stream]
        begin += t
    return out


def _exact_attention(c, s):
    """Head by head over the keys a query sees, in 64 bits."""
    ret, stream = (h.tolist() for h in s["heads"])
    B, Hq, Hkv, D = c["B"], c["Hq"], c["Hkv"], c["D"]
    g = Hq // Hkv
    T = c.get("T", 1)
    q = s["q"].reshape(B, T, Hq, D)
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(s["lens"][b])
        first = n if c["op"] == "prefill" else n - 1
        at = torch.arange(first, first + T, device="cuda")
        if c["op"] == "decode" and n == 0:
            continue
        for h in range(Hkv):
            parts = {}
            for name in ("k", "v"):
                if h in ret:
                    r = ret.index(h)
                    full = n // BLOCK * BLOCK
                    if c["page"]:
                        ids = s["table"][b, r, : -(-full // c["page"])].long()
                        codes = s[name + "_codes"][ids].reshape(-1, D)[:full]
                        scale = s[name + "_scale"][ids].reshape(-1)[: full // BLOCK]
                    else:
                        codes, scale = s[name + "_codes"][b, r, :full], s[name + "_scale"][b, r, : full // BLOCK]
                    rows = [codes.double() * scale.double().repeat_interleave(BLOCK)[:, None],
                            s[name + "_tail"][b, r, : n - full].double()]
                    held = torch.arange(n, device="cuda")
                else:
                    r = stream.index(h)
                    held = s["pos"][b].long()
                    rows = [s[name + "_sr"][b, r][held >= 0].double()]
                    held = held[held >= 0]
                if c["op"] == "prefill":
                    rows.append(s[name][b, :, h].double())
                    held = torch.cat([held, at])
                parts[name] = torch.cat(rows)
            for j in range(h * g, h * g + g):
                for t0 in range(0, T, 1024):
                    i = at[t0:t0 + 1024, None]
                    sees = held[None, :] <= i
                    if h not in ret:
                        sees &= (held[None, :] < c["S"]) | (i - held[None, :] < c["R"])
                    sc = q[b, t0:t0 + 1024, j].double() @ parts["k"].T / math.sqrt(D)
                    p = torch.softmax(sc.masked_fill(~sees, -math.inf), -1)
                    out[b, t0:t0 + 1024, j] = p @ parts["v"]
    return out if c["op"] == "prefill" else out[:, 0]
