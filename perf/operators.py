"""The paged 8-bit context cache: block tables and slots, the quantising append, and attention over it.

Each case is one pass through one operator. In the plain form it is elementary torch arithmetic in 32 bits; with ``own`` set, the calls a
program makes of ``speculative_block_draft_gb300.Cache``. Storage (both forms read and write the same tensors):

  codes   e4m3 [layer][block][kv head][token of the block][head_dim], value = code * scale
  scales  fp32 [layer][block][kv head], one array for K and one for V
  table   int32 [request][blocks]: the block that holds position p of a request is table[request][(p // T) % blocks]
  free    int32 [blocks]: a stack of unused blocks, free_count of them
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_EXP = -64          # smallest scale: 2^-64

#: what several cases share: the 5-layer drafter's 8 K/V heads of 128 behind 40 query heads
DFLASH2 = {"q_heads": 40, "kv_heads": 8, "head_dim": 128}


def listed():
    return [
        # a round's bookkeeping of the batched drafter: 32 requests give back the rejected rows and reserve the next block's 8
        {"name": "slots_round_32x8", "op": "slots", "requests": 32, "len_lo": 512, "len_hi": 16384, "rows": 8, "back": 5, "block": 64},
        # admission of many prompts at once: 1024 requests of 512 rows
        {"name": "slots_prompts_1024x512", "op": "slots", "requests": 1024, "len_lo": 0, "len_hi": 700, "rows": 512, "back": 3, "block": 16},
        # the batched drafter's appends of one round: 1..8 committed rows of 32 requests, every layer
        {"name": "append_round_32x", "op": "append", "layers": 5, "requests": 32, "rows_lo": 1, "rows_hi": 8, "kv_heads": 8, "head_dim": 128,
         "block": 64, "start": 200, "dtype": "bf16"},
        # a long prompt entering the cache, every layer
        {"name": "append_prompt_16384", "op": "append", "layers": 5, "requests": 1, "rows_lo": 16384, "rows_hi": 16384, "kv_heads": 8,
         "head_dim": 128, "block": 64, "start": 0, "dtype": "bf16"},
        # a fp32 drafter with small odd sizes: prompts that end inside a block
        {"name": "append_odd_f32", "op": "append", "layers": 2, "requests": 7, "rows_lo": 61, "rows_hi": 333, "kv_heads": 3, "head_dim": 64,
         "block": 16, "start": 5, "dtype": "f32"},
        # one token of one request, heads not shared: the latency of a call
        {"name": "attn_token_1x1024", "op": "attn", "requests": 1, "rows": 1, "ragged": False, "len_lo": 1024, "len_hi": 1024, "window": 0,
         "own_rows": False, "causal": False, "q_heads": 8, "kv_heads": 8, "head_dim": 128, "block": 64, "dtype": "bf16"},
        # the draft block of one request: 8 rows and their own K/V beside a window of the context
        {"name": "attn_block_1x8_w2048", "op": "attn", "requests": 1, "rows": 8, "ragged": False, "len_lo": 4096, "len_hi": 4096, "window": 2048,
         "own_rows": True, "causal": False, **DFLASH2, "block": 64, "dtype": "f16"},
        # the batched drafter: 32 blocks of 5 rows, ragged contexts, window
        {"name": "attn_block_32x5_w2048", "op": "attn", "requests": 32, "rows": 5, "ragged": False, "len_lo": 512, "len_hi": 16384, "window": 2048,
         "own_rows": True, "causal": False, **DFLASH2, "block": 64, "dtype": "bf16"},
        # plain decoding of 32 requests over their whole contexts, one token each
        {"name": "attn_token_32x16384", "op": "attn", "requests": 32, "rows": 1, "ragged": False, "len_lo": 512, "len_hi": 16384, "window": 0,
         "own_rows": False, "causal": False, **DFLASH2, "block": 64, "dtype": "bf16"},
        # long contexts of few requests: the key axis has to be split
        {"name": "attn_token_4x131072", "op": "attn", "requests": 4, "rows": 1, "ragged": False, "len_lo": 131072, "len_hi": 131072, "window": 0,
         "own_rows": False, "causal": False, **DFLASH2, "block": 64, "dtype": "bf16"},
        # verification of drafted blocks: 1..9 rows a request, already appended, causal; wide heads, smaller blocks
        {"name": "attn_verify_16x9_hd256", "op": "attn", "requests": 16, "rows": 9, "ragged": True, "len_lo": 500, "len_hi": 8192, "window": 0,
         "own_rows": False, "causal": True, "q_heads": 20, "kv_heads": 4, "head_dim": 256, "block": 32, "dtype": "bf16"},
        # a small drafter's heads and short odd contexts
        {"name": "attn_odd_3x4_hd64", "op": "attn", "requests": 3, "rows": 4, "ragged": True, "len_lo": 1, "len_hi": 301, "window": 0,
         "own_rows": True, "causal": False, "q_heads": 4, "kv_heads": 4, "head_dim": 64, "block": 16, "dtype": "f16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["slots", "append", "append", "attn", "attn", "attn", "attn"])
    block = rng.choice([16, 32, 64, 128])
    if op == "slots":
        lo = _log(rng, 1, 3000)
        return {"op": op, "requests": _log(rng, 1, 1024), "len_lo": lo, "len_hi": lo + _log(rng, 1, 8000), "rows": _log(rng, 1, 512),
                "back": rng.randint(0, 9), "block": block}
    dtype = rng.choice(["bf16", "f16"])
    hd = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 3, 4, 8])
    if op == "append":
        requests, layers = _log(rng, 1, 64), rng.randint(1, 5)
        top = max(1, min(12000, 90_000_000 // (layers * kv * hd)) // requests)     # bytes stay below the largest listed case's
        lo = _log(rng, 1, top)
        return {"op": op, "layers": layers, "requests": requests, "rows_lo": lo, "rows_hi": min(top, lo + rng.randint(0, 40)),
                "kv_heads": kv, "head_dim": hd, "block": block, "start": rng.randint(0, 300), "dtype": rng.choice([dtype, "f32"])}
    requests, rows, group = _log(rng, 1, 32), _log(rng, 1, 16), rng.choice([1, 2, 4, 5, 8])
    # bytes of the cache, and operations at 50 a byte, stay below the largest listed case's
    tokens = min(500_000_000 // (kv * hd), 50_000_000_000 // (4 * kv * group * hd * rows))
    hi = _log(rng, 8, max(16, min(100_000, tokens // requests)))
    own_rows = rng.random() < 0.4
    return {"op": op, "requests": requests, "rows": rows, "ragged": rng.random() < 0.4, "len_lo": max(1, int(hi * rng.uniform(0.05, 1.0))),
            "len_hi": hi, "window": rng.choice([0, 0, _log(rng, 16, 4096)]), "own_rows": own_rows, "causal": rng.random() < 0.4,
            "q_heads": kv * group, "kv_heads": kv, "head_dim": hd, "block": block, "dtype": dtype}


# ---- sizes that follow from a case alone --------------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n whole numbers evenly from lo to hi: every seed has the same ones, in another order."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _row_counts(c):
    if c["op"] == "append":
        return _spread(c["rows_lo"], c["rows_hi"], c["requests"])
    return _spread(1, c["rows"], c["requests"]) if c["ragged"] else [c["rows"]] * c["requests"]


DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _first_key(c, length, rows):
    """First cached position that any row of a request reads."""
    if not c["window"]:
        return 0
    newest = length if not c["causal"] else (length if c["own_rows"] else length - rows) + 1
    return max(0, newest - c["window"])


def work(case):
    c = case
    if c["op"] == "slots":
        new = c["requests"] * (-(-c["rows"] // c["block"]))
        return {"bytes": 4 * (c["requests"] * (6 + c["rows"]) + 4 * new), "flops": c["requests"] * c["rows"]}
    if c["op"] == "append":
        rows, size = sum(_row_counts(c)), 4 if c["dtype"] == "f32" else 2
        n = c["layers"] * rows * c["kv_heads"] * c["head_dim"] * 2
        blocks = sum(-(-r // c["block"]) for r in _row_counts(c)) * c["layers"] * c["kv_heads"] * 2
        return {"bytes": n * (size + 1) + 4 * rows + 4 * blocks, "flops": 3 * n}
    keys = flops = 0
    lens = _spread(c["len_lo"], c["len_hi"], c["requests"])
    rows = _row_counts(c)
    for length, r in zip(lens, rows):
        n = max(0, length - _first_key(c, length, r))
        keys += n
        flops += 4 * c["q_heads"] * c["head_dim"] * r * (n + (r if c["own_rows"] else 0))
    total = sum(rows)
    small = total * 2 * c["head_dim"] * (2 * c["q_heads"] + (2 * c["kv_heads"] if c["own_rows"] else 0))
    scales = -(-keys // c["block"]) * (8 * c["kv_heads"] + 4)
    return {"bytes": keys * c["kv_heads"] * c["head_dim"] * 2 + small + scales + 8 * c["requests"], "flops": flops}


# ---- inputs --------------------------------------------------------------------------------------------------------------
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _shuffled(values, seed):
    order = torch.randperm(len(values), generator=torch.Generator().manual_seed(seed))
    return [values[i] for i in order.tolist()]


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(blocks_each, width, seed):
    """Block tables over a shuffled pool, and the pool's unused rest as a stack."""
    used = sum(blocks_each)
    pool = used + max(4, used // 4)
    perm = torch.randperm(pool, generator=torch.Generator().manual_seed(seed + 1)).to(torch.int32)
    table = torch.full((len(blocks_each), width), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(blocks_each):
        table[r, :n] = perm[at:at + n]
        at += n
    return table.cuda(), perm[at:].cuda(), pool


def _random_codes(shape, g):
    """Normal values as the quantising append leaves them: the largest of a block near the top of the code range."""
    x = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    for part in x.view(-1).split(1 << 28):
        part.copy_((torch.randn(part.shape, generator=g, device="cuda") * 64).clamp_(-448, 448))
    return x


def _random_scales(shape, g):
    return torch.exp2(torch.randint(-8, -4, shape, generator=g, device="cuda").float())


def prepare(case, seed):
    c, g = case, _generator(seed)
    T, B = c["block"], c["requests"]
    if c["op"] == "slots":
        # kept rows of each request, and the rows behind them that the target rejected in the last round
        both = _shuffled([(n, n + c["back"] * (i % 3) // 2) for i, n in enumerate(_spread(c["len_lo"], c["len_hi"], B))], seed)
        base, have = [b for b, _ in both], [h for _, h in both]
        width = max(-(-(max(h, b + c["rows"])) // T) for h, b in zip(have, base)) + 1
        each = [-(-h // T) for h in have]
        table, rest, pool = _tables(each, width, seed)
        extra = sum(-(-(b + c["rows"]) // T) for b in base)       # room for every request's next rows
        rest = torch.cat([rest, torch.arange(pool, pool + extra, dtype=torch.int32, device="cuda")])
        free = torch.full((pool + extra,), -1, dtype=torch.int32, device="cuda")
        free[:rest.numel()] = rest
        rows = B * c["rows"]
        return {"case": c, "keep": _ints(base), "n_new": _ints([c["rows"]] * B), "lens": _ints(have), "table": table, "free": free,
                "free_count": _ints([rest.numel()]), "slots": torch.empty(rows + 3, dtype=torch.int32, device="cuda"),
                "row_start": torch.empty(B + 1, dtype=torch.int32, device="cuda"), "granted": torch.empty(B, dtype=torch.int32, device="cuda")}
    if c["op"] == "append":
        both = _shuffled([(n, (c["start"] * (i + 1)) % (3 * T)) for i, n in enumerate(_row_counts(c))], seed)
        counts, starts = [n for n, _ in both], [p for _, p in both]
        each = [-(-(s + n) // T) for s, n in zip(starts, counts)]
        table, _, pool = _tables(each, max(each), seed)
        slots = []
        host = table.cpu().tolist()
        for r, (s, n) in enumerate(zip(starts, counts)):
            slots += [host[r][p // T] * T + p % T for p in range(s, s + n)]
        rows, shape = sum(counts), (c["layers"], pool, c["kv_heads"], T, c["head_dim"])
        kv = [torch.randn((c["layers"], rows, c["kv_heads"], c["head_dim"]), generator=g, device="cuda").to(DTYPES[c["dtype"]]) for _ in range(2)]
        # blocks that already hold rows have scales of 2^-8 to 2^-5: normal rows outgrow the smaller ones
        return {"case": c, "k": _random_codes(shape, g), "v": _random_codes(shape, g), "k_scale": _random_scales(shape[:3], g),
                "v_scale": _random_scales(shape[:3], g), "k_rows": kv[0], "v_rows": kv[1], "slots": _ints(slots)}
    lens = _shuffled(_spread(c["len_lo"], c["len_hi"], B), seed)
    counts = _row_counts(c)
    each = [-(-n // T) for n in lens]
    table, _, pool = _tables(each, max(each), seed)
    shape = (1, pool, c["kv_heads"], T, c["head_dim"])
    rows, dt = sum(counts), DTYPES[c["dtype"]]
    state = {"case": c, "k": _random_codes(shape, g), "v": _random_codes(shape, g), "k_scale": _random_scales(shape[:3], g),
             "v_scale": _random_scales(shape[:3], g), "lens": _ints(lens), "table": table,
             "q": (2 * torch.randn((rows, c["q_heads"], c["head_dim"]), generator=g, device="cuda")).to(dt),
             "row_start": _ints([sum(counts[:i]) for i in range(B + 1)]),
             "out": torch.empty((rows, c["q_heads"], c["head_dim"]), dtype=dt, device="cuda"), "k_own": None, "v_own": None}
    if c["own_rows"]:
        for name in ("k_own", "v_own"):
            state[name] = torch.randn((rows, c["kv_heads"], c["head_dim"]), generator=g, device="cuda").to(dt)
    return state


# ---- the plain forms -----------------------------------------------------------------------------------------------------
def _plain_slots(s):
    c, T = s["case"], s["case"]["block"]
    lens, table, free, count = s["lens"], s["table"], s["free"], s["free_count"]
    at = torch.arange(table.shape[1], device="cuda", dtype=torch.int32)[None]
    # give back the blocks behind the kept rows: request by request, a request's blocks in order, the last one given first
    keep = torch.minimum(lens, s["keep"])
    before, after = (lens + T - 1) // T, (keep + T - 1) // T
    gone = (at >= after[:, None]) & (at < before[:, None])
    order = torch.cumsum(gone.flatten(), 0) - 1
    total = (before - after).sum()
    spot = torch.where(gone.flatten(), count + total - 1 - order, free.numel())
    wide = torch.cat([free, free.new_zeros(1)])
    wide[spot] = table.flatten()
    free.copy_(wide[:-1])
    table.copy_(torch.where(gone, -1, table))
    count.add_(total)
    # reserve the next rows
    n = s["n_new"].clamp_min(0)
    before, after = (keep + T - 1) // T, (keep + n + T - 1) // T
    fits = after <= table.shape[1]
    need = torch.where(fits, after - before, 0)
    sums = torch.cumsum(need, 0)
    granted = fits & ((need == 0) | (sums <= count))
    need, n = torch.where(granted, need, 0), torch.where(granted, n, 0)
    first = torch.cumsum(need, 0) - need
    took = need.sum()
    new = (at >= before[:, None]) & (at < (before + need)[:, None])
    pick = count - 1 - (first[:, None] + at - before[:, None])
    table.copy_(torch.where(new, free[pick.clamp(0, free.numel() - 1)], table))
    count.sub_(took)
    lens.copy_(keep + n)
    s["granted"].copy_(granted)
    s["row_start"][0] = 0
    s["row_start"][1:] = torch.cumsum(n, 0)
    row = torch.arange(s["slots"].numel(), device="cuda", dtype=torch.int32)
    r = (torch.searchsorted(s["row_start"], row, right=True) - 1).clamp_max(c["requests"] - 1)
    pos = keep[r] + row - s["row_start"][r]
    slot = table[r, ((pos // T) % table.shape[1])] * T + pos % T
    s["slots"].copy_(torch.where(row < s["row_start"][-1], slot, -1))
    return {k: s[k] for k in ("slots", "row_start", "granted", "table", "lens", "free", "free_count")}


def _block_exponent(amax):
    """Smallest k with amax <= 448 * 2^k, at least MIN_EXP."""
    m, e = torch.frexp(amax)
    k = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, k, MIN_EXP).clamp_min(MIN_EXP)


def _plain_append_one(codes, scales, rows, slots, T):
    """codes [L][N][H][T][D], scales [L][N][H], rows [L][n][H][D]."""
    L, N, H, _, D = codes.shape
    x = rows.float()
    block, token = (slots // T).long(), (slots % T).long()
    amax = torch.where(torch.isfinite(x), x.abs(), 0).amax(3)                        # [L][n][H]
    top = torch.zeros((L, N, H), device="cuda").index_reduce_(1, block, amax, "amax")
    touched, fresh = torch.zeros((2, N), device="cuda").unbind(0)
    touched[block] = 1
    fresh.index_reduce_(0, block, (token == 0).float(), "amax")
    new = torch.ldexp(torch.ones_like(top), _block_exponent(top))
    new = torch.where(fresh[None, :, None] > 0, new, torch.maximum(new, scales))
    new = torch.where(touched[None, :, None] > 0, new, scales)
    # codes that stay in a block whose scale grew
    old = torch.where(new > scales, 1, 0) * (1 - fresh[None, :, None])
    ratio = torch.where(old > 0, scales / new, 1)
    codes.copy_(torch.where(old[..., None, None] > 0, (codes.float() * ratio[..., None, None]).to(codes.dtype).view(torch.uint8),
                            codes.view(torch.uint8)).view(codes.dtype))
    scales.copy_(new)
    q = (x / new[:, block][..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(codes.dtype)
    codes.view(torch.uint8)[:, block, :, token] = q.view(torch.uint8).permute(1, 0, 2, 3)


def _plain_append(s):
    T = s["case"]["block"]
    _plain_append_one(s["k"], s["k_scale"], s["k_rows"], s["slots"], T)
    _plain_append_one(s["v"], s["v_scale"], s["v_rows"], s["slots"], T)
    return {k: s[k] for k in ("k", "v", "k_scale", "v_scale")}


def _plain_attention(s):
    c, T = s["case"], s["case"]["block"]
    B, H, G, D, R = c["requests"], c["kv_heads"], c["q_heads"] // c["kv_heads"], c["head_dim"], c["rows"]
    lens, start = s["lens"].long(), s["row_start"].long()
    counts = start[1:] - start[:-1]
    # the blocks that any row reads, from the first one of each request on
    newest = lens if not c["causal"] else (lens if c["own_rows"] else lens - counts) + 1
    first = (newest - c["window"]).clamp_min(0) if c["window"] else torch.zeros_like(lens)
    b0 = first // T
    span = c["len_hi"] if not c["window"] else min(c["len_hi"], c["window"] + R + T)
    cols = b0[:, None] + torch.arange(-(-span // T) + 1, device="cuda")
    blocks = torch.gather(s["table"].long(), 1, cols % s["table"].shape[1]).clamp_min(0)    # [B][n]
    pos = (cols[:, :, None] * T + torch.arange(T, device="cuda")).flatten(1)                  # [B][keys]
    there = pos < lens[:, None]

    def values(codes, scales):
        x = codes[0].view(torch.uint8)[blocks].view(torch.float8_e4m3fn).float() * scales[0][blocks][..., None, None]
        x = x.permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
        return torch.where(there[:, None, :, None], x, 0)

    k, v = values(s["k"], s["k_scale"]), values(s["v"], s["v_scale"])
    i = torch.arange(R, device="cuda")
    rows = (start[:-1, None] + i).clamp_max(s["q"].shape[0] - 1)                              # [B][R]
    live = i < counts[:, None]
    q = s["q"].float()[rows].reshape(B, R, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, R * G, D)
    scores = (q @ k.transpose(2, 3)).reshape(B, H, R, G, -1) * D ** -0.5
    at = (lens[:, None] + i if c["own_rows"] else lens[:, None] - counts[:, None] + i)        # [B][R] positions of the rows
    seen = there[:, None].expand(B, R, -1) & (pos >= first[:, None])[:, None]
    if c["causal"]:
        seen = seen & (pos[:, None] <= at[:, :, None])
        if c["window"]:
            seen = seen & (pos[:, None] > at[:, :, None] - c["window"])
    if c["own_rows"]:
        ko, vo = (s[n].float()[rows].permute(0, 2, 1, 3) for n in ("k_own", "v_own"))         # [B][H][R][D]
        scores = torch.cat([scores, (q @ ko.transpose(2, 3)).reshape(B, H, R, G, R) * D ** -0.5], -1)
        mine = live[:, None].expand(B, R, R)
        if c["causal"]:
            mine = mine & (i[None, :] <= i[:, None])
            if c["window"]:
                mine = mine & (i[None, :] > i[:, None] - c["window"])
        seen, v = torch.cat([seen, mine], -1), torch.cat([v, vo], 2)
    seen = seen[:, None, :, None]
    scores = torch.where(seen, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(scores - torch.where(top == -math.inf, 0, top)), 0)
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(B, H, R * G, -1) @ v).reshape(B, H, R, G, D)
    o = torch.where(total > 0, o / total, 0).permute(0, 2, 1, 3, 4).reshape(B, R, H * G, D)
    s["out"][rows[live]] = o[live].to(s["out"].dtype)
    return s["out"]


# ---- the framework's calls -----------------------------------------------------------------------------------------------
def _cache(s):
    """The cache object that a program keeps beside its tensors."""
    if "cache" not in s:
        import speculative_block_draft_gb300 as dflash
        c = s["case"]
        if c["op"] == "slots":
            s["cache"] = dflash.BlockPool(c["block"], max_requests=c["requests"])
        elif c["op"] == "append":
            s["cache"] = dflash.Cache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        else:
            s["cache"] = dflash.Cache(s["k"], s["v"], s["k_scale"], s["v_scale"], max_requests=c["requests"], max_q=c["rows"], n_q_heads=c["q_heads"])
    return s["cache"]


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"slots": _plain_slots, "append": _plain_append, "attn": _plain_attention}[c["op"]](s)
    cache = _cache(s)
    if c["op"] == "slots":
        cache.truncate(s["keep"], s["lens"], s["table"], s["free"], s["free_count"])
        cache.reserve(s["n_new"], s["lens"], s["table"], s["free"], s["free_count"], s["slots"], s["row_start"], s["granted"])
        return {k: s[k] for k in ("slots", "row_start", "granted", "table", "lens", "free", "free_count")}
    if c["op"] == "append":
        cache.append(s["slots"], s["k_rows"], s["v_rows"])
        return {k: s[k] for k in ("k", "v", "k_scale", "v_scale")}
    cache.attention(s["q"], s["lens"], s["table"], s["out"], row_start=s["row_start"], k_own=s["k_own"], v_own=s["v_own"],
                    window=c["window"], causal=c["causal"])
    return s["out"]


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------------
def _exact_append(s):
    T, dev = s["case"]["block"], "cuda"
    slots = s["slots"].cpu().tolist()
    spans, i = [], 0
    while i < len(slots):                                  # rows of one block stand together
        j = i
        while j < len(slots) and slots[j] // T == slots[i] // T:
            j += 1
        spans.append((i, j, slots[i] // T, torch.tensor([x % T for x in slots[i:j]], device=dev)))
        i = j
    out = {}
    for name in ("k", "v"):
        codes, scale = s[name].double(), s[name + "_scale"].double()
        for a, b, n, tok in spans:
            x = s[name + "_rows"][:, a:b].double()                                    # [L][m][H][D]
            big = x.abs().amax((1, 3))
            need = torch.exp2(torch.ceil(torch.log2(big / 448.0)).clamp_min(MIN_EXP))
            need = torch.where(big <= 448.0 * need / 2, need / 2, need)               # log2 may round up across a power of two
            need = torch.where(big > 448.0 * need, need * 2, need).clamp_min(2.0 ** MIN_EXP)
            if 0 not in tok.tolist():
                grown = torch.maximum(need, scale[:, n])
                codes[:, n] = (codes[:, n] * (scale[:, n] / grown)[..., None, None]).float().to(torch.float8_e4m3fn).double()
                need = grown
            scale[:, n] = need
            codes[:, n, :, tok] = (x / need[:, None, :, None]).float().to(torch.float8_e4m3fn).double().permute(0, 2, 1, 3)
        out[name], out[name + "_scale"] = codes, scale
    return out


def _exact_attention(s):
    c, T = s["case"], s["case"]["block"]
    H, G, D = c["kv_heads"], c["q_heads"] // c["kv_heads"], c["head_dim"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lens, start, table = s["lens"].tolist(), s["row_start"].tolist(), s["table"]
    for r in range(c["requests"]):
        n, a, b = lens[r], start[r], start[r + 1]
        ids = table[r, :-(-n // T)].long()
        keys = [[], []]
        for side, name in enumerate(("k", "v")):
            x = s[name][0].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double() * s[name + "_scale"][0][ids].double()[:, :, None, None]
            x = x.transpose(0, 1).reshape(H, -1, D)[:, :n]                            # [H][n][D]
            if c["own_rows"]:
                x = torch.cat([x, s[name + "_own"][a:b].double().transpose(0, 1)], 1)
            keys[side] = x
        where = torch.arange(keys[0].shape[1], device="cuda")                         # own row j stands at position n + j
        for j in range(b - a):
            at = n + j if c["own_rows"] else n - (b - a) + j
            ok = torch.ones_like(where, dtype=torch.bool)
            if c["causal"]:
                ok = where <= at
                if c["window"]:
                    ok = ok & (where > at - c["window"])
            elif c["window"]:
                ok = where >= n - c["window"]
            if not bool(ok.any()):
                continue
            q = s["q"][a + j].double().reshape(H, G, D)
            w = torch.softmax(((q @ keys[0][:, ok].transpose(1, 2)) / math.sqrt(D)), -1)
            out[a + j] = (w @ keys[1][:, ok]).reshape(H * G, D)
    return out


def exact(case, seed):
    if case["op"] == "slots":
        return None                                        # whole numbers: compared as they are
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attention(s)
