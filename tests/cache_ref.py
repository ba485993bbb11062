"""Plain 64-bit restatement of the paged 8-bit context cache, on CPU tensors (imported by the cache tests)."""
import math

import torch

E4M3 = torch.float8_e4m3fn


def pool_reserve(T, ring, lens, table, free, count, n_new, requests=None, n_slots=None):
    """Request by request. lens list, table list of lists, free list, count: changed in place; returns
    (count, slots, row_start, granted)."""
    width, avail = len(table[0]), count
    blocks = (lambda x: min(-(-x // T), width)) if ring else (lambda x: -(-x // T))
    sum_need, taken, slots, start, granted, seen = 0, 0, [], [0], [], set()
    for i, n in enumerate(n_new):
        r = requests[i] if requests is not None else i
        ok = 0 <= r < len(lens) and r not in seen and 0 <= n <= 1 << 20
        seen.add(r)
        ok = ok and (ring or lens[r] + n <= width * T)
        if ok:
            need = blocks(lens[r] + n) - blocks(lens[r])
            sum_need += need
            ok = need == 0 or sum_need <= avail
        if ok:
            had, end = blocks(lens[r]), lens[r] + n
            for k in range(need):
                table[r][had + k] = free[avail - 1 - taken]
                taken += 1
            for p in range(lens[r], end):
                over = ring and p // T + width <= (end - 1) // T
                slots.append(-1 if over else table[r][(p // T) % width] * T + p % T)
            lens[r] = end
        granted.append(int(ok))
        start.append(len(slots))
    n_slots = len(slots) if n_slots is None else n_slots
    return avail - taken, (slots + [-1] * n_slots)[:n_slots], start, granted


def pool_truncate(T, ring, lens, table, free, count, new_len, requests=None):
    width = len(table[0])
    blocks = (lambda x: min(-(-x // T), width)) if ring else (lambda x: -(-x // T))
    back, seen = [], set()
    for i, n in enumerate(new_len):
        r = requests[i] if requests is not None else i
        if not 0 <= r < len(lens) or r in seen:
            continue
        seen.add(r)
        if 0 <= n < lens[r]:
            for k in range(blocks(n), blocks(lens[r])):
                back.append(table[r][k])
                table[r][k] = -1
            lens[r] = n
    for g, b in enumerate(back):
        free[count + len(back) - 1 - g] = b
    return count + len(back)


def fit_scale(amax):
    """Smallest power of two >= 2^-64 with amax <= 448 * it."""
    s = 2.0 ** -64
    while amax > 448.0 * s:
        s *= 2
    return s


def append(codes, scales, rows, slots, T, layer0=0):
    """codes [L][N][H][T][D] uint8, scales [L][N][H] fp32 (both changed), rows [l][n][H][D]."""
    owner = {}
    for r, s in enumerate(slots):
        if s >= 0:
            owner.setdefault(s // T, {})[s % T] = r
    x = rows.double()
    for block, toks in owner.items():
        t, r = list(toks), list(toks.values())
        for li in range(rows.shape[0]):
            for h in range(rows.shape[2]):
                v = x[li, r, h]
                a = v.abs()
                a = a[torch.isfinite(a)]
                new = fit_scale(float(a.max()) if a.numel() else 0.0)
                old = float(scales[layer0 + li, block, h])
                c = codes[layer0 + li, block, h]
                if 0 not in toks:
                    if new > old:
                        c.copy_((c.view(E4M3).double() * (old / new)).float().to(E4M3).view(torch.uint8))
                    new = max(new, old)
                scales[layer0 + li, block, h] = new
                c[t] = (v / new).clamp(-448, 448).float().to(E4M3).view(torch.uint8)


def attention(q, k_codes, v_codes, k_scale, v_scale, lens, table, counts, dtype, k_own=None, v_own=None, window=0, causal=False,
              scale=None, requests=None):
    """q [rows][Hq][D] and own rows as given to the call, codes [N][H][T][D] uint8 of one layer. Returns the
    outputs in 64 bits and, element by element, how far a call may be off:
      the rounding of the result to dtype (u = eps / 2 relative),
      the probabilities as sums of e4m3 terms: each term leaves 2^-4 of what it rounds, so 2^-8 of p with the
        two terms of bf16 and 2^-12 with the three of f16, and at least half the smallest code, 2^-10,
        where the row's largest weight is kept above 2^4: 2^-14 of it,
      the scores: D products of 2 D roundings at 2^-23, and 2^-22 of the exponent's argument itself; a score
        that is off by d (base e) changes p, and the sum of them, by d relative."""
    D, Hq, H, N, T = q.shape[2], q.shape[1], k_codes.shape[1], k_codes.shape[0], k_codes.shape[2]
    scale = D ** -0.5 if scale is None else scale
    kd = k_codes.view(E4M3).double() * k_scale.double()[..., None, None]
    vd = v_codes.view(E4M3).double() * v_scale.double()[..., None, None]
    out, tol = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    terms, u = (2, 2.0 ** -8) if dtype == torch.bfloat16 else (3, 2.0 ** -11)
    row = 0
    for b, n in enumerate(counts):
        r = requests[b] if requests is not None else b
        length, width = lens[r], len(table[r])
        ids = [table[r][(p // T) % width] for p in range(length)]
        there = torch.tensor([0 <= i < N and p >= length - width * T for p, i in enumerate(ids)], dtype=torch.bool)
        safe = [i if 0 <= i < N else 0 for i in ids]
        at = [p % T for p in range(length)]
        k, v = kd[safe, :, at], vd[safe, :, at]                                     # [len][H][D]
        if k_own is not None:
            k = torch.cat([k, k_own[row:row + n].double()])
            v = torch.cat([v, v_own[row:row + n].double()])
            there = torch.cat([there, torch.ones(n, dtype=torch.bool)])
        pos = torch.arange(length + (n if k_own is not None else 0))
        for i in range(n):
            me = length + i if k_own is not None else length - n + i
            ok = there.clone()
            if causal:
                ok &= pos <= me
                if window:
                    ok &= pos > me - window
            elif window:
                ok &= pos >= length - window
            for h in range(Hq):
                if not ok.any():
                    continue
                qh, kk, vv = q[row + i, h].double(), k[ok, h // (Hq // H)], v[ok, h // (Hq // H)]
                s = (kk @ qh) * scale
                size = (kk.abs() @ qh.abs()) * abs(scale)
                off = float(size.max()) * 2 * D * 2.0 ** -23 + float(s.abs().max()) * 2.0 ** -22
                p = torch.softmax(s, 0)
                o, reach = p @ vv, p @ vv.abs()
                out[row + i, h] = o
                tol[row + i, h] = (u * o.abs() + (2.0 ** (-4 * terms) + 2 * off + 2.0 ** -20) * reach
                                   + 2.0 ** -14 * float(p.max()) * vv.abs().sum(0) + 2.0 ** -26)
        row += n
    return out, tol


def random_cache(L, N, H, T, D, seed, spread=3):
    """Codes of normal values and scales of 2^-8 .. 2^-(8 - spread)."""
    g = torch.Generator().manual_seed(seed)
    codes = [(torch.randn((L, N, H, T, D), generator=g) * 64).clamp(-448, 448).to(E4M3).view(torch.uint8) for _ in range(2)]
    scales = [torch.exp2(torch.randint(-8, -8 + spread + 1, (L, N, H), generator=g).float()) for _ in range(2)]
    return codes[0], codes[1], scales[0], scales[1]


def random_table(lens, T, N, width, seed):
    """A table of distinct random blocks; the rest of each row -1."""
    g = torch.Generator().manual_seed(seed)
    perm, at, table = torch.randperm(N, generator=g).tolist(), 0, []
    for n in lens:
        need = min(-(-n // T), width)
        table.append(perm[at:at + need] + [-1] * (width - need))
        at += need
    assert at <= N and math.isfinite(at)
    return table
