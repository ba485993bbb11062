"""Ring tables of the paged 8-bit cache, filled by the calls that a program makes: reserve, append, attend, truncate. What a ring
returns is compared with the rows as a table without reuse holds them."""
import random

import pytest
import torch

import cache_exact as exact
import cache_ref as ref
import speculative_block_draft_gb300 as pkg

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Ring:
    """One request in a ring of `width` blocks, and the same rows appended to a table that never reuses a block (host, 64 bits).
    The size of the rows changes from block to block, so a block that is read at another one's scale shows."""

    H, Hq, D = 2, 4, 64

    def __init__(self, T, width, seed):
        self.T, self.width, self.g = T, width, torch.Generator().manual_seed(seed)
        blocks = width + 3
        self.dev = [x.cuda() for x in ref.random_cache(1, blocks, self.H, T, self.D, seed)]
        self.cache = pkg.Cache(*self.dev, max_requests=1, max_q=64, n_q_heads=self.Hq)
        self.pool = pkg.BlockPool(T, ring=True)
        perm = list(range(blocks))
        random.Random(seed).shuffle(perm)
        self.d = {"lens": ints([0]), "table": ints([[-1] * width]), "free": ints(perm), "free_count": ints([blocks])}
        self.n = 0
        n_all = 60
        self.codes = [torch.zeros((1, n_all, self.H, T, self.D), dtype=torch.uint8) for _ in range(2)]
        self.scales = [torch.ones((1, n_all, self.H)) for _ in range(2)]

    def grow(self, n):
        slots = ints([0] * n)
        self.pool.reserve(ints([n]), **self.d, slots=slots, row_start=ints([0, 0]), granted=ints([0]))
        size = torch.tensor([2.0 ** ((p // self.T * 5) % 9 - 4) for p in range(self.n, self.n + n)])
        rows = [(torch.randn((1, n, self.H, self.D), generator=self.g) * size[:, None, None]).bfloat16() for _ in range(2)]
        self.cache.append(slots, rows[0].cuda(), rows[1].cuda())
        for i in range(2):
            ref.append(self.codes[i], self.scales[i], rows[i], list(range(self.n, self.n + n)), self.T)
        self.n += n

    def shrink(self, n):
        self.pool.truncate(ints([n]), **self.d)
        self.n = n

    def attend(self, rows, window, causal, own=False, first=0):
        """The last `rows` positions attend (or, with own rows, ones behind them); `first`: the first position seen at all."""
        q = torch.randn((rows, self.Hq, self.D), generator=self.g).bfloat16()
        ko, vo = (torch.randn((rows, self.H, self.D), generator=self.g).bfloat16() if own else None for _ in range(2))
        out = torch.zeros_like(q, device="cuda")
        self.cache.attention(q.cuda(), self.d["lens"], self.d["table"], out, window=window, causal=causal,
                             k_own=ko.cuda() if own else None, v_own=vo.cuda() if own else None)
        assert self.cache.check_errors() == 0
        table = list(range(-(-self.n // self.T)))
        kd, vd = (exact.values(c[0], s[0], table, self.n, self.T) for c, s in zip(self.codes, self.scales))
        if own:
            kd, vd = (torch.cat([x, o.double().transpose(0, 1)], 1) for x, o in ((kd, ko), (vd, vo)))
        pos = torch.arange(kd.shape[1])[None]
        at = torch.arange(rows)[:, None] + (self.n if own else self.n - rows)
        seen = (pos >= first).expand(rows, -1)
        if causal:
            seen = seen & (pos <= at) & ((pos > at - window) if window else (pos >= 0))
        elif window:
            seen = seen & (pos >= self.n - window)
        want, tol = exact.attention(q, kd, vd, torch.bfloat16, seen=seen)
        err = (out.cpu().double() - want).abs()
        assert torch.all(err <= tol), f"{self.n} tokens: off by {float((err / tol).max()):.2f} of the tolerance"


def blocks_for(window, rows, T):
    """The blocks that the documentation asks for."""
    return -(-(window + rows - 1) // T) + 1


@pytest.mark.parametrize("T,window,rows", [(64, 64, 8), (16, 64, 9), (16, 50, 16), (32, 90, 5), (128, 200, 1), (16, 17, 40)])
def test_speculation_on_a_ring(T, window, rows):
    """Blocks of rows appended, verified causally, and mostly given back, at every offset within a block."""
    r, rng = Ring(T, blocks_for(window, rows, T), T + rows), random.Random(rows)
    r.grow(window + 3)
    while r.n <= (r.width + 2) * T:
        kept = r.n
        r.grow(rows)
        r.attend(rows, window, True)
        r.shrink(kept + rng.randint(0, rows))
        r.attend(min(rows, 3), window, False, own=True)
        r.attend(rows, window, True, own=True)
        r.grow(rng.randint(1, T // 4))


def test_the_case_that_lost_keys():
    """Window 64, blocks of 64, 125 tokens and 8 more: the block of positions 0..63 is taken again by position 128, while
    the first of the 8 rows still sees 62 and 63."""
    r = Ring(64, blocks_for(64, 8, 64), 1)
    assert r.width == 3
    r.grow(125)
    r.grow(8)
    r.attend(8, 64, True)
    r.shrink(126)
    r.attend(1, 64, False)
    r.attend(1, 64, True)


@pytest.mark.parametrize("T,width", [(16, 5), (32, 4), (64, 2), (128, 2)])
def test_a_ring_without_window_shows_whole_blocks(T, width):
    """Rows that only grow: a call sees the blocks that have not been taken again, and nothing of the one that has."""
    r = Ring(T, width, T)
    for n in (3, T, 1, T - 4, 2 * T, 1, 7, T - 8, T // 2, T // 2 - 1, 1, 1, 2 * T + 3):
        r.grow(n)
        whole = max(0, (-(-r.n // T) - width) * T)
        r.attend(1, 0, False, first=whole)
        r.attend(2, 0, True, own=True, first=whole)
    assert r.n > (width + 2) * T
