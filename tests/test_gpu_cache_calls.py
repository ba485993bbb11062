"""Calls of the paged 8-bit context cache at the ends of what their arguments may be."""
import pytest
import torch

import cache_exact as exact
import cache_ref as ref
import speculative_block_draft_gb300 as pkg

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 31 - 6])
@pytest.mark.parametrize("own", [False, True])
def test_largest_windows(window, own):
    """A window of (nearly) 2^31 shows everything, also to rows that stand before the first position."""
    T, H, Hq, D, n, dt = 16, 2, 4, 64, 9, torch.bfloat16
    for length in (1, 3, 40):
        k, v, ks, vs = ref.random_cache(1, 4, H, T, D, length)
        g = torch.Generator().manual_seed(length)
        q = torch.randn((n, Hq, D), generator=g).to(dt)
        ko, vo = (torch.randn((n, H, D), generator=g).to(dt) if own else None for _ in range(2))
        out = torch.zeros_like(q, device="cuda")
        cache = pkg.Cache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), max_requests=1, max_q=n, n_q_heads=Hq)
        cache.attention(q.cuda(), ints([length]), ints([[2, 0, 1]]), out, causal=True, window=window, k_own=ko.cuda() if own else None,
                        v_own=vo.cuda() if own else None)
        kd, vd = (exact.values(c[0], s[0], [2, 0, 1], length, T) for c, s in ((k, ks), (v, vs)))
        if own:
            kd, vd = (torch.cat([x, o.double().transpose(0, 1)], 1) for x, o in ((kd, ko), (vd, vo)))
        at = torch.arange(n)[:, None] + (length if own else length - n)
        seen = torch.arange(kd.shape[1])[None] <= at
        rows = seen.any(1)
        want, tol = exact.attention(q[rows], kd, vd, dt, seen=seen[rows])
        got = out.cpu()
        assert torch.all((got[rows].double() - want).abs() <= tol) and not got[~rows].any()


@pytest.mark.parametrize("power", [0, 60, 110, 118])
def test_largest_queries(power):
    """bf16 queries of up to 2^120 against keys and a scale as small: the scores are ordinary numbers."""
    T, H, Hq, D, n, dt = 64, 1, 5, 128, 300, torch.bfloat16
    k, v, ks, vs = ref.random_cache(1, 6, H, T, D, power)
    ks.fill_(2.0 ** -6 if power == 0 else 2.0 ** -64)
    scale = D ** -0.5 if power == 0 else D ** -0.5 * 2.0 ** (58 - power)
    q = (torch.randn((3, Hq, D), generator=torch.Generator().manual_seed(1)) * 2.0 ** power).to(dt)
    out = torch.zeros_like(q, device="cuda")
    cache = pkg.Cache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), max_requests=1, max_q=3, n_q_heads=Hq)
    cache.attention(q.cuda(), ints([n]), ints([[4, 2, 0, 1, 5]]), out, scale=scale)
    table = [4, 2, 0, 1, 5]
    want, tol = exact.attention(q, exact.values(k[0], ks[0], table, n, T), exact.values(v[0], vs[0], table, n, T), dt, scale=scale)
    assert torch.all((out.cpu().double() - want).abs() <= tol)


def test_a_call_without_rows():
    """A step in which no request has a row: nothing is done, whatever max_q and however many requests there are."""
    k, v, ks, vs = (x.cuda() for x in ref.random_cache(1, 4, 2, 16, 64, 1))
    cache = pkg.Cache(k, v, ks, vs, max_requests=3, max_q=4, n_q_heads=4)
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    own = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    lens, table = ints([5, 6, 7]), ints([[0], [1], [2]])
    assert cache.attention(q, lens, table, q.clone(), row_start=ints([0, 0, 0, 0]), causal=True) == 0
    assert cache.attention(q, lens, table, q.clone(), row_start=ints([0, 0, 0, 0]), k_own=own, v_own=own) == 0
    assert cache.attention(q, lens, table, q.clone()) == 0
    assert cache.append(ints([]), own, own) == 0
    assert cache.check_errors() == 0
