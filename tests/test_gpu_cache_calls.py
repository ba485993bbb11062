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


def test_an_object_dropped_while_its_calls_run():
    """Calls on a stream other than the object's: its memory is not given to others before they are done."""
    T, H, Hq, D, n, dt = 64, 2, 10, 128, 3000, torch.bfloat16
    k, v, ks, vs = ref.random_cache(1, 50, H, T, D, 1)
    dev, table = [x.cuda() for x in (k, v, ks, vs)], ref.random_table([n], T, 50, 47, 2)
    q = torch.randn((4, Hq, D), generator=torch.Generator().manual_seed(3)).to(dt)
    qd, lens, td, out = q.cuda(), ints([n]), ints(table), torch.zeros((4, Hq, D), dtype=dt, device="cuda")
    pool_state = {"lens": ints([0]), "table": ints([[-1, -1]]), "free": ints([0, 1, 2]), "free_count": ints([3])}
    slots, start, granted, new = ints([7] * 40), ints([0, 0]), ints([0]), ints([40])
    cache, pool = pkg.Cache(*dev, max_requests=1, max_q=4, n_q_heads=Hq), pkg.BlockPool(64)
    sizes = [x.numel() for x in (cache.workspace, pool.scratch)]
    taken = [x.data_ptr() for x in (cache.workspace, pool.scratch)]
    side = torch.cuda.Stream()
    cache.attention(qd, lens, td, out)                 # first launches load the kernels, which may wait for the device
    pool.reserve(ints([0]), **pool_state, slots=slots, row_start=start, granted=granted)
    with torch.cuda.stream(side):
        torch.cuda._sleep(1000)
    out.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)                 # some 0.2 s
        cache.attention(qd, lens, td, out)
    pool.reserve(new, **pool_state, slots=slots, row_start=start, granted=granted, stream=side)
    del cache, pool
    assert not side.query(), "the calls were done too early to tell"
    others = [torch.empty(m, dtype=torch.uint8, device="cuda") for m in sizes]
    assert all(o.data_ptr() != p for o, p in zip(others, taken))
    side.synchronize()
    want, tol = exact.attention(q, exact.values(k[0], ks[0], table[0], n, T), exact.values(v[0], vs[0], table[0], n, T), dt)
    assert torch.all((out.cpu().double() - want).abs() <= tol)
    assert slots.tolist() == list(range(128, 168)) and granted.tolist() == [1]
