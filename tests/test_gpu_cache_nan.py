"""Queries without a softmax over the paged 8-bit cache: the row is NaN however the work is cut, and no other row is."""
import pytest
import torch

import cache_exact as exact
import cache_ref as ref
import speculative_block_draft_gb300 as pkg

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("n,bad", [(100, float("nan")), (9000, float("nan")), (9000, float("inf")), (100, float("-inf")), (0, float("nan")), (0, float("inf")), (0, float("-inf"))])
def test_bad_query(n, bad, own, dtype):
    """One element of row 1 is NaN or infinite. Over no keys at all a row is zeros, whatever its query."""
    T, H, Hq, D, rows, dt = 64, 2, 6, 128, 4, DT[dtype]
    N = -(-n // T) + 1
    k, v, ks, vs = ref.random_cache(1, N, H, T, D, 1)
    table = ref.random_table([n], T, N, N, 2)
    g = torch.Generator().manual_seed(3)
    q = torch.randn((rows, Hq, D), generator=g).to(dt)
    ko, vo = (torch.randn((rows, H, D), generator=g).to(dt) for _ in range(2))
    q[1, :, 17] = bad
    out = torch.full((rows, Hq, D), 7.0, dtype=dt, device="cuda")
    cache = pkg.Cache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), max_requests=1, max_q=rows, n_q_heads=Hq)
    cache.attention(q.cuda(), ints([n]), ints(table), out, k_own=ko.cuda() if own else None, v_own=vo.cuda() if own else None)
    assert cache.check_errors() == 0
    got = out.cpu()
    if n == 0 and not own:
        assert not got.any()
        return
    assert got[1].isnan().all()
    rest = [0, 2, 3]
    kd, vd = (torch.cat([exact.values(c[0], s[0], table[0], n, T), (o if own else o[:0]).double().transpose(0, 1)], 1)
              for c, s, o in ((k, ks, ko), (v, vs, vo)))
    want, tol = exact.attention(q[rest], kd, vd, dt)
    assert torch.all((got[rest].double() - want).abs() <= tol)


def test_keys_of_nothing_but_nan():
    """A stretch of NaN keys that several CTAs hold by themselves makes the rows that see it NaN."""
    T, H, D, n, dt = 64, 1, 128, 9000, torch.bfloat16
    N = -(-n // T)
    k, v, ks, vs = ref.random_cache(1, N, H, T, D, 5)
    k[:, 40:60] = 0x7F
    table = [list(range(N))]
    q = torch.randn((3, 2, D), generator=torch.Generator().manual_seed(1)).to(dt).cuda()
    out = torch.zeros_like(q)
    cache = pkg.Cache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), max_requests=1, max_q=3, n_q_heads=2)
    cache.attention(q, ints([n]), ints(table), out)
    assert out.isnan().all()
    cache.attention(q, ints([n]), ints(table), out, window=n - 60 * T)
    assert not out.isnan().any()
