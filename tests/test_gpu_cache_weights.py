"""Attention over the paged 8-bit cache where most of a row's weight lies in one key and the rest in very many small ones."""
import math

import pytest
import torch

import cache_exact as exact
import speculative_block_draft_gb300 as pkg

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def peaked(n, share, D, H, Hq, rows, dtype, T, spread, at, seed):
    """One key (at position `at`, with a value of 0) that holds about `share` of each row, and n - 1 others of scores 0, or normal
    ones of deviation `spread`, whose values have a mean of their own. Codes, scales, a shuffled table and queries."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    N = -(-n // T) + 2
    table = torch.randperm(N, generator=torch.Generator().manual_seed(seed))[:-(-n // T)]
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")                             # noqa: E731
    kd = randn(N, H, T, D) * (64 * spread)
    kd[..., 0] = 0
    vd = randn(N, H, T, D) * 40 + 90
    block, token = int(table[at // T]), at % T
    kd[block, :, token], vd[block, :, token] = 0, 0
    kd[block, :, token, 0] = 256
    k, v = (x.clamp(-448, 448).to(exact.E4M3).view(torch.uint8) for x in (kd, vd))
    ks, vs = torch.full((N, H), 2.0 ** -6, device="cuda"), torch.full((N, H), 2.0 ** -7, device="cuda")
    # column 0 gives the one key its score, the others give the rest theirs: queries of about 1 against keys of `spread`
    q = randn(rows, Hq, D)
    q = q / q[..., 1:].norm(dim=-1, keepdim=True) * math.sqrt(D)
    q[..., 0] = (math.log(share / (1 - share) * n) + spread * spread / 2) * math.sqrt(D) / 4 + 0.05 * torch.arange(rows, device="cuda")[:, None]
    return k, v, ks, vs, table.tolist(), q.to(DT[dtype])


def check(n, share, D, H, Hq, rows, dtype, T=64, spread=0.0, at=0, copies=1, seed=0, **kw):
    """`copies` requests with the same context and the same queries: the more of them, the fewer CTAs share one."""
    k, v, ks, vs, table, q = peaked(n, share, D, H, Hq, rows, dtype, T, spread, at, seed)
    cache = pkg.Cache(k[None], v[None], ks[None], vs[None], max_requests=copies, max_q=rows, n_q_heads=Hq)
    qd = q.repeat(copies, 1, 1)
    out = torch.zeros_like(qd)
    cache.attention(qd, ints([n]), ints([table]), out, requests=ints([0] * copies), **kw)
    assert cache.check_errors() == 0
    want, tol = exact.attention(q, exact.values(k, ks, table, n, T), exact.values(v, vs, table, n, T), DT[dtype])
    err = (out.double().view(copies, rows, Hq, D) - want).abs()
    assert want.abs().amax() > 0.03
    assert torch.all(err <= tol), f"off by {float((err / tol).max()):.2f} of the tolerance, {float(err.max() / want.abs().max()):.3g} of the output"


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [1024, 4096, 16384, 131072])
@pytest.mark.parametrize("share", [0.5, 0.8, 0.95])
@pytest.mark.parametrize("spread", [0.0, 1.0])
def test_tail_behind_a_peak(n, share, spread, dtype):
    check(n, share, 128, 2, 10, 1, dtype, spread=spread, seed=n)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,T,rows,Hq,H", [(64, 16, 1, 4, 4), (64, 64, 5, 10, 2), (128, 64, 1, 16, 8), (128, 32, 5, 20, 4), (128, 64, 9, 20, 4),
                                           (128, 128, 12, 10, 2), (256, 32, 1, 5, 1), (256, 64, 8, 10, 2), (256, 32, 9, 10, 2), (256, 64, 12, 10, 2)])
def test_tail_in_one_piece(D, T, rows, Hq, H, dtype):
    """Every padding of the rows, with so many requests that each context is one CTA's."""
    check(16384, 0.8, D, H, Hq, rows, dtype, T=T, copies=640 // H, seed=D + rows)
    check(16384, 0.8, D, H, Hq, rows, dtype, T=T, spread=0.5, at=9000, copies=640 // H, seed=D + rows)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("nats", [6, 8, 9, 10, 10.6, 11, 12, 13, 14])
def test_tails_of_equal_scores(nats, dtype):
    """All keys but the first at the same distance below it: each is rounded the same way."""
    n = 131072
    share = math.exp(nats) / (math.exp(nats) + n)
    check(n, share, 128, 1, 5, 1, dtype, at=n - 1, seed=1)
    check(n, share, 128, 1, 5, 1, dtype, at=0, copies=320, seed=2)


def test_calls_repeat_themselves():
    """The same call gives the same bits."""
    k, v, ks, vs, table, q = peaked(9000, 0.5, 128, 4, 20, 5, "bf16", 64, 1.0, 0, 3)
    cache = pkg.Cache(k[None], v[None], ks[None], vs[None], max_requests=1, max_q=5, n_q_heads=20)
    outs = [torch.zeros_like(q) for _ in range(6)]
    for o in outs:
        cache.attention(q, ints([9000]), ints([table]), o, causal=True)
    assert all(torch.equal(o, outs[0]) for o in outs[1:])
