"""Bounded waits of the paged cache's attention: one that runs out is reported, ends by itself, and leaves the next call right."""
import time

import numpy as np
import pytest
import torch

import cache_exact as exact
import cache_ref as ref
import dflash_synth as syn
import speculative_block_draft_gb300 as pkg

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("cta", [0, 7])
@pytest.mark.parametrize("dtype,hd,Hq,H,rows,own,longest", [("bf16", 128, 10, 2, 5, True, 3000), ("f16", 64, 2, 2, 1, False, 3000),
                                                            ("bf16", 256, 5, 1, 9, False, 3000), ("bf16", 128, 24, 2, 16, True, 20000)])
def test_a_wait_that_runs_out(dtype, hd, Hq, H, rows, own, longest, cta):
    """With a limit of 20 ms one CTA gets none of its keys: a tile each of 3000 tokens, several of 20000 (in three chunks of rows).
    Its outputs are undefined; every warp of it leaves."""
    T, lens, dt = 64, [longest, 900, 70], DT[dtype]
    N = sum(-(-n // T) for n in lens)
    k, v, ks, vs = ref.random_cache(1, N, H, T, hd, 1)
    table = ref.random_table(lens, T, N, -(-longest // T), 2)
    g = torch.Generator().manual_seed(3)
    q = torch.randn((3 * rows, Hq, hd), generator=g).to(dt)
    ko, vo = (torch.randn((3 * rows, H, hd), generator=g).to(dt) if own else None for _ in range(2))
    out = torch.zeros_like(q, device="cuda")
    cache = pkg.Cache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), max_requests=3, max_q=rows, n_q_heads=Hq)
    dev = dict(q=q.cuda(), lens=ints(lens), table=ints(table), out=out, k_own=ko.cuda() if own else None, v_own=vo.cuda() if own else None)
    cache.attention(**dev)
    assert cache.check_errors() == 0
    first = out.clone()
    cache.set_wait_limit(20000)
    cache.debug_stall(cta)
    t0 = time.time()
    cache.attention(**dev)
    with pytest.raises(pkg.DFlashError) as e:
        cache.check_errors()
    assert e.value.status == pkg.DFLASH_ETIMEOUT
    assert time.time() - t0 < 0.9                      # below the waits' default limit
    assert cache.check_errors() == 0                   # cleared, and the hook was for one call
    cache.attention(**dev)
    cache.set_wait_limit(0)
    cache.attention(**dev)
    assert cache.check_errors() == 0
    assert torch.equal(out, first)
    for b, n in enumerate(lens):
        mine = slice(b * rows, (b + 1) * rows)
        kd, vd = (exact.values(c[0], s[0], table[b], n, T) for c, s in ((k, ks), (v, vs)))
        if own:
            kd, vd = (torch.cat([x, o[mine].double().transpose(0, 1)], 1) for x, o in ((kd, ko), (vd, vo)))
        want, tol = exact.attention(q[mine], kd, vd, dt)
        assert torch.all((out[mine].cpu().double() - want).abs() <= tol)


def test_a_handle_passes_its_limit_and_stall_on():
    """A handle with the paged cache: in a stalled draft call with a limit of 20 ms the attention's waits end as soon as the
    projections' do. Two layers' attention with the default limit would take 2 s and more; all waits in turn,
    some twenty, take less than one."""
    from speculative_block_draft_gb300.session import Session
    cfg = syn.DraftConfig("w_limit", n_layers=2, d=256, n_q_heads=4, n_kv_heads=2, head_dim=64, inter=512, n_taps=2, target_hidden=256,
                          vocab=1000, gamma=5, window=0, ctx_len=70, wdtype="q4", adtype="bf16", seed=77, batch=1, cache_blocks=8)
    s = Session(syn.make_model(cfg, norm_jitter=0.1), ctx_capacity=200)
    assert s.project([0], [70], syn.taps_rows(cfg, cfg.seed, 0, 0, 70)) == 0
    anchors = np.array([5], dtype=np.int32)
    good = s.draft([0], anchors, logits=True)
    assert s.check() == 0
    s.h.set_wait_limit(20000, stream=s.stream)
    s.h.debug_stall(0)
    t0 = time.time()
    assert s.draft([0], anchors, logits=False)["rc"] == 0
    with pytest.raises(pkg.DFlashError) as e:
        s.check()
    assert e.value.status == pkg.DFLASH_ETIMEOUT
    assert time.time() - t0 < 1.5
    assert s.check() == 0
    s.h.set_wait_limit(0, stream=s.stream)
    again = s.draft([0], anchors, logits=True)
    assert s.check() == 0 and np.array_equal(good["logits"], again["logits"])
    s.close()
