"""The 5120-wide 4-bit drafter with its context K/V in the paged 8-bit cache, at the sizes of its full workloads: what the cache
holds against the oracle's K/V (the newest rows), and drafts against the oracle run on what the cache holds."""
import numpy as np
import pytest
import torch

import dflash_synth as syn
import oracle
from dflash_synth import CONFIGS
from parity_util import cached_model, compare_block

pytestmark = pytest.mark.gpu


def stored(cfg, cache, r, P):
    """K and V [L][n][kvd] of request r's window as the cache holds them, and their scales."""
    n = min(P, cfg.window)
    assert int(cache["lens"][r]) == P
    table = cache["table"][r].tolist()
    at = range(P - n, P)
    blocks, tokens = [table[(p // 64) % len(table)] for p in at], [p % 64 for p in at]
    out = []
    for name in ("k", "v"):
        codes = cache[name].view(torch.float8_e4m3fn)[:, blocks, :, tokens].double()            # [n][L][H][hd]
        scale = cache[name + "_scale"][:, blocks].permute(1, 0, 2).double()[..., None]
        both = (codes * scale, scale.expand_as(codes))
        out.append([np.ascontiguousarray(x.permute(1, 0, 2, 3).reshape(cfg.n_layers, n, -1).cpu().numpy()) for x in both])
    return out


def check_rows(cfg, got, want):
    """As the small cases do: a code within 2^-4, a subnormal one within half its step of 2^-9, twice when its block's
    scale grew, and the projection's own f16 rounding."""
    for (val, scale), ref in zip(got, want):
        n = ref.shape[1]
        val, scale = val[:, -n:], scale[:, -n:]
        slack = 2.0 ** -5 * np.sqrt(np.mean(ref ** 2))
        assert np.all(np.abs(val - ref) <= 2.0 ** -4 * (np.abs(ref) + slack) + slack + 2.0 ** -9 * scale)


def run(cfg, lengths, checked):
    m = cached_model(CONFIGS["c3"], norm_jitter=0.1)
    model = syn.HostModel(cfg, m.mats, dict(m.vecs))
    model.vecs["block_pos"] = syn.normal(cfg.seed, "block_pos", (32, cfg.d), 0.02)[: cfg.gamma].copy()
    model.vecs["mask_emb"] = syn.normal(cfg.seed, "mask_emb", (32, cfg.d), 0.02)[: cfg.gamma - 1].copy()
    from speculative_block_draft_gb300.session import Session
    s, orc, B = Session(model, max_batch=cfg.batch, ctx_capacity=cfg.window), oracle.Oracle(model), cfg.batch
    newest = {b: syn.taps_rows(cfg, cfg.seed, b, int(lengths[b]) - 40, 40) for b in checked}
    for b in range(B):
        done = 0
        while done < lengths[b]:
            n = min(2000, int(lengths[b]) - done)
            assert s.project([b], [n], syn.taps_rows(cfg, cfg.seed, b, done, n)) == 0
            done += n
    pos, reqs, rep = [int(x) for x in lengths], list(range(B)), {}
    for rnd in range(2):
        anchors = syn.anchors(cfg.seed, B, rnd, cfg.vocab)
        g = s.draft(reqs, anchors, logits=True)
        assert g["rc"] == 0 and s.check() == 0
        cache = s.h.ctx_cache()
        for b in checked:
            got = stored(cfg, cache, b, pos[b])
            check_rows(cfg, got, orc.ctx_rows(syn.taps_to_f32(cfg, newest[b]).astype(np.float64)))
            compare_block(cfg, g, orc.draft(int(anchors[b]), got[0][0], got[1][0]), b, rep)
        counts = [int(c) for c in syn.append_counts(cfg, rnd)]
        rows = [syn.taps_rows(cfg, cfg.seed, b, pos[b], counts[b]) for b in reqs]
        assert s.project(reqs, counts, np.concatenate(rows)) == 0
        for b in reqs:
            pos[b] += counts[b]
            if b in checked:
                newest[b] = np.concatenate([newest[b], rows[b]])
    s.close()
    print(cfg.name, rep)


@pytest.mark.parametrize("skinny", [False, True], ids=["gemv", "tc05"])
def test_one_request(skinny):
    """Block 8, window 2048 over 4096 rows."""
    cfg = syn.with_overrides(CONFIGS["c3"], skinny_tc05=skinny, cache_blocks=34)
    run(cfg, [cfg.ctx_len], [0])


@pytest.mark.parametrize("tc05", [False, True], ids=["gemv", "tc05"])
def test_batched_requests(tc05):
    """32 requests, block 5, ragged contexts (an eighth of the workload's, down to 64 rows: positions before the window only move the ring)."""
    cfg = syn.with_overrides(CONFIGS["c5"], large_batch_tc05=tc05, cache_blocks=32 * 34)
    lengths = [max(64, int(n) // 8) if b not in (0, 17) else int(n) % 3000 + 1200 for b, n in enumerate(syn.ctx_lengths(cfg))]
    run(cfg, lengths, [0, 17])
