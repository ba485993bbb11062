"""The drafter with its context K/V in the paged 8-bit cache (config cache_blocks): what it stores against the oracle's
K/V, and its drafts against the oracle run on exactly what it stored."""
import numpy as np
import pytest
import torch

import dflash_synth as syn
import oracle
import speculative_block_draft_gb300 as pkg
from dflash_synth import DraftConfig
from parity_util import compare_block

pytestmark = pytest.mark.gpu


def small(name, **kw):
    base = dict(n_layers=2, d=256, n_q_heads=4, n_kv_heads=2, head_dim=64, inter=512, n_taps=2, target_hidden=256,
                vocab=1000, gamma=5, window=0, ctx_len=70, wdtype="q4", adtype="bf16", seed=77, batch=3, cache_blocks=40)
    base.update(kw)
    return DraftConfig(name, **base)


class Paged:
    """A session with the paged cache, the oracle's K/V of every appended row, and the comparison of both."""

    def __init__(self, cfg, **kw):
        from speculative_block_draft_gb300.session import Session
        self.cfg, model = cfg, syn.make_model(cfg, norm_jitter=0.1)
        self.gpu, self.orc = Session(model, **kw), oracle.Oracle(model)
        self.k, self.v, self.pos, self.taken = {}, {}, {}, {}

    def append(self, reqs, counts):
        c = self.cfg
        for r in reqs:
            self.pos.setdefault(r, 0)
        rows = [syn.taps_rows(c, c.seed, self.taken.get(r, r), self.pos[r], n) for r, n in zip(reqs, counts)]
        assert self.gpu.project(reqs, counts, np.concatenate(rows)) == 0
        for r, n, t in zip(reqs, counts, rows):
            k, v = self.orc.ctx_rows(syn.taps_to_f32(c, t).astype(np.float64))
            self.k[r] = np.concatenate([self.k[r], k], 1) if r in self.k else k
            self.v[r] = np.concatenate([self.v[r], v], 1) if r in self.v else v
            self.pos[r] += n

    def reset(self, r, other_taps):
        self.gpu.h.reset_request(r)
        self.pos[r], self.taken[r] = 0, other_taps
        self.k.pop(r, None), self.v.pop(r, None)

    def stored(self, r):
        """What the cache holds of request r's window, as values [L][n][kvd] of K and V, checked against the oracle's.
        A code is off by 2^-4 relative; a subnormal one by half its step, 2^-10 of the scale, twice when the
        block's scale grew; and the f16 path's own rows are off by a share of their size that 2^-5 of the rms covers
        (2^-11 per rounded input, over sums of a few hundred products that are about 20 times their result in
        magnitude). A row in the wrong place would be off by about the rms."""
        c, s = self.cfg, self.gpu.h.ctx_cache()
        P, n = self.pos[r], min(self.pos[r], c.window) if c.window else self.pos[r]
        assert int(s["lens"][r]) == P
        table, out = s["table"][r].tolist(), []
        at = list(range(P - n, P))
        blocks = [table[(p // 64) % len(table)] for p in at]
        assert all(0 <= b < c.cache_blocks for b in blocks)
        for name, want in (("k", self.k), ("v", self.v)):
            codes = s[name].view(torch.float8_e4m3fn)[:, blocks, :, [p % 64 for p in at]]   # [n][L][H][hd]
            scale = s[name + "_scale"][:, blocks].permute(1, 0, 2)
            val = (codes.double() * scale.double()[..., None]).permute(1, 0, 2, 3).reshape(c.n_layers, n, -1).cpu().numpy()
            scale = scale.permute(1, 0, 2).double().cpu().numpy().repeat(c.head_dim, 2)
            ref = want[r][:, P - n:]
            slack = 2.0 ** -5 * np.sqrt(np.mean(ref ** 2))
            assert np.all(np.abs(val - ref) <= 2.0 ** -4 * (np.abs(ref) + slack) + slack + 2.0 ** -9 * scale)
            out.append(np.ascontiguousarray(val))
        return out

    def round(self, reqs, rnd):
        c, report = self.cfg, {}
        anchors = syn.anchors(c.seed, len(reqs), rnd, c.vocab)
        g = self.gpu.draft(reqs, anchors, logits=True)
        assert g["rc"] == 0
        for i, r in enumerate(reqs):
            k, v = self.stored(r) if self.pos.get(r, 0) else (np.zeros((c.n_layers, 0, c.n_kv_heads * c.head_dim)),) * 2
            compare_block(c, g, self.orc.draft(int(anchors[i]), k, v), i, report)
        assert self.gpu.check() == 0
        return report


@pytest.mark.parametrize("wdtype,hd", [("q4", 64), ("q4", 128), ("bf16", 128), ("q4", 256)])
def test_drafts_over_the_whole_context(wdtype, hd):
    cfg = small(f"p_{wdtype}_{hd}", wdtype=wdtype, head_dim=hd, n_q_heads=512 // hd, n_kv_heads=max(1, 256 // hd), d=512,
                target_hidden=512, inter=1024)
    p = Paged(cfg, ctx_capacity=400)
    p.append([0, 1, 2], [70, 1, 130])
    for rnd in range(3):
        p.round([0, 1, 2], rnd)
        p.append([2, 0], [1 + rnd, 5])
    p.round([1], 3)
    p.gpu.close()


def test_drafts_before_any_context():
    p = Paged(small("p_empty"), ctx_capacity=200)
    p.append([1], [64])
    p.round([0, 1, 2], 0)
    p.gpu.close()


def test_window_rings_reuse_blocks():
    """Windows of two blocks and a half: blocks come round several times, also within one call."""
    cfg = small("p_ring", window=150, ctx_len=300, cache_blocks=3 * 4)
    p = Paged(cfg, ctx_capacity=150)
    p.append([0, 1, 2], [300, 10, 151])
    for rnd in range(4):
        p.round([0, 1, 2], rnd)
        p.append([0, 1, 2], [8, 90 + rnd, 3])
    assert int(p.gpu.h.ctx_cache()["free_count"]) == 12 - (4 + 4 + 3)       # the third request has 163 positions
    p.gpu.close()


def test_many_rows_on_the_tcgen05_contraction():
    """Appends of more than 160 rows and more than 32 block rows through the grouped launches."""
    cfg = small("p_tc05", d=512, target_hidden=512, inter=1024, n_q_heads=4, n_kv_heads=2, head_dim=128, batch=9, large_batch_tc05=True,
                window=192, cache_blocks=9 * 4)
    p = Paged(cfg, ctx_capacity=192)
    reqs = list(range(9))
    p.append(reqs, [400, 3, 64, 65, 1, 0, 20, 33, 192])
    for rnd in range(2):
        p.round(reqs, rnd)
        p.append(reqs, [5, 1, 8, 2, 3, 4, 5, 6, 7])
    p.gpu.close()


def test_pool_capacity_and_reset():
    """Too few free blocks are refused before anything runs; a reset request's blocks serve others."""
    cfg = small("p_pool", cache_blocks=5)
    p = Paged(cfg, ctx_capacity=400)
    p.append([0, 1], [130, 100])                     # 3 + 2 blocks
    with pytest.raises(pkg.DFlashError) as e:
        p.gpu.project([2], [1], syn.taps_rows(cfg, 1, 2, 0, 1))
    assert e.value.status == pkg.DFLASH_ECAPACITY
    with pytest.raises(pkg.DFlashError):
        p.gpu.project([1], [29], syn.taps_rows(cfg, 1, 1, 100, 29))
    p.append([1], [28])                              # fills its second block
    p.round([0, 1], 0)
    p.reset(0, 7)
    p.round([0, 1], 1)                               # without context now
    p.append([2], [190])
    p.round([1, 2], 2)
    p.reset(1, 8)
    p.append([0, 1], [60, 64])
    p.round([0, 1, 2], 3)
    p.gpu.close()


def test_refuses_without_a_paged_cache():
    cfg = small("p_none", cache_blocks=0)
    p = Paged(cfg, ctx_capacity=100)
    with pytest.raises(pkg.DFlashError):
        p.gpu.h.ctx_cache()
    p.gpu.close()
