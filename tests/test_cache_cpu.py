"""The paged 8-bit context cache without a GPU: struct layouts, argument checks of the C entry points and
of the binding, and the plain restatement that the GPU tests compare with."""
import ctypes
import os
import subprocess

import pytest
import torch

import speculative_block_draft_gb300 as pkg
import cache_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    pkg.build()
    return pkg.lib()


def test_struct_layouts_match_c(tmp_path):
    src = tmp_path / "sz.c"
    src.write_text('#include "dflash.h"\n#include <stdio.h>\n#include <stddef.h>\nint main(){printf("%zu %zu %zu %zu %zu %zu %zu",'
                   'sizeof(dflash_cache_config), sizeof(dflash_rows), sizeof(dflash_pool), sizeof(dflash_attention),'
                   'offsetof(dflash_cache_config, max_q), offsetof(dflash_attention, k_own), offsetof(dflash_attention, scale));return 0;}\n')
    exe = tmp_path / "sz"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    got = list(map(int, subprocess.check_output([str(exe)]).split()))
    want = [ctypes.sizeof(pkg.dflash_cache_config), ctypes.sizeof(pkg.dflash_rows), ctypes.sizeof(pkg.dflash_pool),
            ctypes.sizeof(pkg.dflash_attention), pkg.dflash_cache_config.max_q.offset, pkg.dflash_attention.k_own.offset,
            pkg.dflash_attention.scale.offset]
    assert got == want
    # the binding packs three of them in one go
    from speculative_block_draft_gb300 import cache
    assert cache._ROWS.size == ctypes.sizeof(pkg.dflash_rows) and cache._POOL.size == ctypes.sizeof(pkg.dflash_pool)
    assert cache._ATTENTION.size == pkg.dflash_attention.scale.offset + 4
    a = pkg.dflash_attention()
    cache._ATTENTION.pack_into(a, 0, *range(1, 12), *range(20, 36), 40, 41, 0.5)
    assert (a.layer, a.table_blocks, a.requests, a.row_start, a.dtype, a.causal, a.window, a.scale) == (1, 6, 7, 10, 11, 40, 41, 0.5)
    assert [(r.data, r.layer_stride, r.row_stride, r.head_stride) for r in (a.q, a.out, a.k_own, a.v_own)] == \
        [tuple(range(i, i + 4)) for i in (20, 24, 28, 32)]


def config(**kw):
    c = pkg.dflash_cache_config(4096, 8192, 1 << 20, 1 << 21, 2, 10, 64, 8, 128, 10 * 8 * 64 * 128, 8 * 64 * 128, 64 * 128, 128, 40, 32, 8)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_cache_config_checks(lib):
    nbytes = lambda **kw: lib.dflash_cache_workspace_bytes(ctypes.byref(config(**kw)))   # noqa: E731
    assert nbytes() > 0
    assert lib.dflash_cache_workspace_bytes(None) == 0
    assert nbytes(n_q_heads=0, max_requests=0, max_q=0) > 0                  # appends only
    for field, values in (("k", [None, 4100]), ("v", [None, 8]), ("k_scale", [None]), ("v_scale", [None]), ("n_layers", [0, -1]),
                          ("n_blocks", [0, -5, 1 << 25]), ("block_tokens", [0, 8, 48, 256]), ("n_kv_heads", [0, 3]),
                          ("head_dim", [0, 32, 96, 512]), ("layer_stride", [-16, 8]), ("block_stride", [100]), ("head_stride", [-16]),
                          ("token_stride", [64, 136]), ("n_q_heads", [0, 12, 44]), ("max_requests", [0, -1, 1025]), ("max_q", [0, 129])):
        for v in values:
            assert nbytes(**{field: v}) == 0, (field, v)


def test_cache_entry_points_refuse(lib):
    E = pkg.DFLASH_EINVAL
    h = ctypes.c_void_p()
    cfg = config()
    assert lib.dflash_cache_create(ctypes.byref(cfg), None, 1 << 30, None, ctypes.byref(h)) == E
    assert lib.dflash_cache_create(ctypes.byref(cfg), 128, 1 << 30, None, ctypes.byref(h)) == E          # not 256-byte aligned
    assert lib.dflash_cache_create(ctypes.byref(cfg), 256, 16, None, ctypes.byref(h)) == pkg.DFLASH_ECAPACITY
    assert lib.dflash_cache_create(ctypes.byref(cfg), 256, 1 << 30, None, None) == E
    assert not h
    rows = pkg.dflash_rows(256, 0, 1024, 128)
    assert lib.dflash_cache_append(None, 0, 1, 1, 256, ctypes.byref(rows), ctypes.byref(rows), 1, None) == E
    assert lib.dflash_cache_attention(None, ctypes.byref(pkg.dflash_attention()), None) == E
    assert lib.dflash_cache_check_errors(None, None) == E
    lib.dflash_cache_destroy(None)


def test_pool_entry_points_refuse(lib):
    E = pkg.DFLASH_EINVAL

    def pool(**kw):
        p = pkg.dflash_pool(64, 100, 8, 4, 0, 256, 256, 256, 256, 256)
        for k, v in kw.items():
            setattr(p, k, v)
        return p

    def reserve(p, n=4, requests=None, n_new=256, slots=256, n_slots=8, start=256, granted=256):
        return lib.dflash_pool_reserve(ctypes.byref(p) if p else None, n, requests, n_new, slots, n_slots, start, granted, None)

    assert reserve(None) == E
    for kw in ({"block_tokens": 24}, {"n_blocks": 0}, {"n_blocks": 1 << 25}, {"table_rows": 0}, {"table_blocks": 0}, {"ring": 2},
               {"lens": None}, {"table": None}, {"free_list": None}, {"free_count": None}, {"scratch": None}):
        assert reserve(pool(**kw)) == E, kw
        assert lib.dflash_pool_truncate(ctypes.byref(pool(**kw)), 4, None, 256, None) == E, kw
    for kw in ({"n": -1}, {"n": 1025}, {"n": 9}, {"n_new": None}, {"slots": None}, {"n_slots": -1}, {"start": None}, {"granted": None}):
        assert reserve(pool(), **kw) == E, kw
    assert reserve(pool(), n=0, n_slots=0) == pkg.DFLASH_OK
    for args in ((-1, None, 256), (9, None, 256), (4, None, None), (1025, 256, 256)):
        assert lib.dflash_pool_truncate(ctypes.byref(pool()), *args, None) == E
    assert lib.dflash_pool_truncate(ctypes.byref(pool()), 0, None, None, None) == pkg.DFLASH_OK


def test_binding_refuses(lib):
    with pytest.raises(pkg.DFlashError):
        pkg.BlockPool(24, device="cpu")
    with pytest.raises(pkg.DFlashError):
        pkg.BlockPool(64, max_requests=2000, device="cpu")
    k = torch.zeros((1, 4, 2, 16, 64), dtype=torch.uint8)
    s = torch.zeros((1, 4, 2))
    for bad in ((k.float(), k, s, s), (k, k[:, :3], s, s), (k, k, s[:, :3], s), (k, k, s, s.double()), (k, k.permute(0, 1, 3, 2, 4), s, s)):
        with pytest.raises(ValueError):
            pkg.Cache(*bad)
    with pytest.raises(pkg.DFlashError):      # a head_dim without a kernel
        pkg.Cache(k[..., :48].contiguous(), k[..., :48].contiguous(), s, s)
    with pytest.raises(pkg.DFlashError):      # limits that do not fit the heads
        pkg.Cache(k, k, s, s, max_requests=4, max_q=2, n_q_heads=3)


def test_binding_refuses_host_memory(lib):
    k, s = torch.zeros((1, 4, 2, 16, 64), dtype=torch.uint8), torch.zeros((1, 4, 2))
    with pytest.raises(ValueError):
        pkg.Cache(k, k, s, s)
    with pytest.raises(ValueError):
        pkg.BlockPool(64, device="cpu")


def test_reference_scale_and_codes():
    """The restatement's scale keeps every finite value in range and no smaller power of two does; a
    code is off by at most 2^-4 relative, or half the smallest code."""
    assert ref.fit_scale(0.0) == 2.0 ** -64 and ref.fit_scale(448.0) == 1.0 and ref.fit_scale(448.1) == 2.0 and ref.fit_scale(224.0) == 0.5
    g = torch.Generator().manual_seed(1)
    x = torch.randn((1, 16, 2, 64), generator=g) * torch.exp2(torch.randint(-40, 60, (1, 16, 2, 64), generator=g).float())
    codes, scales = torch.zeros((1, 3, 2, 16, 64), dtype=torch.uint8), torch.zeros((1, 3, 2))
    ref.append(codes, scales, x, list(range(16, 32)), 16)
    got = codes[0, 1].view(ref.E4M3).double() * scales[0, 1].double()[:, None, None]
    want = x[0].double().transpose(0, 1)
    assert torch.all((got - want).abs() <= torch.maximum(want.abs() / 16, scales[0, 1].double()[:, None, None] * 2.0 ** -10))
    assert scales[0, 0].abs().sum() == 0 and scales[0, 2].abs().sum() == 0
    top = want.abs().amax((1, 2))
    assert torch.all(top <= 448 * scales[0, 1].double()) and torch.all(top > 224 * scales[0, 1].double())


def test_reference_reserve_after_truncate_takes_the_same_blocks():
    T, lens = 16, [5, 40, 0, 33]
    free = list(range(20))
    table = [[-1] * 6 for _ in lens]
    count, n = 20, lens[:]
    have = [0] * 4
    count, slots, start, granted = ref.pool_reserve(T, False, have, table, free, count, n)
    assert granted == [1] * 4 and start == [0, 5, 45, 45, 78] and count == 20 - 7
    before = (have[:], [r[:] for r in table], free[:count], count)
    count, slots, *_ = ref.pool_reserve(T, False, have, table, free, count, [20, 1, 16, 0])
    count = ref.pool_truncate(T, False, have, table, free, count, before[0])
    assert (have, table, free[:count], count) == before
    _, again, *_ = ref.pool_reserve(T, False, have, table, free, count, [20, 1, 16, 0])
    assert again == slots


def test_drafter_config_with_a_paged_cache(lib):
    import dflash_synth as syn
    nbytes = lambda cfg, **kw: lib.dflash_workspace_bytes(ctypes.byref(pkg.make_config(syn.with_overrides(cfg, **kw))))   # noqa: E731
    c5 = syn.CONFIGS["c5"]
    ring = nbytes(c5)
    # 32 requests x 33 blocks of a 2048-token window, as the ring holds: half the bytes a row, and the join's workspace
    paged = nbytes(c5, cache_blocks=32 * 33)
    row = 5 * 2 * 8 * 128
    assert ring > 0 and paged > 0
    assert ring - nbytes(c5, cache_blocks=1) > 32 * 2048 * row * 2 - (64 << 20)
    assert nbytes(c5, cache_blocks=2000) - nbytes(c5, cache_blocks=1000) == pytest.approx(1000 * (64 * row + 5 * 2 * 8 * 4 + 4), abs=4096)
    assert nbytes(c5, cache_blocks=-1) == 0 and nbytes(c5, cache_blocks=1 << 25) == 0
    assert nbytes(syn.CONFIGS["c1"], cache_blocks=8) == 0                    # fp32 drafter: the ring only
    assert lib.dflash_ctx_cache(None, None, None) == pkg.DFLASH_EINVAL
