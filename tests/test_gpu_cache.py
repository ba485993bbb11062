"""The paged 8-bit context cache on the GPU against the plain 64-bit restatement in cache_ref."""
import random

import pytest
import torch

import cache_ref as ref
import speculative_block_draft_gb300 as pkg

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---- block tables and slots ----------------------------------------------------------------------------------------------
class Pool:
    """The GPU pool and the restatement, fed the same calls and compared after each."""

    def __init__(self, T, rows, width, blocks, ring=False, seed=0):
        perm = list(range(blocks))
        random.Random(seed).shuffle(perm)
        self.T, self.ring = T, ring
        self.lens, self.table, self.free, self.count = [0] * rows, [[-1] * width for _ in range(rows)], perm, blocks
        self.d = {"lens": ints(self.lens), "table": ints(self.table), "free": ints(perm), "free_count": ints([blocks])}
        self.pool = pkg.BlockPool(T, ring=ring)

    def same(self):
        assert self.d["lens"].tolist() == self.lens
        assert self.d["table"].tolist() == self.table
        assert self.d["free_count"].tolist() == [self.count]
        assert self.d["free"].tolist()[:self.count] == self.free[:self.count]

    def reserve(self, n_new, requests=None, extra=5):
        before = self.count
        n_slots = sum(max(0, n) for n in n_new if n <= 1 << 20) + extra
        self.count, slots, start, granted = ref.pool_reserve(self.T, self.ring, self.lens, self.table, self.free, self.count, n_new,
                                                             requests, n_slots)
        out = {"slots": torch.full((n_slots,), 77, dtype=torch.int32, device="cuda"), "row_start": ints([0] * (len(n_new) + 1)),
               "granted": ints([0] * len(n_new))}
        self.pool.reserve(ints(n_new), requests=None if requests is None else ints(requests), **self.d, **out)
        assert out["granted"].tolist() == granted
        assert out["row_start"].tolist() == start
        assert out["slots"].tolist() == slots
        self.same()
        assert self.count <= before
        return out

    def truncate(self, new_len, requests=None):
        self.count = ref.pool_truncate(self.T, self.ring, self.lens, self.table, self.free, self.count, new_len, requests)
        self.pool.truncate(ints(new_len), requests=None if requests is None else ints(requests), **self.d)
        self.same()


@pytest.mark.parametrize("T", [16, 32, 64, 128])
def test_reserve_and_truncate_rounds(T):
    p, rng = Pool(T, 9, 7, 50, seed=T), random.Random(T)
    for _ in range(12):
        p.reserve([rng.choice([0, 1, 2, T - 1, T, T + 1, 3 * T]) for _ in range(9)])
        p.truncate([max(0, n - rng.choice([0, 1, 5, T, 4 * T])) for n in p.lens])
    p.truncate([0] * 9)
    assert p.count == 50


def test_reserve_runs_out_of_blocks_and_of_table():
    p = Pool(16, 5, 4, 6)
    p.reserve([30, 64, 64, 10, 65])       # 2 + 4 blocks fit, the third and the fourth do not, the fifth passes its table
    p.reserve([2, 0, 0, 0, 0])            # needs no block
    p.reserve([1, 0, 0, 0, 0])            # needs one, none is free
    p.truncate([0, 100, 0, 0, 0])
    p.reserve([0, 0, 16, 16, 16])


def test_reserve_names_requests():
    p = Pool(32, 6, 5, 30)
    p.reserve([40, 7, 9, 3, 5], requests=[4, 1, 4, 6, -1])        # twice, out of range, negative
    p.reserve([3, -1, 1 << 21, 0], requests=[1, 0, 2, 4])
    p.truncate([0, 5, 2], requests=[4, 4, 1])
    p.truncate([-1, 9], requests=[1, 7])


def test_reserve_no_rows_and_no_requests():
    p = Pool(64, 3, 2, 5)
    p.reserve([0, 0, 0], extra=3)
    p.reserve([], extra=4)


def test_reserve_many_rows():
    """Several CTAs write the slots; 1024 requests."""
    p, rng = Pool(16, 1024, 40, 30000), random.Random(5)
    p.reserve([rng.randint(0, 90) for _ in range(1024)])
    p.reserve([rng.randint(0, 400) for _ in range(1024)])
    p.truncate([rng.randint(0, n) for n in p.lens])
    p.reserve([rng.randint(0, 30) for _ in range(1000)], requests=rng.sample(range(1024), 1000))


def test_most_requests():
    """As many requests as a call may have; released blocks of all of them by several CTAs."""
    rng = random.Random(5)
    p = Pool(16, 1024, 40, 30000, seed=6)
    p.reserve([rng.choice((0, 1, 16, 17, 300, 640)) for _ in range(1024)])
    p.truncate([rng.randint(0, 640) for _ in range(1024)])
    p.reserve([rng.randint(0, 30) for _ in range(1024)])
    p.truncate([0] * 1024)
    assert p.count == 30000


def test_ring_reuses_blocks():
    p, rng = Pool(16, 4, 5, 17, ring=True), random.Random(3)
    for n in (1, 70, 15, 64, 33, 300, 16):
        p.reserve([n, rng.randint(0, 20), n // 2, 3])
    p.truncate([0, p.lens[1], 0, 0])
    p.reserve([90, 1, 80, 200])


# ---- append ----------------------------------------------------------------------------------------------------------------
def check_append(codes, scales, rows, slots, T, layer0=0, views=None, k_rows=None, v_rows=None):
    """codes, scales: (K, V) on the CPU; rows (K, V) on the CPU."""
    dev = [c.cuda() for c in codes] if views is None else views
    sc = [s.cuda() for s in scales]
    cache = pkg.Cache(dev[0], dev[1], sc[0], sc[1])
    cache.append(ints(slots), rows[0].cuda() if k_rows is None else k_rows, rows[1].cuda() if v_rows is None else v_rows, layer=layer0)
    for i in range(2):
        ref.append(codes[i], scales[i], rows[i], slots, T, layer0)
        assert torch.equal(sc[i].cpu(), scales[i])
        a, b = dev[i].cpu(), codes[i]
        nan = (b & 0x7F) == 0x7F                       # a NaN has two codes
        assert torch.equal((a & 0x7F) == 0x7F, nan)
        assert torch.equal(a[~nan], b[~nan])
    assert cache.check_errors() == 0


def slots_of(table, spans, T):
    return [table[r][p // T] * T + p % T for r, (a, b) in enumerate(spans) for p in range(a, b)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("hd,T,heads,layers", [(128, 64, 8, 5), (64, 16, 3, 2), (256, 128, 2, 1), (128, 32, 1, 1)])
def test_append_matches(dtype, hd, T, heads, layers):
    spans = [(0, 1), (5, 6), (T - 1, T + 1), (3, 3), (0, 2 * T + 7), (T, 2 * T), (2, 2 * T + 1)]
    N = 24
    table = ref.random_table([b for _, b in spans], T, N, 3, 1)
    slots = slots_of(table, spans, T)
    k, v, ks, vs = ref.random_cache(layers, N, heads, T, hd, 2)
    g = torch.Generator().manual_seed(3)
    rows = [(torch.randn((layers, len(slots), heads, hd), generator=g)
             * torch.exp2(torch.randint(-3, 4, (layers, len(slots), heads, 1), generator=g).float())).to(DT[dtype]) for _ in range(2)]
    check_append((k, v), (ks, vs), rows, slots, T)


def test_append_edges():
    """Zeros, infinities, NaN, the largest and smallest magnitudes, negative and repeated slots, a block named
    behind skipped rows, scales that are no power of two, one layer of several."""
    T, N, H, D = 16, 8, 2, 64
    k, v, ks, vs = ref.random_cache(3, N, H, T, D, 5)
    ks[1, 2], vs[1, 2] = 0.3, 3.7
    slots = [-1, 2 * T + 3, 2 * T + 4, -1, 2 * T + 4, 2 * T + 5, -7, 4 * T, 4 * T + 1, 4 * T + 1, 5 * T + 15, 6 * T, -1]
    g = torch.Generator().manual_seed(6)
    rows = [torch.randn((len(slots), H, D), generator=g) for _ in range(2)]
    rows[0][7:10] = 0
    rows[1][8, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 1e30])
    rows[0][10], rows[1][10] = float("nan"), float("inf")
    rows[0][11, :, :3], rows[1][11] = torch.tensor([3.4028234e38, -1e-40, 2.0 ** -74]), 1e-44
    both = [r[None] for r in rows]
    check_append((k, v), (ks, vs), both, slots, T, layer0=1, k_rows=rows[0].cuda(), v_rows=rows[1].cuda())


def test_append_strides():
    """Token-major codes and rows that are slices of a wider projection."""
    T, N, H, D = 32, 6, 4, 128
    k, v, ks, vs = ref.random_cache(2, N, H, T, D, 7)
    views = [c.permute(0, 1, 3, 2, 4).contiguous().cuda().permute(0, 1, 3, 2, 4) for c in (k, v)]
    slots = list(range(T, 3 * T)) + [5 * T + 9]
    wide = torch.randn((2, len(slots), 3 * H * D + 64), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    part = [wide[:, :, o:o + H * D].unflatten(2, (H, D)) for o in (H * D, 2 * H * D + 64)]
    dev = wide.cuda()
    on_gpu = [dev[:, :, o:o + H * D].unflatten(2, (H, D)) for o in (H * D, 2 * H * D + 64)]
    check_append((k, v), (ks, vs), part, slots, T, views=views, k_rows=on_gpu[0], v_rows=on_gpu[1])


def test_append_many_rows():
    """A prompt: several rows per CTA, blocks that begin inside a CTA's rows."""
    T, D = 64, 128
    n = 1500
    N = 30
    k, v, ks, vs = ref.random_cache(1, N, 2, T, D, 9)
    perm = torch.randperm(N, generator=torch.Generator().manual_seed(1)).tolist()
    slots = [perm[p // T] * T + p % T for p in range(13, 13 + n)] + [-1] * 40
    g = torch.Generator().manual_seed(10)
    rows = [torch.randn((1, len(slots), 2, D), generator=g).to(torch.bfloat16) for _ in range(2)]
    check_append((k, v), (ks, vs), rows, slots, T)


def test_append_skips_every_row():
    T, N, H, D = 32, 5, 2, 128
    dev = [x.cuda() for x in ref.random_cache(1, N, H, T, D, 1)]
    before = [x.clone() for x in dev]
    rows = torch.randn((700, H, D), device="cuda")
    pkg.Cache(*dev).append(ints([-1] * 700), rows, rows)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, dev))


def test_append_refuses():
    T, N, H, D = 16, 4, 2, 64
    k, v, ks, vs = (x.cuda() for x in ref.random_cache(1, N, H, T, D, 1))
    cache, rows = pkg.Cache(k, v, ks, vs), torch.randn((3, H, D), device="cuda")
    for call in (lambda: cache.append(ints([0, 1, 2]), rows, rows, layer=1), lambda: cache.append(ints([0, 1, 2]), rows, rows, layer=-1),
                 lambda: cache.append(ints([0, 1, 2]), torch.zeros((3, H, D + 2), device="cuda")[..., :D], rows)):
        with pytest.raises(pkg.DFlashError):
            call()
    for call in (lambda: cache.append(ints([0, 1]), rows, rows), lambda: cache.append(ints([0, 1, 2]), rows.double(), rows.double()),
                 lambda: cache.append(ints([0, 1, 2]), rows, rows.half()), lambda: cache.append(ints([0, 1, 2]).long(), rows, rows),
                 lambda: cache.append(ints([0, 1, 2]), rows, rows[..., :32])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(pkg.DFlashError):          # created without attention limits
        cache.attention(rows.half(), ints([0]), ints([[0]]), rows.half(), max_q=3)
    before = k.clone()
    assert cache.append(ints([]), rows[:0], rows[:0]) == 0
    assert torch.equal(before, k)


# ---- attention ---------------------------------------------------------------------------------------------------------------
def run_attention(lens, counts, Hq, H, D, T, dtype, own=False, causal=False, window=0, ragged=None, requests=None, seed=0, width=None,
                  qstd=2.0, change=None, **kw):
    """One call against the restatement. change(k, v, ks, vs, table) edits the inputs before both see them."""
    dt = DT[dtype]
    width = width or max(1, max(-(-n // T) for n in lens))
    N = sum(-(-n // T) for n in lens) + 3
    k, v, ks, vs = ref.random_cache(1, N, H, T, D, seed)
    table = ref.random_table(lens, T, N, width, seed + 1)
    if change:
        change(k, v, ks, vs, table)
    g = torch.Generator().manual_seed(seed + 2)
    rows = sum(counts)
    q = (qstd * torch.randn((rows, Hq, D), generator=g)).to(dt)
    ko, vo = ((torch.randn((rows, H, D), generator=g).to(dt) for _ in range(2)) if own else (None, None))
    spare = 3
    out = torch.full((rows + spare, Hq, D), 7.0, dtype=dt, device="cuda")
    qd = torch.cat([q, q.new_full((spare, Hq, D), 3)]).cuda()
    pad = lambda t: None if t is None else torch.cat([t, t.new_zeros((spare, H, D))]).cuda()   # noqa: E731
    cache = pkg.Cache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), max_requests=len(counts), max_q=max(max(counts), 1), n_q_heads=Hq)
    ragged = len(set(counts)) > 1 if ragged is None else ragged
    start = ints([sum(counts[:i]) for i in range(len(counts) + 1)]) if ragged else None
    if not ragged and requests is None and len(lens) != len(counts):
        raise AssertionError("lens and counts")
    cache.attention(qd, ints(lens), ints(table), out, row_start=start, max_q=max(max(counts), 1), k_own=pad(ko), v_own=pad(vo),
                    window=window, causal=causal, requests=None if requests is None else ints(requests), **kw)
    assert cache.check_errors() == 0
    want, tol = ref.attention(q, k[0], v[0], ks[0], vs[0], lens, table, counts, dt, ko, vo, window, causal, requests=requests, **kw)
    got = out.cpu()
    assert torch.all(got[rows:] == 7.0), "rows behind the last request changed"
    err = (got[:rows].double() - want).abs()
    assert torch.all(err <= tol), f"off by {float((err / tol).max()):.2f} of the tolerance ({float(err.max()):.3g})"
    return got[:rows], want


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,H,D,T", [(8, 8, 128, 64), (10, 2, 128, 64), (4, 4, 64, 16), (5, 1, 256, 32), (16, 2, 128, 128), (3, 3, 64, 128)])
def test_attention_single_tokens(dtype, Hq, H, D, T):
    run_attention([1, 2, T - 1, T, T + 1, 127, 128, 129, 300, 0], [1] * 10, Hq, H, D, T, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("window", [0, 1, 100])
def test_attention_masks(dtype, causal, own, window):
    run_attention([0, 1, 3, 5, 64, 90, 257], [5] * 7, 10, 2, 128, 32, dtype, own=own, causal=causal, window=window, seed=window)


@pytest.mark.parametrize("D,T,Hq,H", [(64, 32, 6, 2), (128, 16, 16, 2), (256, 64, 10, 2)])
@pytest.mark.parametrize("own,causal", [(True, False), (False, True), (True, True)])
def test_attention_ragged_rows(D, T, Hq, H, own, causal):
    run_attention([200, 7, 0, 131, 40, 513], [3, 0, 2, 9, 1, 16], Hq, H, D, T, "bf16", own=own, causal=causal)


@pytest.mark.parametrize("rows,Hq,H", [(16, 40, 8), (17, 16, 1), (128, 8, 8), (64, 12, 4), (13, 5, 5)])
def test_attention_many_rows(rows, Hq, H):
    """More query rows per KV head than one CTA holds."""
    run_attention([300, 140], [rows] * 2, Hq, H, 128, 64, "bf16", causal=True, seed=rows)
    run_attention([300, 140], [rows] * 2, Hq, H, 64, 32, "f16", own=True, seed=rows)


@pytest.mark.parametrize("rows,Hq,H", [(5, 5, 1), (8, 8, 2), (11, 6, 2), (9, 5, 1), (12, 8, 2), (10, 10, 2)])
@pytest.mark.parametrize("D,T,dtype", [(64, 16, "f16"), (64, 32, "bf16"), (128, 64, "f16"), (128, 128, "bf16"), (256, 32, "f16"), (256, 64, "bf16")])
def test_attention_row_counts(rows, Hq, H, D, T, dtype):
    """Every padding of the rows of a KV head: 25, 32, 33, 45, 48 and 50 of them."""
    run_attention([390, 64, 1], [rows] * 3, Hq, H, D, T, dtype, causal=True, seed=rows)
    run_attention([140, 0, 259], [rows] * 3, Hq, H, D, T, dtype, own=True, window=100, seed=rows)


def test_attention_most_requests():
    """As many requests as a call may have, more pieces of work than CTAs; some without rows, some without keys."""
    rng = random.Random(3)
    lens = [rng.choice((0, 1, 15, 16, 40, 130, 260)) for _ in range(1024)]
    run_attention(lens, [rng.randint(0, 2) for _ in lens], 2, 1, 64, 16, "bf16", causal=True, seed=11)
    run_attention(lens, [1] * 1024, 2, 2, 64, 16, "f16", own=True, window=20, seed=12)
    run_attention([0] * 1024, [1] * 1024, 1, 1, 64, 16, "bf16", seed=13)


def test_attention_names_a_request_twice():
    run_attention([300, 20, 77], [3, 1, 4, 3], 6, 2, 128, 32, "bf16", own=True, requests=[2, 0, 2, 0], seed=14)


def test_attention_writes_over_its_queries():
    """out may be q: a row is written when nobody reads it any more."""
    T, H, Hq, D, lens = 64, 2, 10, 128, [3000, 70, 900]
    k, v, ks, vs = ref.random_cache(1, 66, H, T, D, 1)
    table = ref.random_table(lens, T, 66, 47, 2)
    q = torch.randn((12, Hq, D), generator=torch.Generator().manual_seed(3)).bfloat16()
    cache = pkg.Cache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), max_requests=3, max_q=4, n_q_heads=Hq)
    out, apart = q.cuda(), torch.zeros_like(q, device="cuda")
    cache.attention(q.cuda(), ints(lens), ints(table), apart, causal=True)
    cache.attention(out, ints(lens), ints(table), out, causal=True)
    assert torch.equal(out, apart)


def test_attention_long_contexts():
    """The key axis split over many CTAs, next to requests of a few keys."""
    run_attention([9000, 5, 3001], [1, 1, 1], 5, 1, 128, 64, "bf16", seed=4)
    run_attention([4097, 12], [8, 8], 10, 2, 128, 64, "f16", own=True, window=2048, seed=5)
    run_attention([2500], [4], 4, 2, 256, 128, "bf16", causal=True, seed=6)


def test_attention_ring_table_and_request_rows():
    """A windowed request whose table is a ring, and calls that name other rows of lens and table."""
    T, width, window = 32, 4, 90
    lens = [0, 400, 33, 128, 250]
    n_all = 20

    def ring(k, v, ks, vs, table):
        for r, n in enumerate(lens):
            for j in range(min(width, -(-n // T))):
                table[r][j] = (r * width + j) % n_all

    run_attention(lens, [3] * 5, 4, 2, 128, T, "bf16", own=True, window=window, width=width, change=ring, seed=7)
    run_attention(lens, [2, 5, 1], 4, 2, 128, T, "bf16", causal=True, window=window, width=width, change=ring, requests=[4, 1, 3], seed=8)
    run_attention(lens, [3] * 5, 4, 2, 128, T, "bf16", causal=True, width=width, change=ring, seed=9)     # no window: what the ring still holds


def test_attention_garbage_in_masked_places():
    """Tokens behind a request's end, before its window, blocks of nobody: NaN codes there change nothing."""
    lens, T, window = [70, 129, 5], 64, 40

    def spoil(k, v, ks, vs, table):
        used = torch.zeros(k.shape[1:4:2], dtype=torch.bool)                     # [N][T]
        for r, n in enumerate(lens):
            for p in range(max(0, n - window), n):
                used[table[r][p // T], p % T] = True
        for c in (k, v):
            c[0].permute(0, 2, 1, 3)[~used] = 0x7F
        free = ~used.any(1)
        ks[0, free], vs[0, free] = float("nan"), float("inf")

    run_attention(lens, [4] * 3, 8, 2, 128, T, "bf16", window=window, change=spoil)
    run_attention(lens, [4] * 3, 8, 2, 128, T, "f16", own=True, window=window, change=spoil)


def test_attention_nan_behind_a_causal_row():
    """A NaN key or value reaches the rows that see it and no other."""
    T, lens, n = 16, [40], 6

    def spoil(k, v, ks, vs, table):
        p = 40 - n + 3
        v[0, table[0][p // T], :, p % T, 5] = 0x7F

    dt = torch.bfloat16
    k, v, ks, vs = ref.random_cache(1, 6, 2, T, 128, 0)
    table = ref.random_table(lens, T, 6, 3, 1)
    spoil(k, v, ks, vs, table)
    q = torch.randn((n, 4, 128), generator=torch.Generator().manual_seed(2)).to(dt)
    out = torch.zeros((n, 4, 128), dtype=dt, device="cuda")
    cache = pkg.Cache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), max_requests=1, max_q=n, n_q_heads=4)
    cache.attention(q.cuda(), ints(lens), ints(table), out, causal=True)
    nan = out.isnan().cpu()
    assert not nan[:3].any() and nan[3:, :, 5].all()
    cache.attention(q.cuda(), ints(lens), ints(table), out, causal=False)
    assert out.isnan().cpu()[:, :, 5].all()


def test_attention_table_entries_out_of_range():
    """Keys of a block number that the cache does not have are not seen."""
    def wrong(k, v, ks, vs, table):
        table[0][1], table[1][0] = 1000000, -5

    run_attention([200, 100, 60], [2] * 3, 4, 2, 128, 64, "bf16", change=wrong)


def test_attention_peaked_and_flat_scores():
    """One key far above the rest, early and late, and scales that differ by 2^20 between blocks."""
    def peaks(k, v, ks, vs, table):
        ks[0, table[0][0]], ks[0, table[1][6]] = 2.0, 4.0
        vs[0, table[0][3]], vs[0, table[1][2]], vs[0, table[2][0]] = 2.0 ** 8, 2.0 ** -20, 2.0 ** -60

    run_attention([450, 450, 450], [3] * 3, 8, 2, 128, 64, "bf16", change=peaks, qstd=4.0)
    run_attention([450, 450, 450], [3] * 3, 8, 2, 128, 64, "f16", change=peaks, qstd=0.01)


def test_attention_rows_of_very_different_size():
    """Each row's scores are as exact as its own magnitude allows."""
    T = 64
    k, v, ks, vs = ref.random_cache(1, 8, 2, T, 128, 3)
    table = ref.random_table([300], T, 8, 5, 4)
    size = torch.tensor([1e-3, 100.0, 1.0, 0.0, 1e-7]).view(5, 1, 1)
    q = (torch.randn((5, 4, 128), generator=torch.Generator().manual_seed(5)) * size).to(torch.bfloat16)
    out = torch.zeros((5, 4, 128), dtype=torch.bfloat16, device="cuda")
    cache = pkg.Cache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), max_requests=1, max_q=5, n_q_heads=4)
    cache.attention(q.cuda(), ints([300]), ints(table), out, scale=1.0)
    want, tol = ref.attention(q, k[0], v[0], ks[0], vs[0], [300], table, [5], torch.bfloat16, scale=1.0)
    assert torch.all((out.cpu().double() - want).abs() <= tol)


def test_attention_strides_and_layers():
    """Token-major codes, query and output rows that are slices, the second of three layers."""
    T, N, H, D, Hq = 32, 9, 2, 128, 6
    k, v, ks, vs = ref.random_cache(3, N, H, T, D, 11)
    views = [c.permute(0, 1, 3, 2, 4).contiguous().cuda().permute(0, 1, 3, 2, 4) for c in (k, v)]
    lens, counts = [100, 40], [4, 4]
    table = ref.random_table(lens, T, N, 4, 12)
    wide = torch.randn((8, Hq * D + 2 * H * D), generator=torch.Generator().manual_seed(13)).to(torch.float16)
    dev = wide.cuda()
    q, ko, vo = dev[:, :Hq * D].unflatten(1, (Hq, D)), dev[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D)), dev[:, (Hq + H) * D:].unflatten(1, (H, D))
    out = torch.zeros((8, 2, Hq, D), dtype=torch.float16, device="cuda")
    cache = pkg.Cache(views[0], views[1], ks.cuda(), vs.cuda(), max_requests=2, max_q=4, n_q_heads=Hq)
    cache.attention(q, ints(lens), ints(table), out[:, 1], layer=1, k_own=ko, v_own=vo)
    want, tol = ref.attention(q.cpu(), k[1], v[1], ks[1], vs[1], lens, table, counts, torch.float16, ko.cpu(), vo.cpu())
    assert torch.all((out[:, 1].cpu().double() - want).abs() <= tol) and not out[:, 0].any()


def test_attention_beyond_32_bit_offsets():
    """Blocks whose codes lie more than 4 GB into the cache."""
    T, H, D = 64, 8, 128
    N = (5 << 30) // (H * T * D)
    k = torch.zeros((1, N, H, T, D), dtype=torch.uint8, device="cuda")
    v, ks, vs = torch.zeros_like(k), torch.ones((1, N, H), device="cuda"), torch.ones((1, N, H), device="cuda")
    lens, table = [150], [[N - 1, N // 2, N - 3]]
    g = torch.Generator().manual_seed(1)
    rows = [torch.randn((150, H, D), generator=g) for _ in range(2)]
    slots = [table[0][p // T] * T + p % T for p in range(150)]
    cache = pkg.Cache(k, v, ks, vs, max_requests=1, max_q=2, n_q_heads=H)
    cache.append(ints(slots), rows[0].cuda(), rows[1].cuda())
    q = torch.randn((2, H, D), generator=g).half()
    out = torch.zeros((2, H, D), dtype=torch.float16, device="cuda")
    cache.attention(q.cuda(), ints(lens), ints(table), out)
    at = table[0]
    small = [[0, 1, 2]]
    want, tol = ref.attention(q, k[0, at].cpu(), v[0, at].cpu(), ks[0, at].cpu(), vs[0, at].cpu(), lens, small, [2], torch.float16)
    assert torch.all((out.cpu().double() - want).abs() <= tol)
    assert int((k[0, :N // 2] != 0).sum()) == 0 and want.abs().max() > 0.1


def test_attention_refuses():
    T, N, H, D, Hq = 16, 4, 2, 64, 4
    k, v, ks, vs = (x.cuda() for x in ref.random_cache(1, N, H, T, D, 1))
    cache = pkg.Cache(k, v, ks, vs, max_requests=2, max_q=3, n_q_heads=Hq)
    q = torch.zeros((6, Hq, D), dtype=torch.bfloat16, device="cuda")
    out, lens, table = torch.ones_like(q), ints([5, 6]), ints([[0], [1]])
    own = torch.zeros((6, H, D), dtype=torch.bfloat16, device="cuda")
    for kw in ({"layer": 1}, {"window": -1}, {"max_q": 4}, {"k_own": own}, {"v_own": own}, {"scale": float("nan")}, {"scale": float("inf")}):
        with pytest.raises(pkg.DFlashError):
            cache.attention(q, lens, table, out, **kw)
    with pytest.raises(pkg.DFlashError):
        cache.attention(q[:5], lens, table, out[:5], max_q=3)              # fewer rows than requests * max_q
    with pytest.raises(pkg.DFlashError):
        cache.attention(q, ints([1, 2, 3]), ints([[0], [1], [2]]), out, max_q=2)   # more requests than the limit
    for call in (lambda: cache.attention(q.float(), lens, table, out.float()), lambda: cache.attention(q, lens, table, out.half()),
                 lambda: cache.attention(q[..., :32], lens, table, out), lambda: cache.attention(q, lens[:1], table, out),
                 lambda: cache.attention(q, lens.long(), table, out), lambda: cache.attention(q, lens, table, out, row_start=ints([0, 3]), requests=lens)):
        with pytest.raises((ValueError, pkg.DFlashError)):
            call()
    assert torch.all(out == 1)


# ---- together ------------------------------------------------------------------------------------------------------------------
def test_rounds_of_reserve_append_attend_truncate():
    """Speculative rounds as a program runs them: reserve a block's rows, append their K/V, attend causally
    over everything, give the rejected rows back. Captured as one graph and replayed with new inputs."""
    T, L, H, Hq, D, B, n = 32, 2, 2, 6, 128, 5, 4
    N, width = 60, 12
    g = torch.Generator().manual_seed(20)
    zeros = lambda: torch.zeros((L, N, H, T, D), dtype=torch.uint8)      # noqa: E731
    host = {"k": zeros(), "v": zeros(), "ks": torch.ones((L, N, H)), "vs": torch.ones((L, N, H))}
    dev = {x: t.cuda() for x, t in host.items()}
    cache = pkg.Cache(dev["k"], dev["v"], dev["ks"], dev["vs"], max_requests=B, max_q=n, n_q_heads=Hq)
    p = Pool(T, B, width, N, seed=2)
    # prompts
    prompt = [1, 31, 100, 64, 7]
    out = p.reserve(prompt, extra=0)
    rows = [torch.randn((L, sum(prompt), H, D), generator=g).bfloat16() for _ in range(2)]
    cache.append(out["slots"], rows[0].cuda(), rows[1].cuda())
    for x, r in (("k", rows[0]), ("v", rows[1])):
        ref.append(host[x], host[x + "s"], r, out["slots"].tolist(), T)
    # one round, captured
    io = {"n_new": ints([n] * B), "keep": ints([0] * B), "slots": ints([0] * (B * n)), "start": ints([0] * (B + 1)), "granted": ints([0] * B),
          "kr": torch.zeros((L, B * n, H, D), dtype=torch.bfloat16, device="cuda"), "vr": torch.zeros((L, B * n, H, D), dtype=torch.bfloat16, device="cuda"),
          "q": torch.zeros((L, B * n, Hq, D), dtype=torch.bfloat16, device="cuda"), "out": torch.zeros((L, B * n, Hq, D), dtype=torch.bfloat16, device="cuda")}

    def one_round():
        p.pool.truncate(io["keep"], **p.d)
        p.pool.reserve(io["n_new"], **p.d, slots=io["slots"], row_start=io["start"], granted=io["granted"])
        cache.append(io["slots"], io["kr"], io["vr"])
        for layer in range(L):
            cache.attention(io["q"][layer], p.d["lens"], p.d["table"], io["out"][layer], layer=layer, row_start=io["start"], causal=True)

    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    io["keep"].copy_(p.d["lens"])
    saved = {x: t.clone() for x, t in p.d.items()}
    codes = {x: t.clone() for x, t in dev.items()}
    with torch.cuda.stream(stream):
        one_round()                                    # first use outside of the capture
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            one_round()
    for x, t in saved.items():
        p.d[x].copy_(t)
    for x, t in codes.items():
        dev[x].copy_(t)
    rng = random.Random(1)
    for _ in range(4):
        keep = [m - rng.randint(0, min(3, m)) for m in p.lens]
        p.count = ref.pool_truncate(T, False, p.lens, p.table, p.free, p.count, keep)
        p.count, slots, start, granted = ref.pool_reserve(T, False, p.lens, p.table, p.free, p.count, [n] * B)
        assert granted == [1] * B
        new = {x: torch.randn((L, B * n, h, D), generator=g).bfloat16() for x, h in (("kr", H), ("vr", H), ("q", Hq))}
        io["keep"].copy_(ints(keep))
        for x, t in new.items():
            io[x].copy_(t)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        p.same()
        assert io["slots"].tolist() == slots
        for x, r in (("k", new["kr"]), ("v", new["vr"])):
            ref.append(host[x], host[x + "s"], r, slots, T)
            assert torch.equal(dev[x].cpu(), host[x]) and torch.equal(dev[x + "s"].cpu(), host[x + "s"])
        for layer in range(L):
            want, tol = ref.attention(new["q"][layer], host["k"][layer], host["v"][layer], host["ks"][layer], host["vs"][layer], p.lens, p.table,
                                      [n] * B, torch.bfloat16, causal=True)
            assert torch.all((io["out"][layer].cpu().double() - want).abs() <= tol)
    assert cache.check_errors() == 0


def test_two_caches_on_two_streams():
    """Objects of their own on streams of their own at the same time."""
    T, H, D, Hq = 64, 4, 128, 8
    lens, counts = [700, 300], [3, 3]
    jobs = []
    for seed in (1, 2):
        k, v, ks, vs = ref.random_cache(1, 18, H, T, D, seed)
        table = ref.random_table(lens, T, 18, 11, seed)
        q = torch.randn((6, Hq, D), generator=torch.Generator().manual_seed(seed)).half()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            cache = pkg.Cache(k.cuda(), v.cuda(), ks.cuda(), vs.cuda(), max_requests=2, max_q=3, n_q_heads=Hq)
            jobs.append((cache, s, q.cuda(), ints(lens), ints(table), torch.zeros_like(q, device="cuda"),
                         ref.attention(q, k[0], v[0], ks[0], vs[0], lens, table, counts, torch.float16)))
    torch.cuda.synchronize()
    for _ in range(20):
        for cache, s, q, ln, table, out, _ in jobs:
            cache.attention(q, ln, table, out, stream=s)
    torch.cuda.synchronize()
    for *_, out, (want, tol) in jobs:
        assert torch.all((out.cpu().double() - want).abs() <= tol)
