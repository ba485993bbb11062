"""Out-of-range numbers on the device in the paged cache's calls: the debug build (DFL_DEBUG_CHECKS) reports them, every build skips
what they name. As in test_gpu_debug_checks, the debug library runs in a child process."""
import os
import subprocess
import sys

import pytest
import torch

import cache_ref as ref
import speculative_block_draft_gb300 as pkg

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DEBUG = os.environ.get("DFLASH_DEBUG_CHECKS") == "1"


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def reported(cache):
    """Whether the calls before left a report; the release build leaves none. Clears it."""
    if not DEBUG:
        assert cache.check_errors() == 0
        return
    with pytest.raises(pkg.DFlashError) as e:
        cache.check_errors()
    assert e.value.status == pkg.DFLASH_EBOUNDS
    assert cache.check_errors() == 0


def test_numbers_out_of_range():
    T, H, Hq, D, N, dt = 16, 2, 4, 64, 8, torch.bfloat16
    k, v, ks, vs = (x.cuda() for x in ref.random_cache(1, N, H, T, D, 1))
    cache = pkg.Cache(k, v, ks, vs, max_requests=3, max_q=4, n_q_heads=Hq)
    q = torch.randn((9, Hq, D), generator=torch.Generator().manual_seed(2)).to(dt).cuda()
    lens, table = ints([20, 30, 40]), ints([[0, 1, -1], [2, 3, -1], [4, 5, 6]])

    def attend(start, table=table, requests=None, n=9):
        out = torch.full_like(q, 7.0)
        cache.attention(q[:n], lens, table, out[:n], row_start=ints(start), max_q=3, requests=requests)
        return out

    good = attend([0, 3, 6, 9])
    assert cache.check_errors() == 0 and not (good == 7).any()
    # more rows than max_q: the first max_q as ever, the others left as they were
    out = attend([0, 3, 8, 9])
    reported(cache)
    assert torch.equal(out[:6], good[:6]) and (out[6:8] == 7).all()
    # rows behind the tensor's, a request of no table row: all of its rows left as they were
    out = attend([0, 3, 6, 9], n=8)
    reported(cache)
    assert torch.equal(out[:6], good[:6]) and (out[6:] == 7).all()
    out = attend([0, 3, 6, 9], requests=ints([0, 5, 2]))
    reported(cache)
    assert torch.equal(out[:3], good[:3]) and (out[3:6] == 7).all() and torch.equal(out[6:], good[6:])
    # a block that the cache does not have: its keys are not seen
    out = attend([0, 3, 6, 9], table=ints([[0, 1, -1], [2, 1000, -1], [4, 5, 6]]))
    reported(cache)
    assert torch.equal(out[:3], good[:3]) and torch.equal(out[6:], good[6:]) and not torch.equal(out[3:6], good[3:6])
    # a slot behind the last block: the row is skipped
    before = [x.clone() for x in (k, v, ks, vs)]
    rows = torch.randn((2, H, D), device="cuda")
    cache.append(ints([N * T, N * T + 5]), rows, rows)
    reported(cache)
    assert all(torch.equal(a, b) for a, b in zip(before, (k, v, ks, vs)))
    if os.environ.get("DFLASH_DEBUG_MARK"):
        with open(os.environ["DFLASH_DEBUG_MARK"], "w") as f:
            f.write("ok\n")


def test_debug_build_reports():
    if DEBUG:
        pytest.skip("already the child process")
    pkg.build(debug=True)
    mark = os.path.join(ROOT, "speculative_block_draft_gb300", "_build_debug", "cache_reports.ok")
    if os.path.exists(mark):
        os.remove(mark)
    env = dict(os.environ, DFLASH_DEBUG_CHECKS="1", DFLASH_DEBUG_MARK=mark)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-k", "numbers_out_of_range or ragged_rows or speculation",
                        "tests/test_gpu_cache_debug.py", "tests/test_gpu_cache.py", "tests/test_gpu_cache_rings.py"], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=1200)
    print(r.stdout[-3000:], r.stderr[-2000:])
    assert r.returncode == 0
    assert os.path.exists(mark), "the reporting case did not run on the debug library"
