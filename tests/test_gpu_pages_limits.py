"""Page calls at the ends of their documented range: batch sizes whose sums just
fill a block's default shared memory, and the largest batch."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from test_gpu_pages import Model, dev, run_release, run_reserve, sv, up, world  # noqa: F401

pytestmark = pytest.mark.gpu


def release_all(sv, B):  # noqa: F811
    ps, mp, spare = 8, 4, 21
    _, lens, table, free, n = world(B, B, ps, mp, ps * mp, spare)
    m = Model(table, free, spare, ps, n)
    pool = {"free": dev(free), "state": dev(np.array([spare, 0, 0, 0], np.int32))}
    run_release(sv, m, pool, dev(table), lens, np.zeros(B, np.int32))
    assert m.count == n


def test_release_where_its_sums_fill_the_default_shared_memory(sv):  # noqa: F811
    """In a process of its own: a larger batch before these would raise the limit."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import speculative_decoding_tree_03_gb300 as sv\n"
            "from test_gpu_pages_limits import release_all\n"
            "for B in (6031, 6032, 6040, 6048, 6049): release_all(sv, B)\n"
            % (here, os.path.dirname(here)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("scarce", [False, True])
def test_reserve_for_the_largest_batch(sv, scarce):  # noqa: F811
    B, ps, mp = 8192, 16, 9
    rng, lens, table, free, n = world(77, B, ps, mp, 100, 12000)
    new = rng.integers(0, 41, B).astype(np.int32)
    need = sum(up(int(a + b), ps) - up(int(a), ps) for a, b in zip(lens, new))
    assert need < 12000
    m = Model(table, free, need // 2 if scarce else 12000, ps, n)
    run_reserve(sv, m, lens, new, int(new.sum()) + 5)


def test_batches_past_the_limit_are_refused(sv):  # noqa: F811
    B = 8193
    i = torch.zeros(B, dtype=torch.int32, device="cuda")
    table = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    pool = sv.page_pool(4)
    for call in (lambda: sv.page_reserve(pool, table, i, i, 16, 4),
                 lambda: sv.page_release(pool, table, i, i, 16)):
        with pytest.raises(sv.SpecVerifyError):
            call()
