"""How the adapter projection cuts a call into tiles: every way that the kernel
has is taken by a size that is checked here against the definition, and no size
gets tiles that the kernel's shared memory, tensor memory or clusters do not
hold."""

import ctypes
import random

import numpy as np
import pytest

from test_gpu_lora_proj import case, check, sv  # noqa: F401

pytestmark = pytest.mark.gpu


def plan_of(sv, R, per, H, O, adapters, rank):  # noqa: F811
    p = (ctypes.c_int32 * 6)()
    rc = sv.load_library().svf_debug_lora_plan(R, per, H, O, adapters, rank, p)
    assert rc == 0, (rc, R, per, H, O, adapters, rank)
    return dict(zip(("ctas", "rows", "share", "tiles", "stages", "resident"), p))


# rows, rows per id, H, O, adapters, rank; then: CTAs of a tile, K shared, several tiles each,
# more than 64 rows of x per tile
VARIANTS = [
    ((64, 1, 2048, 1024, 64, 16), (1, True, False, False)),
    ((128, 1, 1024, 6144, 60, 16), (1, False, False, False)),
    ((64, 4, 256, 20480, 8, 24), (1, False, True, False)),
    ((1000, 1, 64, 100, 8, 16), (1, False, False, True)),
    ((200, 1, 4096, 100, 60, 40), (1, True, False, True)),
    ((40000, 5, 64, 100, 8, 16), (1, False, True, True)),
    ((240, 60, 4096, 6144, 3, 64), (2, False, False, True)),
    ((256, 16, 4104, 4099, 9, 24), (2, True, False, True)),
    ((240, 1, 2048, 6144, 60, 96), (2, True, False, True)),
    ((600, 1, 256, 40000, 60, 40), (2, False, True, True)),
]


@pytest.mark.parametrize("size,variant", VARIANTS)
def test_each_variant_against_the_definition(sv, size, variant):  # noqa: F811
    R, per, H, O, adapters, rank = size
    p = plan_of(sv, *size)
    assert (p["ctas"], p["share"] > 1, p["tiles"] > p["resident"], p["rows"] > 64) == variant, p
    rng = np.random.default_rng(R + O)
    ids = rng.integers(-1, adapters, R // per)
    ids[rng.integers(0, len(ids), max(1, len(ids) // 20))] = adapters   # bad ids
    check(sv, case(R + H, R, H, O, rank, adapters, ids))


def test_no_size_gets_tiles_that_do_not_fit(sv):  # noqa: F811
    rng = random.Random(5)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))  # noqa: E731
    for _ in range(3000):
        per = rng.choice([1, 1, log(1, 4096)])
        R = max(per, min(1 << 17, log(1, 1 << 17)) // per * per)
        H, O = 8 * log(1, 8192), log(1, 1 << 20)
        adapters, rank = log(1, 65536), 8 * rng.randint(1, 16)
        size = (R, per, H, O, adapters, rank)
        p = plan_of(sv, *size)
        n, share, ctas = p["rows"], p["share"], p["ctas"]
        assert ctas in (1, 2) and n % 32 == 0 and 32 * ctas <= n <= 256, (size, p)
        assert 1 <= share <= 8 // ctas and share <= (H + 63) // 64, (size, p)
        assert p["tiles"] == -(-O // (128 * ctas)) * -(-R // n), (size, p)
        ring = p["stages"] * (16384 + n // ctas * 128)
        assert 2 <= p["stages"] <= 12 and ring <= 192 * 1024, (size, p)
        assert (1 if share > 1 else 2) * n <= 512, (size, p)            # tensor-memory columns
        if share > 1:   # a partial tile and the other CTAs' parts of one; one tile per cluster
            assert 512 * (n + (share - 1) * -(-n // share)) <= ring, (size, p)
            assert p["tiles"] <= p["resident"], (size, p)
