"""The inner products of the adapter projection: every size of their tiles and
every way to share them out among CTAs, against the definition."""

import numpy as np
import pytest

from test_gpu_lora_proj import case, check, sv  # noqa: F401

pytestmark = pytest.mark.gpu

# groups, rows each, H, O, adapters, ranks: tiles of 32 rows (groups of 31 rows or more, 1024 rows
# or more) and of 16, each with 8, 16 and 32 columns of a rank
SHAPES = [
    (35, 31, 520, 40, 5, (8, 16, 24, 128)),      # 1085 rows: the last tile is cut
    (32, 32, 4096, 64, 9, (8, 16, 64)),
    (8, 128, 1000, 33, 3, (8, 16, 40)),          # the rows of a tile have one adapter
    (64, 16, 264, 40, 30, (8, 16, 32)),          # groups of 16 rows
    (2, 513, 72, 40, 2, (8, 16, 96)),            # the two requests meet in one tile
    (24, 21, 600, 40, 24, (8, 16, 56)),          # 504 rows
]


@pytest.mark.parametrize("G,per,H,O,adapters,rank",
                         [s[:5] + (r,) for s in SHAPES for r in s[5]])
def test_tiles(sv, G, per, H, O, adapters, rank):  # noqa: F811
    rng = np.random.default_rng(G + per + rank)
    ids = rng.integers(-1, adapters, G)
    ids[0] = adapters - 1
    check(sv, case(rank, G * per, H, O, rank, adapters, ids))


# K shared by up to 8 CTAs; an adapter of a tile per CTA, and several; what is read small and large
@pytest.mark.parametrize("G,per,H,O,adapters,rank", [
    (1, 1, 8192, 40, 1, 16), (32, 1, 4096, 40, 32, 128), (64, 1, 14336, 40, 40, 16),
    (256, 1, 4096, 40, 200, 16), (384, 1, 4096, 33, 300, 16), (160, 4, 4096, 40, 160, 32),
    (128, 4, 4096, 40, 128, 16), (512, 1, 4096, 40, 400, 32), (1000, 1, 2048, 40, 900, 16),
    (4000, 1, 512, 40, 100, 16), (700, 2, 1024, 40, 300, 64)])
def test_shares(sv, G, per, H, O, adapters, rank):  # noqa: F811
    ids = np.arange(G) * 7 % (adapters + 1) - 1
    ids[G // 2] = adapters - 1
    check(sv, case(G + rank, G * per, H, O, rank, adapters, ids))
