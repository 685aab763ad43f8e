"""Sizes that 32 bits do not hold are refused through the public calls."""

import pytest
import torch

from test_gpu_pages import sv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page_size", [(1 << 32) + 16, 1 << 31, -(1 << 32) + 16])
def test_page_sizes(sv, page_size):  # noqa: F811
    i32 = dict(dtype=torch.int32, device="cuda")
    pool, table = sv.page_pool(8), torch.full((2, 4), -1, **i32)
    lens, new = torch.zeros(2, **i32), torch.tensor([5, 6], **i32)
    o = {k: torch.zeros(n, **i32) for k, n in (("slots", 11), ("positions", 11),
                                               ("row_offsets", 3), ("status", 2))}
    r = {"n_released": torch.zeros(2, **i32), "status": torch.zeros(2, **i32)}
    for given in (o, None):
        with pytest.raises(sv.SpecVerifyError):
            sv.page_reserve(pool, table, lens, new, page_size, 11, outputs=given)
    for given in (r, None):
        with pytest.raises(sv.SpecVerifyError):
            sv.page_release(pool, table, new, lens, page_size, outputs=given)
    torch.cuda.synchronize()
    assert pool["state"].tolist() == [8, 0, 0, 0] and bool((table == -1).all())
