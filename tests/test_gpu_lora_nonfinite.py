"""Infinite inner products that meet infinities of the same adapter: every
element is what the definition gives in 64 bits, infinity or NaN, and rows of
other requests are bit for bit as without them."""

import numpy as np
import pytest
import torch

from test_gpu_lora_proj import case, check, sv  # noqa: F401

pytestmark = pytest.mark.gpu


# one CTA per tile; K shared by a cluster; pairs; pairs that share K; several tiles each
@pytest.mark.parametrize("R,H,O,rank", [(64, 512, 256, 16), (64, 2048, 1024, 16),
                                        (240, 2048, 6144, 64), (256, 4104, 4099, 24),
                                        (600, 256, 40000, 40), (33, 64, 40, 96)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
def test_infinity_times_infinity(sv, value, R, H, O, rank):  # noqa: F811
    ids = np.arange(R) % 4 - 1          # every 16-row window holds every adapter
    c = case(3 + R, R, H, O, rank, 3, ids)
    c["x"][:, 60] = torch.where(c["x"][:, 60] == 0, 1.0, c["x"][:, 60])
    c["scales"][1] = 0.75
    clean = check(sv, c)
    mine = torch.as_tensor(ids == 1, device="cuda")
    d = dict(c, lora_a=c["lora_a"].clone(), lora_b=c["lora_b"].clone())
    last = rank - 1
    d["lora_a"][1, last, 60] = value    # t is infinite there, with the sign of x
    for col, j, b in ((17, last, "inf"), (18, last, "-inf"), (19, last, "nan"), (20, last, "0"),
                      (21, 3, "inf"), (O - 1, last, "inf")):
        d["lora_b"][1, col, j] = float(b)
    t = d["scales"][1].double() * (d["x"][mine].double() @ d["lora_a"][1].double().T)
    assert bool(t[:, last].isinf().all()) and bool(t[:, :last].isfinite().all())
    want = d["x"][mine].double() @ d["weight"].double().T + t @ d["lora_b"][1].double().T
    assert bool(want[:, 17].isinf().all())
    got, status = sv.lora_proj(**d)
    torch.cuda.synchronize()
    assert int(status.abs().sum()) == 0
    assert torch.equal(got[~mine], clean[~mine])
    got = got[mine].double()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.nan_to_num(0.0, 1.0, -1.0), want.nan_to_num(0.0, 1.0, -1.0))
