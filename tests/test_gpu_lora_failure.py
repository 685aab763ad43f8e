"""The adapter projection's waits run out: the call comes back, says so, and the
next one is exact. A deadline of 1 ns makes the first wait that is not already
over give up; the others end at different places of the kernels."""

import numpy as np
import pytest
import torch

from test_gpu_lora_plan import plan_of
from test_gpu_lora_proj import case, check, sv  # noqa: F401

pytestmark = pytest.mark.gpu

TIMEOUT = 16

# rows, rows per id, H, O, adapters, rank; then: CTAs of a tile, K shared, several tiles each
SIZES = [
    ((128, 1, 1024, 6144, 60, 16), (1, False, False)),
    ((64, 4, 256, 20480, 8, 24), (1, False, True)),
    ((64, 1, 2048, 1024, 64, 16), (1, True, False)),
    ((1, 1, 4096, 6144, 1, 16), (1, True, False)),
    ((240, 60, 4096, 6144, 3, 64), (2, False, False)),
    ((600, 1, 256, 40000, 60, 40), (2, False, True)),
    ((256, 16, 4104, 4099, 9, 24), (2, True, False)),
]


@pytest.mark.parametrize("size,variant", SIZES)
def test_waits_run_out_and_the_next_call_is_exact(sv, size, variant):  # noqa: F811
    lib = sv.load_library()
    R, per, H, O, adapters, rank = size
    p = plan_of(sv, *size)
    assert (p["ctas"], p["share"] > 1, p["tiles"] > p["resident"]) == variant, p
    ids = np.arange(R // per) % (adapters + 1) - 1
    ids[-1] = adapters - 1
    c = case(R, R, H, O, rank, adapters, ids)
    want = check(sv, c)
    try:
        for ns in (1, 500, 2000, 5000, 10000, 20000, 40000):
            assert lib.svf_debug_set_lora_wait_ns(ns) == 0
            _, status = sv.lora_proj(**c)
            torch.cuda.synchronize()
            assert int(status[0]) in ((TIMEOUT,) if ns == 1 else (0, TIMEOUT)), (ns, status[0])
            assert not bool(status[1:].any()), ns
            assert lib.svf_debug_set_lora_wait_ns(0) == 0
            for _ in range(3):
                got, status = sv.lora_proj(**c)
                torch.cuda.synchronize()
                assert torch.equal(got, want) and not bool(status.any()), ns
    finally:
        lib.svf_debug_set_lora_wait_ns(0)
