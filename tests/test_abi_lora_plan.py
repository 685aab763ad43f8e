"""Refusals of the adapter projection's plan query (before any CUDA call)."""

import ctypes

import pytest


@pytest.mark.parametrize("size,rc", [((0, 1, 64, 64, 1, 8), -1), ((4, 0, 64, 64, 1, 8), -1),
                                     ((4, 3, 64, 64, 1, 8), -1), ((4, 1, 60, 64, 1, 8), -2),
                                     ((4, 1, 64, 0, 1, 8), -2), ((4, 1, 64, 64, 0, 8), -2),
                                     ((4, 1, 64, 64, 1, 12), -2)])
def test_refusals(size, rc):
    from speculative_decoding_tree_03_gb300 import build as b
    b.build()
    import speculative_decoding_tree_03_gb300 as sv
    lib = sv.load_library()
    assert lib.svf_debug_lora_plan(*size, (ctypes.c_int32 * 6)()) == rc
    assert lib.svf_debug_lora_plan(*size, None) == -1


def test_deadline_hook():
    import speculative_decoding_tree_03_gb300 as sv
    lib = sv.load_library()
    assert lib.svf_debug_set_lora_wait_ns(1) == sv.SVF_OK
    assert lib.svf_debug_set_lora_wait_ns(-5) == sv.SVF_OK   # the default again
