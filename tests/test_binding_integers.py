"""Integers that the C interface does not hold are refused, not cut to 32 bits."""

import ctypes
import types

import pytest


@pytest.fixture
def sv(monkeypatch):
    from speculative_decoding_tree_03_gb300 import build as b
    b.build()
    import speculative_decoding_tree_03_gb300 as m
    m.load_library()
    monkeypatch.setattr(m, "_current_device", lambda: 0)
    return m


def test_integers_past_32_bits(sv):
    stream = types.SimpleNamespace(cuda_stream=0)
    seen = []

    def fn(*args):
        seen.append(args)
        return sv.SVF_OK

    fn.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t,
                   ctypes.c_void_p]
    sv._call(fn, "call", 0, stream, 1 << 40, (1 << 31) - 1, 1 << 40, 1 << 40)
    assert seen == [(1 << 40, (1 << 31) - 1, 1 << 40, 1 << 40, 0)]
    for v in (1 << 31, (1 << 32) + 16, -(1 << 31) - 1):
        with pytest.raises(sv.SpecVerifyError, match="32 bits"):
            sv._call(fn, "call", 0, stream, 0, v, 0, 0)
    assert len(seen) == 1


def test_the_declared_signatures_are_what_is_checked(sv):
    """A page size of 2^32 + 16 is not one of 16 (the library returns 0 for no sequences)."""
    lib, stream = sv.load_library(), types.SimpleNamespace(cuda_stream=0)
    args = lambda ps: (0, 4, ps, 0, 0, 8, 0, 0, 0, 0, 0)  # noqa: E731
    sv._call(lib.svf_page_release, "svf_page_release", 0, stream, *args(16))
    with pytest.raises(sv.SpecVerifyError, match="svf_page_release"):
        sv._call(lib.svf_page_release, "svf_page_release", 0, stream, *args((1 << 32) + 16))
