"""EAGLE-2 pools whose arrays just fill a block's default shared memory."""

import os
import subprocess
import sys

import numpy as np
import pytest

from test_gpu_eagle2 import _build_both, _compare_final

pytestmark = pytest.mark.gpu


def finalize(sv, capacity):
    rng = np.random.default_rng(capacity)
    gout, oout, exact = _build_both(sv, rng, 2, 300, 4, 4, 40, capacity=capacity)
    _compare_final(gout, oout, exact)


def test_finalize_where_the_pool_fills_the_default_shared_memory():
    """In a process of its own: a larger pool before these would raise the limit."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = ("import sys; sys.path[:0] = [%r, %r]\n"
            "import speculative_decoding_tree_03_gb300 as sv\n"
            "from test_gpu_eagle2_limits import finalize\n"
            "for C in (1114, 1115, 1116, 1117, 1118, 2048): finalize(sv, C)\n"
            % (here, os.path.dirname(here)))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
