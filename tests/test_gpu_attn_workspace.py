"""The attention workspaces that the binding makes itself begin at zero, as the
persistent kernel's counters have to, wherever their memory comes from."""

import numpy as np
import pytest
import torch

from gpu_common import device_inputs, oracle_attention
from synth import make_inputs
from synth.gen import Workload

pytestmark = pytest.mark.gpu

W = Workload("two_halves", B=2, N=31, tree="binary", binary_depth=4, L=3000, Hq=32, Hkv=2, D=128,
             dtype="bf16", V=2000, target_sigma=3.0, draft_sigma=1.5, page_size=16)
TOL = 2e-2


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_tree_03_gb300 import build as _b
    _b.build()
    import speculative_decoding_tree_03_gb300 as m
    return m


@pytest.fixture
def persistent(sv):
    lib = sv.load_library()
    assert lib.svf_debug_set_attn_kernel(2) == 0
    yield lib
    lib.svf_debug_set_attn_kernel(0)


@pytest.fixture(scope="module")
def data():
    inp = make_inputs(W, 5)
    return device_inputs(inp), oracle_attention(inp)[0]


def size(sv, d):
    return sv.tree_verify_attn_workspace_size(W.B, W.N, W.Hq, W.Hkv, W.D, torch.bfloat16,
                                              d["page_table"].shape[1], d["k"].shape[1])


def leave_ones(need):
    """Free memory of the workspace's size, on the current stream, full of ones."""
    held = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del held


def check(out, status, ref):
    assert not bool(status.any())
    assert np.abs(out.float().cpu().numpy() - ref.reshape(out.shape)).max() <= TOL


@pytest.mark.parametrize("side", [False, True])
def test_verify_step(sv, persistent, data, side):
    d, ref = data
    need = size(sv, d)
    assert need > 0
    stream = torch.cuda.Stream() if side else None
    with torch.cuda.stream(stream):
        leave_ones(need)
    torch.cuda.synchronize()
    for _ in range(2):
        out, _, _, bufs = sv.verify_step(d["parent"], d["tokens"], d["q"], d["k"], d["v"],
                                         d["page_table"], d["seq_lens"], d["target"], d["draft"],
                                         d["u_accept"], d["u_bonus"], stream=stream)
        torch.cuda.synchronize()
        check(out, bufs["attn_status"], ref)
        # every call leaves the counters, the workspace's last bytes, at zero
        assert not bool(bufs["attn_ws"][-16:].any())


def attend(sv, d, stream=None):
    out, _, status, *_ = sv.tree_mask_attn(d["parent"], d["q"], d["k"], d["v"], d["page_table"],
                                           d["seq_lens"], stream=stream)
    return out, status


def test_the_shared_workspace_is_zeroed_on_the_call_s_stream(sv, persistent, data, monkeypatch):
    """The current stream is busy while the call runs on another one."""
    d, ref = data
    attend(sv, d)                # whatever a first call sets up
    torch.cuda.synchronize()
    monkeypatch.setattr(sv, "_ZEROED_WS", {})
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        leave_ones(size(sv, d))
    leave_ones(size(sv, d))
    torch.cuda._sleep(40_000_000)      # about 20 ms of the current stream
    out, status = attend(sv, d, stream=side)
    torch.cuda.synchronize()
    check(out, status, ref)


@pytest.mark.parametrize("kept", [False, True])
def test_a_captured_call_has_a_workspace_of_the_graph(sv, persistent, data, monkeypatch, kept):
    """The graph's first call makes no workspace for eager calls, and a larger
    eager shape does not take the graph's away."""
    d, ref = data
    attend(sv, d)
    torch.cuda.synchronize()
    if not kept:
        monkeypatch.setattr(sv, "_ZEROED_WS", {})
    before = dict(sv._ZEROED_WS)
    leave_ones(size(sv, d))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, status = attend(sv, d)
    assert {k: t.data_ptr() for k, t in sv._ZEROED_WS.items()} == {
        k: t.data_ptr() for k, t in before.items()}
    check(*attend(sv, d), ref)            # eager, before the first replay
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(out, status, ref)
    need = size(sv, d)
    sv._zeroed_workspace(4 * max(need, max(t.numel() for t in sv._ZEROED_WS.values())),
                         torch.device("cuda", 0))    # a larger shape: the kept one is replaced
    leave_ones(need)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    check(out, status, ref)


def test_verify_step_first_called_in_a_capture(sv, persistent, data):
    """The buffers that such a call leaves serve an eager call before any replay."""
    d, ref = data
    args = [d[k] for k in ("parent", "tokens", "q", "k", "v", "page_table", "seq_lens", "target",
                           "draft", "u_accept", "u_bonus")]
    sv.verify_step(*args)
    leave_ones(size(sv, d))
    bufs = {}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.verify_step(*args, buffers=bufs)
    for call in (lambda: sv.verify_step(*args, buffers=bufs), g.replay,
                 lambda: sv.verify_step(*args, buffers=bufs), g.replay):
        if "attn_out" in bufs:
            bufs["attn_out"].zero_()
        call()
        torch.cuda.synchronize()
        check(bufs["attn_out"], bufs["attn_status"], ref)
