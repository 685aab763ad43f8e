"""The rotary K/V write against its definition in 64 bits.

Bound per element, derived from the kernel's arithmetic: one product rounded
to fp32, one fused multiply-add (two roundings of at most 2^-24 of the terms),
and the rounding to the element type (half a step: 2^-8 relative for bf16, 2^-24
for fp32, the latter in the 2^-24 of the result already):
    |y - y64| <= 2 * 2^-24 (|x_a c| + |x_b s|) + half_step * |y64|,
with 1 + 2^-6 on top of half_step for the step taken at the rounded value.
What is copied (v, elements from rot on, rows that are left out) is equal bit
for bit."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BAD_PAGE, BAD_LENGTH = 4, 8
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_tree_03_gb300 import build as _b
    _b.build()
    import speculative_decoding_tree_03_gb300 as m
    return m


def table(max_pos, rot, base=10000.0):
    i = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda")
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * base ** (-i / rot)
    return torch.cat([a.cos(), a.sin()], 1).float()


def turned(x, cs, rot, inter):
    """The definition in 64 bits, and the magnitude of its terms."""
    x, cs = x.double(), cs.double()
    y, mag = x.clone(), torch.zeros_like(x)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        c, s = cs[:, None, i], cs[:, None, rot // 2 + i]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = (x[..., a] * c).abs() + (x[..., b] * s).abs()
        mag[..., b] = (x[..., b] * c).abs() + (x[..., a] * s).abs()
    return y, mag


def close(got, x, cs, rot, inter):
    y, mag = turned(x, cs, rot, inter)
    half = HALF[x.dtype] * (1 + 2.0 ** -6) if x.dtype == torch.bfloat16 else 0.0
    bound = 2 * 2.0 ** -24 * mag + half * y.abs()
    err = (got.double() - y).abs()
    assert bool((err <= bound).all()), float((err - bound).max())
    assert torch.equal(got[..., rot:], x[..., rot:])


def case(seed, T, Hq, Hkv, D, rot, dt, ps=16, max_pos=5000, fused=False, pad=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)
    if fused:  # a fused projection with other columns in front and behind
        unit = 16 // r(1).element_size()
        f = r(T, (Hq + 2 * Hkv) * D + 3 * unit)
        cut = lambda at, h: f[:, at:at + h * D].unflatten(1, (h, D))
        q, k, v = cut(unit, Hq), cut(unit + Hq * D, Hkv), cut(unit + (Hq + Hkv) * D, Hkv)
    else:
        q, k, v = r(T, Hq, D), r(T, Hkv, D), r(T, Hkv, D)
    pages = -(-T // ps) + 2
    slots = torch.randperm(pages * ps, generator=g, device="cuda")[:T].int()
    pos = torch.randint(0, max_pos, (T,), generator=g, device="cuda").int()
    return dict(q=q, k=k, v=v, rope=table(max_pos, rot), positions=pos, slots=slots,
                k_cache=r(pages, ps, Hkv, D), v_cache=r(pages, ps, Hkv, D))


def check(sv, c, inter=False, q_out=None):
    kc, vc = c["k_cache"].clone(), c["v_cache"].clone()
    ins = {n: c[n].clone() for n in ("q", "k", "v")}
    q_out = torch.full_like(c["q"], 7.0).contiguous() if q_out is None else q_out
    before = q_out.clone()
    rot, max_pos = c["rope"].shape[1], c["rope"].shape[0]
    out, status = sv.rope_kv_write(**c, q_out=q_out, interleaved=inter)
    torch.cuda.synchronize()
    assert out is q_out
    slots, pos = c["slots"].long(), c["positions"].long()
    n_slots = kc.shape[0] * kc.shape[1]
    out_row = slots == -1
    st = torch.zeros_like(slots)
    st[(slots < -1) | (slots >= n_slots)] |= BAD_PAGE
    st[(pos < 0) | (pos >= max_pos)] |= BAD_LENGTH
    st[out_row] = 0
    assert torch.equal(status.long(), st)
    good = ~out_row & (st == 0)
    cs = c["rope"][pos[good]]
    close(out[good], ins["q"][good], cs, rot, inter)
    assert bool((out[st != 0] == 0).all())
    assert torch.equal(out[out_row], before[out_row])
    for cache, old, x, turn in ((c["k_cache"], kc, ins["k"], True), (c["v_cache"], vc, ins["v"], False)):
        flat = cache.flatten(0, 1)
        if turn:
            close(flat[slots[good]], x[good], cs, rot, inter)
        else:
            assert torch.equal(flat[slots[good]], x[good])
        rest = torch.ones(n_slots, dtype=torch.bool, device="cuda")
        rest[slots[good]] = False
        assert torch.equal(flat[rest], old.flatten(0, 1)[rest])


SHAPES = [  # T, Hq, Hkv, D, rot
    (1, 32, 8, 128, 128), (31, 4, 4, 64, 64), (5, 7, 1, 64, 32), (3, 1, 1, 16, 16),
    (67, 64, 8, 128, 128), (700, 32, 8, 128, 64), (2, 9, 3, 256, 256), (9, 5, 5, 512, 496),
    (4, 3, 2, 40, 16), (130, 64, 64, 96, 96), (1500, 8, 2, 80, 48)]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", SHAPES)
def test_matches_definition(sv, T, Hq, Hkv, D, rot, dt, inter):
    check(sv, case(T + D, T, Hq, Hkv, D, rot, dt), inter)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_fp32_only_rotary_widths(sv, dt):
    """8 rotated elements in a head of 12: fp32 alone takes them."""
    if dt == torch.float32:
        check(sv, case(1, 6, 3, 1, 12, 8, dt))
    else:
        with pytest.raises(sv.SpecVerifyError):
            check(sv, case(1, 6, 3, 1, 16, 8, dt))


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_slices_of_a_fused_projection(sv, dt, inter):
    check(sv, case(2, 93, 16, 4, 128, 128, dt, fused=True), inter)
    check(sv, case(3, 1, 16, 4, 64, 32, dt, fused=True), inter)


def test_rows_without_slot_and_bad_rows(sv):
    c = case(4, 40, 8, 2, 128, 128, torch.bfloat16)
    n = c["k_cache"].shape[0] * 16
    c["slots"][[0, 7, 39]] = -1
    c["slots"][5], c["slots"][6] = -2, n
    c["positions"][[7, 8, 9]] = torch.tensor([-5, -1, 5000], dtype=torch.int32, device="cuda")
    c["slots"][10], c["positions"][10] = 2 ** 31 - 1, -2 ** 31
    # what is left out or flagged may hold anything
    for x in (c["q"], c["k"], c["v"]):
        x[[0, 5, 7, 8]] = float("nan")
    check(sv, c)


def test_non_finite_values_stay_in_their_pair(sv):
    c = case(5, 3, 2, 1, 64, 64, torch.float32)
    c["positions"][:] = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    c["q"][1, 0, 3] = float("inf")
    out, _ = sv.rope_kv_write(**c)
    bad = ~torch.isfinite(out)
    assert bad.nonzero().tolist() == [[1, 0, 3], [1, 0, 35]]


def test_in_place_and_positions_far_out(sv):
    c = case(6, 50, 8, 2, 128, 128, torch.bfloat16, max_pos=140000)
    c["positions"][:] = torch.arange(139950, 140000, dtype=torch.int32, device="cuda")
    check(sv, c, q_out=c["q"])


def test_slots_past_32_bits_of_offset(sv):
    """Rows behind element 2^31 of a cache, and behind byte 2^32."""
    c = case(7, 4, 2, 8, 128, 128, torch.bfloat16)
    pages = (2 ** 31 // (8 * 128)) // 16 + 40
    c["k_cache"] = torch.empty((pages, 16, 8, 128), dtype=torch.bfloat16, device="cuda")
    c["v_cache"] = torch.empty((pages, 16, 8, 128), dtype=torch.bfloat16, device="cuda")
    n = pages * 16
    at = torch.tensor([n - 1, 2 ** 21 + 1, 2 ** 20, 0], device="cuda")
    c["slots"] = at.int()
    for x in (c["k_cache"], c["v_cache"]):
        x.view(-1, 8, 128)[at - torch.tensor([1, 1, 1, -1], device="cuda")] = 3.0
    ins = {x: c[x].clone() for x in "kv"}
    sv.rope_kv_write(**c)
    torch.cuda.synchronize()
    cs = c["rope"][c["positions"].long()]
    close(c["k_cache"].view(-1, 8, 128)[at], ins["k"], cs, 128, False)
    assert torch.equal(c["v_cache"].view(-1, 8, 128)[at], ins["v"])
    for x in (c["k_cache"], c["v_cache"]):
        assert bool((x.view(-1, 8, 128)[at - torch.tensor([1, 1, 1, -1], device="cuda")] == 3.0).all())


def test_k_and_v_alone_and_no_rows(sv):
    c = case(8, 9, 4, 2, 64, 64, torch.float32)
    c["q"] = c["q"][:, :0]
    check(sv, c)
    c = case(8, 9, 4, 2, 64, 64, torch.float32)
    for n in ("q", "k", "v", "positions", "slots"):
        c[n] = c[n][:0]
    kc = c["k_cache"].clone()
    sv.rope_kv_write(**c)
    assert torch.equal(c["k_cache"], kc)


def test_stream_and_capture(sv):
    c = case(9, 64, 8, 2, 128, 128, torch.bfloat16)
    q0 = torch.empty_like(c["q"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    status = torch.empty(64, dtype=torch.int32, device="cuda")
    sv.rope_kv_write(**c, q_out=q0, status=status, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want, wk = q0.clone(), c["k_cache"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.rope_kv_write(**c, q_out=q0, status=status)
    for _ in range(2):
        q0.zero_()
        c["k_cache"].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(q0, want)
        s = c["slots"].long()
        assert torch.equal(c["k_cache"].flatten(0, 1)[s], wk.flatten(0, 1)[s])


def test_binding_refusals(sv):
    c = case(10, 6, 4, 2, 64, 64, torch.bfloat16)
    for change in (dict(q=c["q"].float()), dict(k=c["k"].half()), dict(k=c["k"][:5]),
                   dict(v=c["v"][:, :1]), dict(rope=c["rope"].double()), dict(rope=c["rope"][0]),
                   dict(slots=c["slots"].long()), dict(positions=c["positions"][:5]),
                   dict(k_cache=c["k_cache"].float()), dict(v_cache=c["v_cache"][:1]),
                   dict(k_cache=c["k_cache"].transpose(0, 1)), dict(q=c["q"].transpose(1, 2)),
                   dict(q=c["q"].cpu()), dict(k=c["k"].cpu()), dict(q_out=c["q"][:3]),
                   dict(q=torch.empty(6, 8, 4, device="cuda", dtype=torch.bfloat16).transpose(1, 2)),
                   dict(status=c["slots"][:2])):
        with pytest.raises(sv.SpecVerifyError):
            sv.rope_kv_write(**{**c, **change})
