"""Per-head norms with rotary positions and the K/V write against the definition in 64 bits.

Bound per element, derived from the kernel's arithmetic (u = 2^-24): the sum of D squares in fp32 is off
by at most (D + 2) u relative, its mean with eps by two more roundings, rsqrt by 2 units (4 u); a
square root halves what is inside it, so the factor of the norm is off by ((D + 4) / 2 + 4) u, and
x r g has two roundings more: n = (D / 2 + 8) u relative. The turn then adds what rope_kv_write's
adds: 2 u (|y_a c| + |y_b s|), on terms that are off by n: (n + 2 u) (|y_a c| + |y_b s|) in
all, and the rounding to bf16 half a step, 2^-8 (1 + 2^-6) of the value. Without weights n = 0.
What is copied is equal bit for bit."""

import pytest
import torch

from test_gpu_rope_kv import BAD_LENGTH, BAD_PAGE, case, table

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_tree_03_gb300 import build as _b
    _b.build()
    import speculative_decoding_tree_03_gb300 as m
    return m


def expected(x, w, eps, cs, rot, inter):
    """The definition in 64 bits and its bound; cs [rows, rot] gathered per pair."""
    D = x.shape[-1]
    y, n = x.double(), 0.0
    if w is not None:
        y = y * (y.square().mean(-1, keepdim=True) + eps).rsqrt() * w.double()
        n = (D / 2 + 8) * U
    cs = cs.double()
    z, mag = y.clone(), torch.zeros_like(y)
    tol = n * y.abs()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        c, s = cs[:, None, i], cs[:, None, rot // 2 + i]
        z[..., a] = y[..., a] * c - y[..., b] * s
        z[..., b] = y[..., b] * c + y[..., a] * s
        mag[..., a] = (y[..., a] * c).abs() + (y[..., b] * s).abs()
        mag[..., b] = (y[..., b] * c).abs() + (y[..., a] * s).abs()
    tol[..., :rot] = (n + 2 * U) * mag[..., :rot]
    if x.dtype == BF:
        tol = tol * (1 + 2.0 ** -7) + 2.0 ** -8 * (1 + 2.0 ** -6) * z.abs()
    else:
        tol = tol + U * z.abs()
    return z, tol


def axes_of(c, seed, axes, rot, max_pos):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T = c["q"].shape[0]
    pos = torch.randint(0, max_pos, (axes, T), generator=g, device="cuda").int()
    axis = torch.randint(0, axes, (rot // 2,), generator=g, device="cuda").int()
    return pos, axis


def gathered(rope, pos, axis, rot):
    if axis is None:
        return rope[pos.view(-1).long()]
    i = torch.arange(rot // 2, device="cuda")
    p = pos.long()[axis.long()].T
    return torch.cat([rope[p, i], rope[p, rot // 2 + i]], 1)


def check(sv, c, w, pos, axis, inter=False, eps=1e-6, q_out=None):
    rope, rot = c["rope"], c["rope"].shape[1]
    kc, vc = c["k_cache"].clone(), c["v_cache"].clone()
    ins = {n: c[n].clone() for n in ("q", "k", "v")}
    q_out = torch.full_like(c["q"], 7.0).contiguous() if q_out is None else q_out
    before = q_out.clone()
    out, status = sv.norm_rope_kv_write(c["q"], c["k"], c["v"], w[0], w[1], rope, pos, c["slots"],
                                        c["k_cache"], c["v_cache"], eps=eps, pair_axis=axis,
                                        q_out=q_out, interleaved=inter)
    torch.cuda.synchronize()
    slots = c["slots"].long()
    n_slots, max_pos = kc.shape[0] * kc.shape[1], rope.shape[0]
    left_out = slots == -1
    st = torch.zeros_like(slots)
    st[(slots < -1) | (slots >= n_slots)] |= BAD_PAGE
    p2 = pos.view(-1, pos.shape[-1])
    st[((p2 < 0) | (p2 >= max_pos)).any(0)] |= BAD_LENGTH
    if axis is not None and p2.shape[0] > 1 and bool(((axis < 0) | (axis >= p2.shape[0])).any()):
        st |= BAD_LENGTH
    st[left_out] = 0
    assert torch.equal(status.long(), st)
    good = ~left_out & (st == 0)
    assert bool((out[st != 0] == 0).all())
    assert torch.equal(out[left_out], before[left_out])
    rest = torch.ones(n_slots, dtype=torch.bool, device="cuda")
    rest[slots[good]] = False
    for cache, old in ((c["k_cache"], kc), (c["v_cache"], vc)):
        assert torch.equal(cache.flatten(0, 1)[rest], old.flatten(0, 1)[rest])
    assert torch.equal(c["v_cache"].flatten(0, 1)[slots[good]], ins["v"][good])
    if not bool(good.any()):
        return
    cs = gathered(rope, p2[:, good] if axis is not None else p2[0][good], axis, rot)
    for got, x, g in ((out[good], ins["q"], w[0]),
                      (c["k_cache"].flatten(0, 1)[slots[good]], ins["k"], w[1])):
        z, tol = expected(x[good], g, eps, cs, rot, inter)
        err = (got.double() - z).abs()
        assert bool((err <= tol).all()), float((err / tol.clamp(min=1e-30)).max())
        if g is None:
            assert torch.equal(got[..., rot:], x[good][..., rot:])


def weights(seed, D, dt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dt) for _ in range(2)]


SHAPES = [  # T, Hq, Hkv, D, rot
    (1, 32, 8, 128, 128), (31, 4, 4, 64, 64), (5, 7, 1, 64, 32), (3, 1, 1, 16, 16),
    (67, 64, 8, 128, 128), (700, 32, 8, 128, 64), (2, 9, 3, 256, 256), (9, 5, 5, 256, 240),
    (4, 3, 2, 40, 16), (130, 64, 64, 96, 96), (1500, 8, 2, 80, 48), (3, 0, 2, 128, 128),
    (40, 3, 1, 112, 16)]


@pytest.mark.parametrize("axes", [1, 3])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot", SHAPES)
def test_matches_definition(sv, T, Hq, Hkv, D, rot, dt, inter, axes):
    c = case(T + D, T, Hq, Hkv, D, rot, dt)
    pos, axis = axes_of(c, T, axes, rot, 5000) if axes > 1 else (c["positions"], None)
    check(sv, c, weights(D, D, dt), pos, axis, inter)


@pytest.mark.parametrize("dt", [BF, F32])
def test_norm_of_one_side_or_none(sv, dt):
    for i, w in enumerate(((None, None), (0, None), (None, 1))):
        c = case(5 + i, 90, 6, 2, 64, 32, dt, fused=True)
        g = weights(3, 64, dt)
        pos, axis = axes_of(c, 9, 2, 32, 5000)
        check(sv, c, [None if k is None else g[k] for k in w], pos, axis)


def test_without_norms_one_axis_is_rope_kv_write(sv):
    c = case(8, 200, 8, 2, 128, 64, BF)
    q, st = sv.rope_kv_write(**c)
    kc, vc = c["k_cache"].clone(), c["v_cache"].clone()
    c["k_cache"].zero_()
    c["v_cache"].zero_()
    q2, st2 = sv.norm_rope_kv_write(c["q"], c["k"], c["v"], None, None, c["rope"],
                                    c["positions"].view(1, -1), c["slots"], c["k_cache"],
                                    c["v_cache"])
    at = c["slots"].long()
    assert torch.equal(q, q2) and torch.equal(st, st2)
    for a, b in ((kc, c["k_cache"]), (vc, c["v_cache"])):
        assert torch.equal(a.flatten(0, 1)[at], b.flatten(0, 1)[at])


@pytest.mark.parametrize("dt", [BF, F32])
def test_large_small_and_zero_heads(sv, dt):
    """Heads of zeros (eps keeps them 0), tiny ones (eps is all there is) and large ones."""
    c = case(12, 64, 4, 2, 128, 128, dt)
    for n in ("q", "k"):
        c[n][::4] = 0
        c[n][1::4] *= 1e-12
        c[n][2::4] *= 1e12
    check(sv, c, weights(1, 128, dt), c["positions"], None)
    check(sv, c, weights(1, 128, dt), c["positions"], None, eps=0.01)


@pytest.mark.parametrize("axes", [1, 4])
def test_bad_rows(sv, axes):
    c = case(13, 60, 4, 2, 128, 128, BF)
    pos, axis = axes_of(c, 2, axes, 128, 5000) if axes > 1 else (c["positions"], None)
    c["slots"][3] = -1
    c["slots"][4] = -2
    c["slots"][5] = c["k_cache"].shape[0] * c["k_cache"].shape[1]
    pos[..., 7] = 5000
    pos.view(-1, 60)[axes - 1, 8] = -1
    pos[..., 3] = -4   # left out all the same
    check(sv, c, weights(2, 128, BF), pos, axis)
    if axes > 1:
        axis[17] = axes
        check(sv, c, weights(2, 128, BF), pos, axis)


def test_non_finite_heads_stay_alone(sv):
    c = case(14, 8, 4, 2, 128, 128, BF)
    w = weights(2, 128, BF)
    want, _ = sv.norm_rope_kv_write(c["q"], c["k"], c["v"], *w, c["rope"], c["positions"],
                                    c["slots"], c["k_cache"].clone(), c["v_cache"].clone())
    c["q"] = c["q"].clone()
    c["q"][2, 1, 5], c["q"][4, 3, 100] = float("nan"), float("inf")
    got, _ = sv.norm_rope_kv_write(c["q"], c["k"], c["v"], *w, c["rope"], c["positions"],
                                   c["slots"], c["k_cache"], c["v_cache"])
    same = torch.ones(8, 4, dtype=torch.bool, device="cuda")
    same[2, 1] = same[4, 3] = False
    assert torch.equal(got[same], want[same])
    assert bool(got[2, 1].isnan().all()) and bool(got[4, 3].isnan().any())


def test_in_place_other_stream_and_captured(sv):
    c = case(15, 300, 8, 2, 128, 128, BF)
    w = weights(4, 128, BF)
    c["q"] = c["q"].contiguous()
    check(sv, dict(c, q=c["q"].clone()), w, c["positions"], None)
    pos, axis = axes_of(c, 6, 3, 128, 5000)
    args = lambda: (c["q"], c["k"], c["v"], *w, c["rope"], pos, c["slots"], c["k_cache"], c["v_cache"])  # noqa: E731
    want, _ = sv.norm_rope_kv_write(*args(), pair_axis=axis)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, _ = sv.norm_rope_kv_write(*args(), pair_axis=axis, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out, status = torch.zeros_like(want), torch.zeros(300, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.norm_rope_kv_write(*args(), pair_axis=axis, q_out=out, status=status)
    pos.copy_(pos.flip(0))
    want, _ = sv.norm_rope_kv_write(*args(), pair_axis=axis)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    want = want.clone()
    q = c["q"]
    sv.norm_rope_kv_write(*args(), pair_axis=axis, q_out=q)
    assert torch.equal(q, want)


def test_table_of_many_positions(sv):
    assert table(4, 16).shape == (4, 16)
    c = case(16, 33, 2, 1, 64, 64, F32, max_pos=40000)
    check(sv, c, weights(4, 64, F32), c["positions"], None)
