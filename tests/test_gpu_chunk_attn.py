"""Chunk attention over the paged cache against its definition in 64 bits.

Bounds, from the kernels' arithmetic (u = 2^-24). A score is a sum of D products in fp32; its
error, and that of the scale and of 2^x (2 units each), is at most
    d = (D + 8) u (scale sum |q k|) + 4 u |score|      (fp32; 4 times that for the tensor cores,
                                                        whose sums may be cut, not rounded)
so a weight is off by a factor of at most e^(2 d). The sum of n weighted rows in fp32 adds n + 16 u of
sum w |v| (the running rescales and the joined pieces are in the 16; at most half as many tiles
again), and bf16 rounds each weight and the result by half a step, 2^-8 relative. lse is off by d,
by n u and by 4 u of its own size."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BAD_PAGE, BAD_LENGTH, NO_PAGES, TIMEOUT = 4, 8, 128, 16
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_tree_03_gb300 import build as _b
    _b.build()
    import speculative_decoding_tree_03_gb300 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def case(seed, lens, new, Hq, Hkv, ps, dt, D=128, pad=0, spare=3, extra=2, sharp=2.0):
    """Sequences of lens[b] cached and new[b] new tokens on permuted pages; unused slots are NaN."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    held = [-(-(L + n) // ps) for L, n in zip(lens, new)]
    pages = sum(held) + spare
    perm = torch.randperm(pages, generator=g, device="cuda").int()
    width = max(held + [1]) + extra
    table = torch.full((len(lens), width), -7, dtype=torch.int32, device="cuda")
    kc = torch.full((pages, ps, Hkv, D), float("nan"), device="cuda", dtype=dt)
    vc = kc.clone()
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = perm[at:at + h]
        T = lens[b] + new[b]
        if T:
            t = torch.arange(T, device="cuda")
            p = table[b].long()[t // ps]
            kc[p, t % ps] = torch.randn(T, Hkv, D, generator=g, device="cuda").to(dt)
            vc[p, t % ps] = torch.randn(T, Hkv, D, generator=g, device="cuda").to(dt)
        at += h
    rows = sum(new) + pad
    q = (torch.randn(rows, Hq, D, generator=g, device="cuda") * sharp).to(dt)
    if pad:
        q[sum(new):] = float("nan")
    offs = [0]
    for n in new:
        offs.append(offs[-1] + n)
    return dict(q=q, k_cache=kc, v_cache=vc, page_table=table, seq_lens=i32(lens),
                row_offsets=i32(offs)), (list(lens), list(new))


def reference(c, host, scale):
    """out, its bound, lse, its bound; rows of sequences that are there."""
    q, kc, vc, table = c["q"], c["k_cache"], c["v_cache"], c["page_table"]
    rows, Hq, D = q.shape
    Hkv, ps = kc.shape[2], kc.shape[1]
    G, bf = Hq // Hkv, q.dtype == BF
    out = torch.zeros(rows, Hq, D, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(out)
    lse = torch.zeros(rows, Hq, dtype=torch.float64, device="cuda")
    ltol = torch.zeros_like(lse)
    at = 0
    for b, (L, n) in enumerate(zip(*host)):
        if n == 0:
            continue
        T = L + n
        t = torch.arange(T, device="cuda")
        p = table[b].long()[t // ps]
        k = kc[p, t % ps].double().repeat_interleave(G, 1)   # [T, Hq, D]
        v = vc[p, t % ps].double().repeat_interleave(G, 1)
        step = max(1, int(4e7 // (T * Hq)))
        for i in range(0, n, step):
            m = min(step, n - i)
            qq = q[at + i:at + i + m].double()
            s = torch.einsum("mhd,thd->mht", qq, k) * scale
            mag = torch.einsum("mhd,thd->mht", qq.abs(), k.abs()) * scale
            seen = t[None, None] <= (L + i + torch.arange(m, device="cuda"))[:, None, None]
            s = s.masked_fill(~seen, -math.inf)
            mag = mag.masked_fill(~seen, 0)
            z = torch.logsumexp(s, -1)
            w = (s - z[..., None]).exp()
            d = ((D + 8) * U * (4 if bf else 1) * mag + 4 * U * s.masked_fill(~seen, 0).abs()).amax(-1)
            sl = slice(at + i, at + i + m)
            out[sl] = torch.einsum("mht,thd->mhd", w, v)
            wv = torch.einsum("mht,thd->mhd", w, v.abs())
            rel = torch.expm1(2 * d) + (1.5 * T + 16) * U + (2.0 ** -8 if bf else 0)
            tol[sl] = rel[..., None] * wv
            if bf:
                tol[sl] = tol[sl] * (1 + 2.0 ** -7) + 2.0 ** -8 * out[sl].abs()
            lse[sl] = z
            ltol[sl] = d + (1.5 * T + 16) * U + 4 * U * z.abs()
        at += n
    return out, tol, lse, ltol


def check(sv, c, host, sm_scale=0.0, **kw):
    rows, Hq, D = c["q"].shape
    used = sum(host[1])
    scale = sm_scale if sm_scale > 0 else D ** -0.5
    out = torch.full_like(c["q"], 7.0)
    lse = torch.full((rows, Hq), 5.0, device="cuda")
    got, glse, status = sv.chunk_attn(**c, sm_scale=sm_scale, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert status.tolist() == [0] * len(host[0])
    ref, tol, rl, lt = reference(c, host, scale)
    err = (got[:used].double() - ref[:used]).abs()
    assert bool((err <= tol[:used]).all()), float((err / tol[:used].clamp(min=1e-30)).max())
    lerr = (glse[:used].double() - rl[:used]).abs()
    assert bool((lerr <= lt[:used]).all()), float((lerr / lt[:used].clamp(min=1e-30)).max())
    assert bool((got[used:] == 7.0).all()) and bool((glse[used:] == 5.0).all())
    return got, glse


CASES = [  # lens, new, Hq, Hkv, page_size
    ([0], [1], 4, 4, 16),
    ([5], [1], 8, 1, 16),
    ([128], [1], 32, 8, 16),
    ([127], [2], 32, 8, 64),
    ([2048], [1], 32, 8, 16),
    ([0], [128], 4, 4, 32),
    ([0], [129], 4, 4, 128),
    ([0], [257], 8, 2, 16),
    ([1000], [300], 8, 8, 256),
    ([0, 0, 0], [0, 0, 3], 8, 2, 16),
    ([700, 0, 33, 4000], [1, 0, 100, 2], 28, 4, 32),
    ([17, 300, 0, 64, 1], [40, 1, 513, 64, 127], 14, 2, 16),
    ([100] * 20, [1] * 20, 64, 8, 16),
    ([i * 37 % 900 for i in range(180)], [(i * 5) % 3 for i in range(180)], 8, 4, 16),
    ([60], [70], 5, 5, 16),
    ([3], [9], 64, 1, 64),
    ([0, 900], [1000, 31], 48, 1, 16),
    ([20000], [3], 10, 10, 16),
    ([6000], [700], 24, 24, 64),
]


@pytest.mark.parametrize("lens,new,Hq,Hkv,ps", CASES)
@pytest.mark.parametrize("dt,D", [(F32, 64), (F32, 128), (BF, 128)])
def test_matches_definition(sv, lens, new, Hq, Hkv, ps, dt, D):
    c, host = case(len(lens) + Hq, lens, new, Hq, Hkv, ps, dt, D, pad=3)
    check(sv, c, host)


@pytest.mark.parametrize("dt", [F32, BF])
def test_scale_and_no_lse(sv, dt):
    c, host = case(3, [50, 9], [40, 1], 8, 4, 16, dt)
    got, _ = check(sv, c, host, sm_scale=0.031)
    out, lse, _ = sv.chunk_attn(**c, sm_scale=0.031, want_lse=False)
    assert lse is None and torch.equal(out, got)


@pytest.mark.parametrize("dt", [F32, BF])
def test_same_bits_every_time_and_workspace_of_other_shapes(sv, dt):
    ws = torch.zeros(sv.chunk_attn_workspace_size(4000, 8, 32, 8, 128, dt), dtype=torch.uint8,
                     device="cuda")
    a, ha = case(1, [9000], [33], 32, 8, 16, dt)
    b, hb = case(2, [100, 2000, 50], [700, 1, 30], 28, 4, 32, dt)
    first = check(sv, a, ha, workspace=ws)
    other = check(sv, b, hb, workspace=ws)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(check(sv, a, ha, workspace=ws), first))
        assert all(torch.equal(x, y) for x, y in zip(check(sv, b, hb, workspace=ws), other))


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_later_tokens_hold_what_they_like(sv, dt, what):
    """A token of the chunk whose K and V are not finite reaches its own and later rows only."""
    lens, new, at = [200, 40], [150, 90], [60, 89]
    c, host = case(5, lens, new, 8, 2, 16, dt)
    clean, clse = check(sv, c, host)
    for b in range(2):
        t = lens[b] + at[b]
        page = c["page_table"][b, t // 16].long()
        c["k_cache"][page, t % 16] = what
        c["v_cache"][page, t % 16, :, ::3] = what
    out, lse, _ = sv.chunk_attn(**c)
    torch.cuda.synchronize()
    # a row that is computed again has other roundings
    ref, tol, rl, lt = reference(*case(5, lens, new, 8, 2, 16, dt), 128 ** -0.5)
    row = 0
    for b in range(2):
        before = slice(row, row + at[b])
        assert bool(((out[before].double() - ref[before]).abs() <= tol[before]).all())
        assert bool(((lse[before].double() - rl[before]).abs() <= lt[before]).all())
        assert not bool(torch.isfinite(out[row + at[b]:row + new[b]][..., ::3]).any())
        row += new[b]


@pytest.mark.parametrize("dt", [F32, BF])
def test_bad_pages_and_lengths(sv, dt):
    lens, new = [100, 40, 300, 7, 64], [30, 50, 5, 20, 3]
    c, host = case(6, lens, new, 8, 2, 16, dt)
    ref, tol, rl, _ = reference(c, host, 128 ** -0.5)
    pages = c["k_cache"].shape[0]
    c["page_table"][1, 4] = pages          # tokens 64.. of sequence 1
    c["page_table"][2, 0] = -1             # all of sequence 2
    c["seq_lens"][3] = -5
    c["seq_lens"][4] = c["page_table"].shape[1] * 16 - 2
    out = torch.full_like(c["q"], 7.0)
    out, lse, status = sv.chunk_attn(**c, out=out)
    torch.cuda.synchronize()
    assert status.tolist() == [0, BAD_PAGE, BAD_PAGE, BAD_LENGTH, BAD_LENGTH]
    good = list(range(0, 30)) + list(range(30, 30 + 24))
    assert bool(((out[good].double() - ref[good]).abs() <= tol[good]).all())
    rest = [r for r in range(sum(new)) if r not in good]
    assert bool((out[rest] == 0).all()) and bool((lse[rest] == 0).all())


@pytest.mark.parametrize("dt", [F32, BF])
def test_bad_page_in_a_split_unit(sv, dt):
    c, host = case(7, [9000], [40], 8, 2, 16, dt)
    ref, tol, _, _ = reference(c, host, 128 ** -0.5)
    c["page_table"][0, 9008 // 16] = 1 << 30
    out, lse, status = sv.chunk_attn(**c)
    assert status.tolist() == [BAD_PAGE]
    assert bool(((out[:8].double() - ref[:8]).abs() <= tol[:8]).all())
    assert bool((out[8:] == 0).all()) and bool((lse[8:] == 0).all())


@pytest.mark.parametrize("dt", [F32, BF])
def test_bad_offsets_write_nothing(sv, dt):
    c, host = case(8, [10, 20, 30], [5, 6, 7], 8, 2, 16, dt)
    for offs, want in (([0, 5, 3, 10], [0, BAD_LENGTH, 0]), ([-1, 5, 11, 18], [BAD_LENGTH, 0, 0]),
                       ([0, 5, 11, 19], [0, 0, BAD_LENGTH]),
                       ([0, 1 << 30, 11, 18], [BAD_LENGTH, BAD_LENGTH, 0])):
        c["row_offsets"].copy_(i32(offs))
        out = torch.full_like(c["q"], 7.0)
        out, _, status = sv.chunk_attn(**c, out=out)
        assert status.tolist() == want, offs
        written = set()
        for b in range(3):
            if want[b] == 0:
                written |= set(range(offs[b], offs[b + 1]))
        rest = [r for r in range(18) if r not in written]
        assert bool((out[rest] == 7.0).all()), offs


def test_no_rows_and_no_sequences(sv):
    c, _ = case(9, [10, 20], [0, 0], 8, 2, 16, BF, pad=2)
    out = torch.full_like(c["q"], 7.0)
    out, lse, status = sv.chunk_attn(**c, out=out)
    assert status.tolist() == [0, 0] and bool((out == 7.0).all())
    c["q"] = c["q"][:0]
    out, lse, status = sv.chunk_attn(**c)
    assert status.tolist() == [0, 0] and out.shape == (0, 8, 128)
    c["page_table"], c["seq_lens"] = c["page_table"][:0], c["seq_lens"][:0]
    c["row_offsets"] = c["row_offsets"][:1]
    out, lse, status = sv.chunk_attn(**c)
    assert status.shape == (0,)


@pytest.mark.parametrize("dt", [F32, BF])
def test_captured_with_changing_lengths(sv, dt):
    """Two graphs on one workspace, replayed with other lengths; an eager call in between."""
    shapes = [([400, 0, 1000], [60, 30, 1]), ([3, 900, 200], [1, 0, 90]), ([0, 0, 30], [10, 70, 11])]
    built = [case(20 + i, l, n, 16, 4, 16, dt, pad=0, spare=100, extra=40) for i, (l, n) in
             enumerate(shapes)]
    pages = max(c["k_cache"].shape[0] for c, _ in built)
    width = max(c["page_table"].shape[1] for c, _ in built)
    buf = dict(q=torch.zeros(91, 16, 128, dtype=dt, device="cuda"),
               k_cache=torch.zeros(pages, 16, 4, 128, dtype=dt, device="cuda"),
               v_cache=torch.zeros(pages, 16, 4, 128, dtype=dt, device="cuda"),
               page_table=torch.zeros(3, width, dtype=torch.int32, device="cuda"),
               seq_lens=i32([0] * 3), row_offsets=i32([0] * 4))
    ws = torch.zeros(sv.chunk_attn_workspace_size(91, 3, 16, 4, 128, dt), dtype=torch.uint8,
                     device="cuda")
    s = torch.cuda.Stream()
    graphs, outs = [], []
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(sv.chunk_attn(**buf, workspace=ws))
        graphs.append(g)
    for turn in range(4):
        c, host = built[turn % 3]
        n = sum(host[1])
        buf["q"][:n] = c["q"]
        for k in ("k_cache", "v_cache"):
            buf[k][:c[k].shape[0]] = c[k]
        buf["page_table"].fill_(-1)
        buf["page_table"][:, :c["page_table"].shape[1]] = c["page_table"]
        buf["seq_lens"].copy_(c["seq_lens"])
        buf["row_offsets"].copy_(c["row_offsets"])
        for g in graphs:
            g.replay()
        eager = sv.chunk_attn(**buf)
        torch.cuda.synchronize()
        ref, tol, _, _ = reference(c, host, 128 ** -0.5)
        for out, _, status in outs + [eager]:
            assert status.tolist() == [0, 0, 0]
            assert bool(((out[:n].double() - ref).abs() <= tol).all())


@pytest.mark.parametrize("dt", [F32, BF])
def test_streams(sv, dt):
    """Two streams at once, each with a workspace; a stream argument that is not current."""
    a, ha = case(31, [3000], [500], 16, 4, 16, dt)
    b, hb = case(32, [100, 7000], [300, 1], 8, 2, 32, dt)
    want = [check(sv, a, ha)[0], check(sv, b, hb)[0]]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    wss = [torch.zeros(sv.chunk_attn_workspace_size(c["q"].shape[0], 2, c["q"].shape[1],
                                                    c["k_cache"].shape[2], 128, dt),
                       dtype=torch.uint8, device="cuda") for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(10):
        res = []
        for c, s, ws in zip((a, b), streams, wss):
            res.append(sv.chunk_attn(**c, workspace=ws, stream=s)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(res, want))


@pytest.mark.parametrize("dt", [F32, BF])
def test_streams_without_a_workspace(sv, dt):
    """Calls on two streams that pass no workspace do not meet in one, sizes that grow among them."""
    cs = [case(33 + i, [3000 * (i // 2 + 1), 40], [300 * (i // 2 + 1), 7], 16, 4, 16, dt)
          for i in range(4)]
    want = [sv.chunk_attn(**c)[:2] for c, _ in cs]
    for c, h in cs:
        check(sv, c, h)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        res = [sv.chunk_attn(**c, stream=streams[i % 2])[:2] for i, (c, _) in enumerate(cs)]
        torch.cuda.synchronize()
        for x, y in zip(res, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_offsets_past_32_bits(sv):
    """Pages whose elements lie beyond 2^31, and beyond 2^32 bytes."""
    ps, Hkv, D, pages = 16, 8, 128, 150000
    kc = torch.zeros(pages, ps, Hkv, D, dtype=BF, device="cuda")
    vc = torch.zeros(pages, ps, Hkv, D, dtype=BF, device="cuda")
    c, host = case(41, [500, 30], [20, 100], 32, 8, 16, BF)
    n = c["k_cache"].shape[0]
    kc[pages - n:], vc[pages - n:] = c["k_cache"], c["v_cache"]
    want = check(sv, c, host)[0]
    c["page_table"] = torch.where(c["page_table"] >= 0, c["page_table"] + (pages - n), -1).int()
    c["k_cache"], c["v_cache"] = kc, vc
    got = sv.chunk_attn(**c)[0]
    assert torch.equal(got, want)


def test_the_same_as_a_chain_of_the_tree_attention(sv):
    """A chunk is a chain: both calls see the same tokens."""
    for dt in (F32, BF):
        c, host = case(51, [130, 1000, 0], [33, 33, 33], 16, 4, 16, dt)
        ref, tol, _, _ = reference(c, host, 128 ** -0.5)
        got = check(sv, c, host)[0]
        parent = torch.arange(-1, 32, device="cuda", dtype=torch.int32).repeat(3, 1)
        out, _, status, _, _, _ = sv.tree_mask_attn(
            parent, c["q"].view(3, 33, 16, 128), c["k_cache"], c["v_cache"],
            c["page_table"], c["seq_lens"])
        assert status.tolist() == [0, 0, 0]
        assert bool(((out.view_as(got).double() - got.double()).abs() <= 2 * tol).all())


def test_two_kept_workspaces_do_not_mix(sv):
    """Tree attention and chunk attention without a workspace, in turn (large batches of the
    tree attention count in theirs)."""
    sv.load_library().svf_debug_set_attn_kernel(2)
    try:
        c, host = case(61, [3000] * 3, [33] * 3, 16, 4, 16, BF)
        parent = torch.arange(-1, 32, device="cuda", dtype=torch.int32).repeat(3, 1)
        first = None
        for _ in range(4):
            check(sv, c, host)
            out = sv.tree_mask_attn(parent, c["q"].view(3, 33, 16, 128), c["k_cache"], c["v_cache"],
                                    c["page_table"], c["seq_lens"])
            assert out[2].tolist() == [0, 0, 0]
            first = out[0].clone() if first is None else first
            assert torch.equal(out[0], first)
    finally:
        sv.load_library().svf_debug_set_attn_kernel(0)


@pytest.mark.parametrize("ns", [1, 3000, 20000])
def test_waits_that_run_out(sv, ns):
    """Deadlines that pass: the status says so, and the next call is exact."""
    lib = sv.load_library()
    for lens, new, Hq, Hkv in (([9000], [40], 32, 8), ([0, 500], [1000, 300], 8, 2),
                               ([100] * 9, [1] * 9, 8, 8)):
        c, host = case(71, lens, new, Hq, Hkv, 16, BF)
        want = check(sv, c, host)
        ws = torch.zeros(sv.chunk_attn_workspace_size(c["q"].shape[0], len(lens), Hq, Hkv, 128, BF),
                         dtype=torch.uint8, device="cuda")
        for _ in range(3):
            lib.svf_debug_set_chunk_wait_ns(ns)
            try:
                _, _, status = sv.chunk_attn(**c, workspace=ws)
                torch.cuda.synchronize()
            finally:
                lib.svf_debug_set_chunk_wait_ns(0)
            assert set(status.tolist()) <= {0, TIMEOUT}
            if ns == 1:
                assert TIMEOUT in status.tolist()
            got = check(sv, c, host, workspace=ws)
            assert all(torch.equal(x, y) for x, y in zip(got, want))
