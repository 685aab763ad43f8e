"""The projection with per-request adapters against its definition in 64 bits.

Bound per element, from the kernel's arithmetic (u = 2^-24):
  - the accumulator of the shared product and the adapter columns is rounded
    once per 16-element MMA step (and inside a step: the slack of 16, as for
    the LM head): (H/16 + r/8 + 16) u (sum |x W| + sum |t b|), plus one rounding
    per partial tile that a cluster adds up (8 at most);
  - t is an fp32 sum over H: each of its terms sees at most H/16/8 + 8 + 16
    roundings of its warp's accumulator and of the sums over warps and CTAs,
    and one by the scale: (H/16 + 40) u s sum |x a|, which B_a carries on;
  - t enters as hi + lo, two bf16 values: |t - hi - lo| <= 2^-8 * 2^-8 |t| (half
    a step of the remainder, itself half a step of t);
  - the result is rounded to bf16: half a step, 2^-8 of the value."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BAD_ADAPTER = 256
U = 2.0 ** -24


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_tree_03_gb300 import build as _b
    _b.build()
    import speculative_decoding_tree_03_gb300 as m
    return m


def case(seed, R, H, O, rank, adapters, ids, scales=True):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda s, *z: (torch.randn(*z, generator=g, device="cuda") * s).bfloat16()
    return dict(x=n(1.0, R, H), weight=n(H ** -0.5, O, H), lora_a=n(H ** -0.5, adapters, rank, H),
                lora_b=n(rank ** -0.5, adapters, O, rank),
                ids=torch.as_tensor(ids, dtype=torch.int32, device="cuda"),
                scales=torch.rand(adapters, generator=g, device="cuda") * 2 - 0.5 if scales else None)


def reference(c):
    """y and its error bound in 64 bits, row group by row group."""
    x, w = c["x"].double(), c["weight"].double()
    R, H = x.shape
    G = c["ids"].numel()
    A = c["lora_a"].shape[0]
    rank = c["lora_a"].shape[1]
    y, mag = x @ w.T, x.abs() @ w.abs().T
    steps = (H / 16 + rank / 8 + 24) * U
    extra = torch.zeros_like(y)
    per = R // G
    for a in sorted(set(c["ids"].tolist())):
        rows = (c["ids"] == a).repeat_interleave(per)
        if a < -1 or a >= A:
            y[rows], mag[rows] = 0, 0
        elif a >= 0:
            s = float(c["scales"][a]) if c["scales"] is not None else 1.0
            la, lb = c["lora_a"][a].double(), c["lora_b"][a].double()
            xs = x[rows]
            t = s * (xs @ la.T)
            y[rows] += t @ lb.T
            mag[rows] += t.abs() @ lb.abs().T
            terr = (H / 16 + 40) * U * abs(s) * (xs.abs() @ la.abs().T) + 2.0 ** -16 * t.abs()
            extra[rows] += terr @ lb.abs().T
    bound = steps * mag + extra
    return y, bound + 2.0 ** -8 * (y.abs() + bound)


def check(sv, c, out=None, **kw):
    y, bound = reference(c)
    got, status = sv.lora_proj(**c, out=out, **kw)
    torch.cuda.synchronize()
    bad = (c["ids"] < -1) | (c["ids"] >= c["lora_a"].shape[0])
    assert torch.equal(status, torch.where(bad, BAD_ADAPTER, 0).int())
    err = (got.double() - y).abs()
    worst = float((err / bound.clamp(min=1e-300)).nan_to_num(0).max())
    assert bool((err <= bound).all()), worst
    return got


CASES = [  # groups, rows each, H, O, rank, adapters
    (1, 1, 64, 128, 8, 1),
    (1, 1, 4096, 6144, 16, 1),
    (1, 31, 4096, 4096, 16, 2),
    (3, 5, 8, 7, 8, 2),                # one k step, one tile of 7 columns
    (4, 60, 1000, 515, 64, 3),
    (64, 1, 2048, 1024, 16, 64),       # an adapter per row
    (64, 1, 512, 300, 128, 5),
    (16, 16, 4104, 1029, 24, 9),
    (7, 37, 256, 256, 40, 3),          # 259 rows: two row tiles
    (300, 1, 200, 130, 72, 300),       # two tiles, every row its own adapter
    (64, 31, 512, 20480, 16, 24),      # every CTA takes several tiles
    (2, 700, 136, 5000, 96, 1),
    (1, 4000, 64, 200, 32, 1),
]


@pytest.mark.parametrize("G,per,H,O,rank,adapters", CASES)
def test_matches_definition(sv, G, per, H, O, rank, adapters):
    rng = np.random.default_rng(G * 7 + H)
    ids = rng.integers(-1, adapters, G)
    if G > 1:
        ids[rng.integers(G)] = adapters - 1
    check(sv, case(G + H, G * per, H, O, rank, adapters, ids))


@pytest.mark.parametrize("kind", ["all", "none", "alternate", "far apart", "bad"])
@pytest.mark.parametrize("per", [1, 3, 16, 33])
def test_orders_of_ids(sv, kind, per):
    G = 400 // per
    ids = {"all": np.zeros(G), "none": np.full(G, -1), "alternate": np.arange(G) % 2,
           "far apart": np.where(np.arange(G) % (G // 2 + 1) == 0, 3, -1),
           "bad": np.where(np.arange(G) % 5 == 0, 4, np.arange(G) % 4 - 1)}[kind].astype(np.int32)
    if kind == "bad":
        ids[1], ids[-1] = -2, 2 ** 31 - 1
    check(sv, case(per, G * per, 192, 333, 16, 4, ids))


def test_without_scales_and_three_dims(sv):
    c = case(5, 4 * 15, 256, 100, 16, 3, [0, 2, -1, 2], scales=False)
    y = check(sv, c)
    x3 = c["x"].view(4, 15, 256)
    got, _ = sv.lora_proj(**{**c, "x": x3})
    assert got.shape == (4, 15, 100)
    assert torch.equal(got.view(60, 100), y)


@pytest.mark.parametrize("O,cols", [(96, 104), (97, 101), (130, 133)])
def test_strided_rows_and_what_lies_beside_them(sv, O, cols):
    """x a slice of a wider tensor, out a slice of another, whose other
    elements stay; a workspace full of NaN."""
    R = 70
    c = case(6, R, 128, O, 8, 2, [0, -1, 1, 1, 0, -1, 1])
    wide = torch.full((R, 128 + 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:136] = c["x"]
    c["x"] = wide[:, 8:136]
    buf = torch.full((R + 2, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((sv.lora_proj_workspace_size(R, 8) // 4,), float("nan"), device="cuda")
    out = buf[1:R + 1, 2:2 + O]
    y, bound = reference(c)
    got, _ = sv.lora_proj(**c, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert bool(((got.double() - y).abs() <= bound).all())
    keep = torch.ones_like(buf, dtype=torch.bool)
    keep[1:R + 1, 2:2 + O] = False
    assert bool((buf[keep] == 7.0).all())


@pytest.mark.parametrize("R,H,O", [(64, 512, 256), (600, 256, 40000)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_non_finite_adapters_reach_their_rows_only(sv, value, R, H, O):
    """Infinities and NaN in one adapter's matrices, or in one row of x."""
    ids = np.arange(R) % 4 - 1          # every 16-row window holds every adapter
    c = case(7, R, H, O, 16, 3, ids)
    clean = check(sv, c)
    mine = torch.as_tensor(ids == 1, device="cuda")
    for name, at in (("lora_b", (1, 17, 3)), ("lora_a", (1, 5, 60))):
        d = {**c, name: c[name].clone()}
        d[name][at] = value
        got, _ = sv.lora_proj(**d)
        torch.cuda.synchronize()
        assert torch.equal(got[~mine], clean[~mine]), name
        if name == "lora_b":
            cols = torch.arange(O, device="cuda") != 17
            assert torch.equal(got[mine][:, cols], clean[mine][:, cols])
            t = (c["x"].double() @ c["lora_a"][1].double().T)[mine, 3] * float(c["scales"][1])
            want = t * value
            assert torch.equal(got[mine][:, 17].isnan(), want.isnan())
            if value == value:
                assert torch.equal(got[mine][:, 17].double(), want)
        else:
            assert not bool(got[mine].isfinite().any())
    x = c["x"].clone()
    x[9, 33] = value
    got, _ = sv.lora_proj(**{**c, "x": x})
    rest = torch.arange(R, device="cuda") != 9
    assert torch.equal(got[rest], clean[rest])
    assert not bool(got[9].isfinite().any())


def test_unused_adapters_are_not_read(sv):
    c = case(8, 50, 128, 200, 32, 5, [0, 3, -1, 3, 0])
    clean = check(sv, c)
    for a in (1, 2, 4):
        c["lora_a"][a], c["lora_b"][a], c["scales"][a] = float("nan"), float("nan"), float("nan")
    got, _ = sv.lora_proj(**c)
    assert torch.equal(got, clean)


def test_repeats_bit_for_bit(sv):
    c = case(9, 240, 4096, 6144, 64, 3, [0, 1, 2, -1])
    first, _ = sv.lora_proj(**c)
    for _ in range(20):
        again, _ = sv.lora_proj(**c)
        assert torch.equal(again, first)


def test_empty_batch(sv):
    c = case(10, 4, 64, 32, 8, 1, [0])
    y, st = sv.lora_proj(**{**c, "x": c["x"][:0], "ids": c["ids"][:0]})
    assert y.shape == (0, 32) and st.shape == (0,)


def test_two_streams_with_workspaces_of_their_own(sv):
    cs = [case(20 + i, 64 * 31, 512, 2048, 16, 8, np.arange(64) % 9 - 1) for i in range(2)]
    want = [sv.lora_proj(**c)[0].clone() for c in cs]
    ws = [torch.empty(sv.lora_proj_workspace_size(64 * 31, 16), dtype=torch.uint8, device="cuda")
          for _ in cs]
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, w, o, s in zip(cs, ws, outs, streams):
            sv.lora_proj(**c, out=o, workspace=w, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_capture_and_replay_with_new_contents(sv):
    c = case(30, 64, 1024, 1500, 16, 6, np.arange(64) % 7 - 1)
    out = torch.empty((64, 1500), dtype=torch.bfloat16, device="cuda")
    status = torch.empty(64, dtype=torch.int32, device="cuda")
    ws = torch.empty(sv.lora_proj_workspace_size(64, 16), dtype=torch.uint8, device="cuda")
    sv.lora_proj(**c, out=out, workspace=ws, status=status)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.lora_proj(**c, out=out, workspace=ws, status=status)
    d = case(31, 64, 1024, 1500, 16, 6, (np.arange(64) * 5) % 8 - 1)  # one id is bad
    want, bound = reference(d)
    for k in ("x", "ids", "lora_b", "lora_a", "scales", "weight"):
        c[k].copy_(d[k])
    g.replay()
    torch.cuda.synchronize()
    assert bool(((out.double() - want).abs() <= bound).all())
    assert torch.equal(status, torch.where(d["ids"] >= 6, BAD_ADAPTER, 0).int())


def test_binding_refusals(sv):
    c = case(11, 12, 64, 40, 8, 2, [0, 1, -1])
    bf = torch.bfloat16
    for change in (dict(x=c["x"].float()), dict(x=c["x"][:, :56]), dict(x=c["x"].cpu()),
                   dict(x=c["x"].T), dict(x=c["x"][:11]), dict(weight=c["weight"].float()),
                   dict(weight=c["weight"].T), dict(weight=c["weight"][0]),
                   dict(lora_a=c["lora_a"][:, :, :32]), dict(lora_a=c["lora_a"][0]),
                   dict(lora_b=c["lora_b"][:1]), dict(lora_b=c["lora_b"].transpose(1, 2)),
                   dict(ids=c["ids"].long()), dict(ids=c["ids"].cpu()), dict(ids=c["ids"][:0]),
                   dict(ids=c["ids"][None]), dict(scales=c["scales"].double()),
                   dict(scales=c["scales"][:1]), dict(out=torch.empty(12, 40, device="cuda")),
                   dict(out=torch.empty(12, 39, dtype=bf, device="cuda")),
                   dict(out=torch.empty(40, 12, dtype=bf, device="cuda").T),
                   dict(status=c["ids"][:2]),
                   dict(workspace=torch.empty(12 * 8 * 4 - 1, dtype=torch.uint8, device="cuda")),
                   dict(lora_a=c["lora_a"][:, :4].contiguous(),
                        lora_b=c["lora_b"][:, :, :4].contiguous())):
        with pytest.raises(sv.SpecVerifyError):
            sv.lora_proj(**{**c, **change})


# pairs of CTAs: one tile each, one tile shared by two pairs, several tiles each; one CTA per
# tile of 64 rows
@pytest.mark.parametrize("G,H,O,rank", [(240, 2048, 6144, 16), (256, 4104, 4099, 24),
                                        (520, 256, 40000, 40), (128, 1024, 6144, 16)])
def test_bad_ids_and_non_finite_adapters_at_the_end_of_wide_tiles(sv, G, H, O, rank):
    """The last rows of every 16 have a bad id, an adapter with an infinity, and
    one with a NaN; all others are as without them."""
    adapters = 60
    ids = np.arange(G) * 7 % (adapters - 2)
    want = case(G, G, H, O, rank, adapters, ids)
    y, bound = reference(want)
    ids = ids.copy()
    ids[13::16], ids[14::16], ids[15::16] = adapters, adapters - 2, adapters - 1
    c = dict(want, ids=torch.as_tensor(ids, dtype=torch.int32, device="cuda"))
    c["lora_b"] = want["lora_b"].clone()
    c["lora_b"][adapters - 2, 3::5, rank - 1] = float("inf")
    c["lora_b"][adapters - 1, 3::5, 0] = float("nan")
    got, status = sv.lora_proj(**c)
    row = torch.arange(G, device="cuda") % 16
    assert torch.equal(status, torch.where(row == 13, BAD_ADAPTER, 0).int())
    plain = row < 13
    assert bool(((got.double() - y).abs() <= bound)[plain].all())
    assert bool((got[row == 13] == 0).all())
    hit = torch.zeros(O, dtype=torch.bool, device="cuda")
    hit[3::5] = True
    for r in (14, 15):
        assert not bool(got[row == r][:, hit].isfinite().any())
        assert bool(got[row == r][:, ~hit].isfinite().all())
