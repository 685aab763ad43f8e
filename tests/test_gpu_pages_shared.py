"""Forks, copies of pages and releases of shared pages against a plain model of them."""

import random

import pytest
import torch

pytestmark = pytest.mark.gpu

BAD_PAGE, BAD_LENGTH, NO_PAGES, BAD_ROW = 4, 8, 128, 512


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_tree_03_gb300 import build as _b
    _b.build()
    import speculative_decoding_tree_03_gb300 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    """The pool, the table and the lengths as lists."""

    def __init__(self, pages, B, mp, ps):
        self.n, self.B, self.mp, self.ps = pages, B, mp, ps
        self.free = list(range(pages - 1, -1, -1))
        self.table = [[-1] * mp for _ in range(B)]
        self.lens = [0] * B
        self.shares = [0] * pages

    def fork(self, src, dst):
        F = len(src)
        res = dict(copy_src=[-1] * F, copy_dst=[-1] * F, copy_len=[0] * F, status=[0] * F)
        asked, top = 0, len(self.free)
        ok_row = lambda r: 0 <= r < self.B  # noqa: E731
        for f in range(F):
            s, d = src[f], dst[f]
            if not (ok_row(s) and ok_row(d)) or dst.count(d) > 1 or d in src or s in dst:
                res["status"][f] = BAD_ROW
                continue
            L = self.lens[s]
            if L < 0 or L > self.mp * self.ps:
                res["status"][f] = BAD_LENGTH
                continue
            full, part = divmod(L, self.ps)
            asked += part > 0
            self.table[d] = [-1] * self.mp
            if part and asked > top:
                res["status"][f], self.lens[d] = NO_PAGES, 0
                continue
            self.lens[d] = L
            for i in range(full):
                p = self.table[s][i]
                if 0 <= p < self.n:
                    self.table[d][i] = p
                    self.shares[p] += 1
                else:
                    res["status"][f] = BAD_PAGE
            if part:
                new, old = self.free.pop(), self.table[s][full]
                self.table[d][full] = new
                if 0 <= old < self.n:
                    res["copy_src"][f], res["copy_dst"][f], res["copy_len"][f] = old, new, part
                else:
                    res["status"][f] = BAD_PAGE
        return res

    def release(self, old, keep):
        res = dict(n_released=[0] * self.B, status=[0] * self.B)
        left = {}
        cut = []
        for b in range(self.B):
            if keep[b] < 0 or old[b] < keep[b] or old[b] > self.mp * self.ps:
                res["status"][b] = BAD_LENGTH
                continue
            span = range(-(-keep[b] // self.ps), -(-old[b] // self.ps))
            if any(not 0 <= self.table[b][i] < self.n for i in span):
                res["status"][b] = BAD_PAGE
                continue
            for i in span:
                p = self.table[b][i]
                left[p] = left.get(p, 0) + 1
                cut.append((b, i, p))
        last = {p: b for b, _, p in cut}
        back = []
        for b, i, p in cut:
            if left[p] > self.shares[p] and last[p] == b:
                back.append(p)
                res["n_released"][b] += 1
            self.table[b][i] = -1
        for p, c in left.items():
            self.shares[p] = 0 if c > self.shares[p] else self.shares[p] - c
        self.free += reversed(back)
        return res

    def reserve(self, new):
        for b, n in enumerate(new):
            need = -(-(self.lens[b] + n) // self.ps) - -(-self.lens[b] // self.ps)
            assert need <= len(self.free)
            for i in range(need):
                self.table[b][-(-self.lens[b] // self.ps) + i] = self.free.pop()
            self.lens[b] += n


def device(m):
    free = m.free + [-1] * (m.n - len(m.free))
    return {"pool": {"free": i32(free), "state": i32([len(m.free), 0, 0, 0]),
                     "shares": i32(m.shares)}, "table": i32(m.table), "lens": i32(m.lens)}


def same(d, m):
    torch.cuda.synchronize()
    n = len(m.free)
    assert d["pool"]["state"].tolist() == [n, 0, 0, 0]
    assert d["pool"]["free"][:n].tolist() == m.free
    assert d["pool"]["shares"].tolist() == m.shares
    assert d["table"].tolist() == m.table
    assert d["lens"].tolist() == m.lens


def equal(got, want):
    torch.cuda.synchronize()
    for k, v in want.items():
        assert got[k].tolist() == v, k


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("ps", [1, 16, 50])
def test_a_life_of_forks(sv, seed, ps):
    """Prompts, forks of prompts and of forks, growth, and releases in any order, step by step."""
    r = random.Random(1000 * ps + seed)
    B, mp, pages = 40, 30, 900
    m = Model(pages, B, mp, ps)
    used = list(range(5))
    new = [0] * B
    for b in used:
        new[b] = r.randint(0, 20 * ps)
    m.reserve(new)
    d = device(m)
    for step in range(12):
        idle = [b for b in range(B) if b not in used]
        k = min(len(idle), r.randint(1, 9))
        dst = r.sample(idle, k)
        src = [r.choice(used) for _ in range(k)]
        want = m.fork(src, dst)
        equal(sv.page_fork(d["pool"], d["table"], d["lens"], i32(src), i32(dst), ps), want)
        same(d, m)
        used += dst
        new = [r.randint(0, 2 * ps) if b in used and m.lens[b] + 2 * ps <= mp * ps else 0
               for b in range(B)]
        sv.page_reserve(d["pool"], d["table"], d["lens"], i32(new), ps, sum(new))
        m.reserve(new)
        d["lens"] += i32(new)
        same(d, m)
        old, keep = list(m.lens), list(m.lens)
        for b in r.sample(used, min(len(used), r.randint(0, 6))):
            keep[b] = 0  # finished
            used.remove(b)
        if not used:
            break
        want = m.release(old, keep)
        equal(sv.page_release(d["pool"], d["table"], i32(old), i32(keep), ps), want)
        for b in range(B):
            m.lens[b] = keep[b]
        d["lens"].copy_(i32(keep))
        same(d, m)
    keep = [0] * B
    want = m.release(list(m.lens), keep)
    equal(sv.page_release(d["pool"], d["table"], d["lens"], i32(keep), ps), want)
    m.lens = keep
    d["lens"].zero_()
    same(d, m)
    assert sorted(m.free) == list(range(pages)) and m.shares == [0] * pages


def test_fork_refusals_on_the_device(sv):
    m = Model(50, 10, 6, 4)
    m.reserve([9, 4, 0, 0, 0, 0, 0, 0, 0, 3])
    m.lens[6], m.lens[7] = -1, 25
    d = device(m)
    src = [0, 0, 10, 0, 1, 1, 8, -1, 6, 7, 2, 9]
    dst = [3, 0, 4, -1, 5, 5, 9, 4, 4, 8, 2, 4]
    # 4 is written four times; 0, 2, 8 and 9 are read by one and written by another or the same
    want = m.fork(src, dst)
    assert set(want["status"]) == {BAD_ROW}
    equal(sv.page_fork(d["pool"], d["table"], d["lens"], i32(src), i32(dst), 4), want)
    same(d, m)
    src, dst = [6, 7, 0, 2, 9], [4, 5, 8, 2, 1]
    m2 = m.fork(src, dst)
    assert m2["status"] == [BAD_LENGTH, BAD_LENGTH, 0, BAD_ROW, 0]
    equal(sv.page_fork(d["pool"], d["table"], d["lens"], i32(src), i32(dst), 4), m2)
    same(d, m)


def test_forks_without_pages_are_empty(sv):
    m = Model(12, 9, 5, 4)
    m.reserve([9, 8, 13, 0, 0, 0, 0, 0, 0])
    while len(m.free) > 2:
        m.free.pop()
    d = device(m)
    src, dst = [0, 2, 1, 0, 1, 2], [3, 4, 5, 6, 7, 8]
    want = m.fork(src, dst)
    assert want["status"] == [0, 0, 0, NO_PAGES, 0, NO_PAGES]
    equal(sv.page_fork(d["pool"], d["table"], d["lens"], i32(src), i32(dst), 4), want)
    same(d, m)


def test_bad_pages(sv):
    m = Model(30, 6, 5, 4)
    m.reserve([9, 8, 13, 0, 0, 0])
    m.table[0][1] = 30
    m.table[2][3] = -3
    d = device(m)
    want = m.fork([0, 1, 2], [3, 4, 5])
    assert want["status"] == [BAD_PAGE, 0, BAD_PAGE]
    equal(sv.page_fork(d["pool"], d["table"], d["lens"], i32([0, 1, 2]), i32([3, 4, 5]), 4), want)
    same(d, m)
    old = list(m.lens)
    old[1] = 21
    keep = [0, 0, 0, 0, 4, -1]
    want = m.release(old, keep)
    assert want["status"] == [BAD_PAGE, BAD_LENGTH, BAD_PAGE, BAD_PAGE, 0, BAD_LENGTH]
    equal(sv.page_release(d["pool"], d["table"], i32(old), i32(keep), 4), want)
    same(d, m)


def test_without_shares_a_release_is_page_release(sv):
    r = random.Random(3)
    for B, top in ((1, 40), (3, 2000), (300, 200), (2000, 9)):
        m = Model(B * top, B, top, 3)
        m.reserve([r.randint(0, 3 * top) for _ in range(B)])
        d, e = device(m), device(m)
        del e["pool"]["shares"]
        keep = i32([r.randint(0, L) for L in m.lens])
        a = sv.page_release(d["pool"], d["table"], d["lens"], keep, 3)
        b = sv.page_release(e["pool"], e["table"], e["lens"], keep, 3)
        for k in a:
            assert torch.equal(a[k], b[k])
        assert torch.equal(d["table"], e["table"])
        for k in ("free", "state"):
            assert torch.equal(d["pool"][k], e["pool"][k])
        assert not bool(d["pool"]["shares"].any())


def test_many_holders_leave_at_once(sv):
    """8191 forks of one sequence, the most rows there are; all leave in one call."""
    B, ps = 8192, 16
    m = Model(B + 20, B, 4, ps)
    m.reserve([49] + [0] * (B - 1))
    d = device(m)
    src, dst = i32([0] * (B - 1)), torch.arange(1, B, device="cuda", dtype=torch.int32)
    f = sv.page_fork(d["pool"], d["table"], d["lens"], src, dst, ps)
    torch.cuda.synchronize()
    assert not bool(f["status"].any())
    assert d["pool"]["shares"][d["table"][0, :3].long()].tolist() == [B - 1] * 3
    assert int(d["pool"]["state"][0]) == B + 20 - 4 - (B - 1)
    assert len(set(f["copy_dst"].tolist())) == B - 1
    before = d["table"][0, :3].tolist()
    res = sv.page_release(d["pool"], d["table"], d["lens"], torch.zeros_like(d["lens"]), ps)
    torch.cuda.synchronize()
    assert res["n_released"].tolist() == [1] * (B - 1) + [4]  # the last holder puts them back
    assert not bool(d["pool"]["shares"].any())
    n = int(d["pool"]["state"][0])
    assert n == B + 20 and sorted(d["pool"]["free"].tolist()) == list(range(B + 20))
    assert set(before) <= set(d["pool"]["free"].tolist())


@pytest.mark.parametrize("rows,top", [(60, 2000), (300, 1000)])
def test_long_rows_leave_at_once(sv, rows, top):
    """Releases of 120 and 300 thousand entries (a thread keeps its share, or reads it again), without
    sharing as page_release does them, then of a third of rows and their forks, step by step."""
    ps = 2
    m = Model(rows * top + rows, rows, top, ps)
    m.reserve([top * ps - 1] * rows)
    d, e = device(m), device(m)
    del e["pool"]["shares"]
    keep = torch.zeros_like(d["lens"])
    a = sv.page_release(d["pool"], d["table"], d["lens"], keep, ps)
    b = sv.page_release(e["pool"], e["table"], e["lens"], keep, ps)
    for k in a:
        assert torch.equal(a[k], b[k])
    assert torch.equal(d["table"], e["table"])
    for k in ("free", "state"):
        assert torch.equal(d["pool"][k], e["pool"][k])
    assert not bool(d["pool"]["shares"].any())
    third = rows // 3
    m = Model(rows * top + rows, rows, top, ps)
    m.reserve([top * ps - 1] * third + [0] * (rows - third))
    d = device(m)
    src = torch.arange(third, device="cuda", dtype=torch.int32)
    for i in (1, 2):
        f = sv.page_fork(d["pool"], d["table"], d["lens"], src, src + i * third, ps)
        assert not bool(f["status"].any())
    # the first third leaves what the others hold on to, the rest all but a page, then all
    lens = d["lens"].clone()
    keep = lens.clone()
    keep[:third] = 0
    r = sv.page_release(d["pool"], d["table"], lens, keep, ps)
    assert r["n_released"].tolist() == [1] * third + [0] * (rows - third)  # its own last page
    assert sorted(d["pool"]["shares"].unique().tolist()) == [0, 1]
    lens, keep = keep.clone(), keep.clone()
    keep[third:] = ps
    r = sv.page_release(d["pool"], d["table"], lens, keep, ps)
    assert r["n_released"].tolist() == [0] * third + [1] * third + [top - 1] * third
    r = sv.page_release(d["pool"], d["table"], keep, torch.zeros_like(keep), ps)
    assert r["n_released"].tolist() == [0] * 2 * third + [1] * third
    assert not bool(d["pool"]["shares"].any()) and bool((d["table"] == -1).all())
    assert sorted(d["pool"]["free"].tolist()) == list(range(rows * top + rows))


def test_a_captured_release_of_long_rows(sv):
    """Forks of long rows and their release, replayed: everything is as before each time."""
    B, top, ps = 40, 1500, 4
    m = Model(B * 10 + 8 * top, B, top, ps)
    m.reserve([top * ps - 1] * 5 + [0] * (B - 5))
    d = device(m)
    src = i32([i % 5 for i in range(B - 5)])
    dst = torch.arange(5, B, device="cuda", dtype=torch.int32)
    keep = d["lens"].clone()
    torch.cuda.synchronize()
    before = [d["table"].clone(), d["pool"]["free"].clone(), d["pool"]["state"].clone()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f = sv.page_fork(d["pool"], d["table"], d["lens"], src, dst, ps)
        held = d["lens"].clone()
        r = sv.page_release(d["pool"], d["table"], held, keep, ps)
        d["lens"].copy_(keep)
    for _ in range(3):
        g.replay()
        torch.cuda.synchronize()
        assert not bool(f["status"].any()) and not bool(r["status"].any())
        assert held.tolist() == [top * ps - 1] * B
        assert r["n_released"].tolist() == [0] * 5 + [1] * (B - 5)
        assert not bool(d["pool"]["shares"].any())
        assert torch.equal(d["table"], before[0])
        assert torch.equal(d["pool"]["state"], before[2])
        assert sorted(d["pool"]["free"].tolist()) == sorted(before[1].tolist())


def test_more_released_than_the_stack_holds(sv):
    """Pages given back twice: nothing is written behind the stack."""
    m = Model(6, 3, 4, 2)
    d = device(m)
    guard = torch.full((64,), -9, dtype=torch.int32, device="cuda")
    guard[:6] = d["pool"]["free"]
    d["pool"]["free"] = guard[:6]
    d["table"].copy_(i32([[0, 1, 2, 3], [4, 5, 0, 1], [-1] * 4]))
    res = sv.page_release(d["pool"], d["table"], i32([8, 8, 0]), i32([0, 0, 0]), 2)
    torch.cuda.synchronize()
    assert bool((guard[6:] == -9).all())
    assert int(d["pool"]["state"][0]) == 6 and BAD_PAGE in res["status"].tolist()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layers,pages,ps,Hkv,D", [(1, 7, 16, 8, 128), (5, 40, 16, 2, 64),
                                                   (3, 9, 128, 8, 128), (2, 300, 1, 1, 8),
                                                   (0, 12, 5, 3, 40)])
def test_copy(sv, dt, layers, pages, ps, Hkv, D):
    g = torch.Generator(device="cuda")
    g.manual_seed(pages)
    shape = ((layers,) if layers else ()) + (pages, ps, Hkv, D)
    kc = torch.randn(*shape, generator=g, device="cuda").to(dt)
    vc = torch.randn(*shape, generator=g, device="cuda").to(dt)
    r = random.Random(pages)
    ids = r.sample(range(pages), pages)
    k = (pages - 2) // 2
    # (the last entry copies a page that no other entry uses onto itself)
    src, dst = ids[:k] + [-1, -1, pages, ids[-2]], ids[k:2 * k] + [-1, ids[-1], ids[-1], ids[-2]]
    lens = [r.randint(0, ps) for _ in range(k)] + [0, 1, 1, ps]
    lens[0] = ps
    bad = {k + 1: BAD_PAGE, k + 2: BAD_PAGE}
    if k > 2:
        lens[1], lens[2] = -1, ps + 1
        bad.update({1: BAD_LENGTH, 2: BAD_LENGTH})
    for use_lens in (True, False):
        want = []
        for cache in (kc, vc):
            c = cache.clone()
            for i, (s, d) in enumerate(zip(src, dst)):
                wrong = bad.get(i, 0) & (BAD_PAGE if not use_lens else BAD_PAGE | BAD_LENGTH)
                if s >= 0 and not wrong:
                    n = lens[i] if use_lens else ps
                    c[..., d, :n, :, :] = cache[..., s, :n, :, :]
            want.append(c)
        got = [kc.clone(), vc.clone()]
        st = sv.page_copy(*got, i32(src), i32(dst), i32(lens) if use_lens else None)
        torch.cuda.synchronize()
        exp = [bad.get(i, 0) if use_lens or bad.get(i, 0) == BAD_PAGE else 0 for i in range(len(src))]
        assert st.tolist() == exp
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_copy_in_layers_with_gaps(sv):
    """A layer stride beyond the layer, as in one buffer that holds K and V of each layer."""
    both = torch.randn(4, 2, 20, 16, 2, 64, device="cuda").bfloat16()
    k, v = both[:, 0], both[:, 1]
    want = both.clone()
    want[:, :, 9, :7] = both[:, :, 3, :7]
    sv.page_copy(k, v, i32([3]), i32([9]), i32([7]))
    torch.cuda.synchronize()
    assert torch.equal(both, want)


def test_copy_past_32_bits(sv):
    pages, ps, Hkv, D = 150000, 16, 8, 128
    k = torch.zeros(pages, ps, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[pages - 1], v[pages - 1] = 3.0, 4.0
    sv.page_copy(k, v, i32([pages - 1]), i32([pages - 2]), i32([9]))
    torch.cuda.synchronize()
    assert bool((k[pages - 2, :9] == 3).all()) and bool((k[pages - 2, 9:] == 0).all())
    assert bool((v[pages - 2, :9] == 4).all()) and not bool(k[:pages - 2].any())


def test_captured_steps(sv):
    """Release, fork and copy as one graph: beams that are forked anew every step."""
    m = Model(60, 6, 8, 4)
    m.reserve([21, 10, 0, 0, 0, 0])
    d = device(m)
    kc = torch.randn(2, 60, 4, 2, 64, device="cuda")
    vc = torch.randn(2, 60, 4, 2, 64, device="cuda")
    keep, src, dst = i32([21, 10, 0, 0, 0, 0]), i32([0, 0, 1, 0]), i32([2, 3, 4, 5])
    rel, out = {}, {}
    st = torch.zeros(4, dtype=torch.int32, device="cuda")
    rel["n_released"], rel["status"] = i32([0] * 6), i32([0] * 6)
    for k in ("copy_src", "copy_dst", "copy_len", "status"):
        out[k] = i32([0] * 4)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.page_release(d["pool"], d["table"], d["lens"], keep, 4, outputs=rel)
        sv.page_fork(d["pool"], d["table"], d["lens"], src, dst, 4, outputs=out)
        sv.page_copy(kc, vc, out["copy_src"], out["copy_dst"], out["copy_len"], status=st)
    for choice in ([0, 0, 1, 0], [1, 1, 1, 1], [0, 1, 0, 1]):
        src.copy_(i32(choice))
        torch.cuda.synchronize()
        wk, wv = kc.clone(), vc.clone()
        equal_to = m.release(list(m.lens), keep.tolist())
        f = m.fork(choice, [2, 3, 4, 5])
        for a, b, n in zip(f["copy_src"], f["copy_dst"], f["copy_len"]):
            if a >= 0:
                wk[:, b, :n], wv[:, b, :n] = wk[:, a, :n].clone(), wv[:, a, :n].clone()
        g.replay()
        equal(rel, equal_to)
        equal(out, f)
        same(d, m)
        assert torch.equal(kc, wk) and torch.equal(vc, wv)


def test_no_forks_no_entries(sv):
    m = Model(5, 2, 3, 4)
    d = device(m)
    none = i32([])
    f = sv.page_fork(d["pool"], d["table"], d["lens"], none, none, 4)
    assert f["status"].shape == (0,)
    kc = torch.zeros(5, 4, 1, 8, device="cuda")
    assert sv.page_copy(kc, kc.clone(), none, none).shape == (0,)
    same(d, m)


def test_a_pool_for_forks(sv):
    p = sv.page_pool(9, shared=True)
    assert p["shares"].tolist() == [0] * 9 and "shares" not in sv.page_pool(9)
    plain = sv.page_pool(9)
    with pytest.raises(sv.SpecVerifyError, match="shares"):
        sv.page_fork(plain, i32([[0], [-1]]), i32([1, 0]), i32([0]), i32([1]), 4)
