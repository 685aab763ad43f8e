"""Page tables and slot maps on the device against a sequential model of the
pool, value for value, and the order that the results do not depend on."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

NO_PAGES, BAD_LENGTH, BAD_PAGE = 128, 8, 4


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_tree_03_gb300 import build as _b
    _b.build()
    import speculative_decoding_tree_03_gb300 as m
    return m


def up(x, ps):
    return -(-x // ps)


class Model:
    """The pool, one sequence and one page after the other."""

    def __init__(self, table, free, count, ps, num_pages):
        self.table, self.free, self.count = table.copy(), free.copy(), int(count)
        self.ps, self.num_pages = ps, num_pages

    def good(self, p):
        return 0 <= p < self.num_pages

    def reserve(self, lens, new, rows, depth=None):
        ps, B, mp = self.ps, len(lens), self.table.shape[1]
        slots, pos = np.full(rows, -1, np.int32), np.zeros(rows, np.int32)
        status = np.zeros(B, np.int32)
        n_rows = np.maximum(new.astype(np.int64), 0)
        over = n_rows.sum() > rows
        off = np.concatenate([[0], np.cumsum(n_rows)])
        asked, top = 0, self.count
        for b in range(B):
            L, n = int(lens[b]), int(new[b])
            ok = L >= 0 and n >= 0 and L + n <= mp * ps
            r0 = off[b]
            need = up(L + n, ps) - up(L, ps) if ok else 0
            asked += need
            if not ok or (over and n > 0):
                status[b] = BAD_LENGTH
                continue
            pos[r0:r0 + n] = L + (depth[r0:r0 + n] if depth is not None else np.arange(n))
            held = up(L, ps)
            if need and asked > self.count:
                status[b] = NO_PAGES
                self.table[b, held:held + need] = -1
                continue
            for j in range(need):
                top -= 1
                p = self.free[top]
                self.table[b, held + j] = p if self.good(p) else -1
            for i in range(n):
                p = self.table[b, (L + i) // ps]
                if self.good(p):
                    slots[r0 + i] = p * ps + (L + i) % ps
                else:
                    status[b] = BAD_PAGE
        self.count = top
        return slots, pos, np.minimum(off, rows).astype(np.int32), status

    def release(self, old, keep):
        ps, B, mp = self.ps, len(old), self.table.shape[1]
        status, n_rel, out = np.zeros(B, np.int32), np.zeros(B, np.int32), []
        for b in range(B):
            o, k = int(old[b]), int(keep[b])
            if k < 0 or o < k or o > mp * ps:
                status[b] = BAD_LENGTH
                continue
            ids = self.table[b, up(k, ps):up(o, ps)]
            if not all(self.good(p) for p in ids):
                status[b] = BAD_PAGE
                continue
            n_rel[b] = len(ids)
            out += list(ids)
        if self.count + len(out) > self.num_pages:
            status[n_rel > 0] = BAD_PAGE
            return np.zeros(B, np.int32), status
        for b in range(B):
            if n_rel[b]:
                lo = up(int(keep[b]), ps)
                self.table[b, lo:lo + n_rel[b]] = -1
        for p in reversed(out):
            self.free[self.count] = p
            self.count += 1
        return n_rel, status


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def world(seed, B, ps, max_pages, max_len, spare, stray=0):
    """Tables that hold the pages of random lengths, and a pool with the rest."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, max_len + 1, B).astype(np.int32)
    held = np.array([up(int(x), ps) for x in lens])
    num_pages = int(held.sum()) + spare + stray
    perm = rng.permutation(num_pages).astype(np.int32)
    table = np.full((B, max_pages), -7, np.int32)   # entries past the held ones are anything
    at = spare
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    free = np.full(num_pages, -9, np.int32)
    free[:spare] = perm[:spare]
    return rng, lens, table, free, num_pages


def run_reserve(sv, m, lens, new, rows, depth=None):
    """One call against the model; returns the device pool and table."""
    pool = {"free": dev(m.free), "state": dev(np.array([m.count, 0, 0, 0], np.int32))}
    table = dev(m.table)
    free0 = m.free.copy()
    o = {k: torch.full((n,), 12345, dtype=torch.int32, device="cuda")
         for k, n in (("slots", rows), ("positions", rows), ("row_offsets", len(lens) + 1),
                      ("status", len(lens)))}
    sv.page_reserve(pool, table, dev(lens), dev(new), m.ps, rows,
                    depth=None if depth is None else dev(depth), outputs=o)
    slots, pos, off, status = m.reserve(lens, new, rows, depth)
    got = {k: v.cpu().numpy() for k, v in o.items()}
    assert np.array_equal(got["status"], status)
    assert np.array_equal(got["row_offsets"], off)
    assert np.array_equal(got["slots"], slots)
    assert np.array_equal(got["positions"], pos)
    assert np.array_equal(table.cpu().numpy(), m.table)
    assert np.array_equal(pool["free"].cpu().numpy(), free0)
    assert pool["state"].cpu().tolist() == [m.count, 0, 0, 0]
    return pool, table


def run_release(sv, m, pool, table, old, keep):
    r = sv.page_release(pool, table, dev(old), dev(keep), m.ps)
    n_rel, status = m.release(old, keep)
    assert np.array_equal(r["n_released"].cpu().numpy(), n_rel)
    assert np.array_equal(r["status"].cpu().numpy(), status)
    assert np.array_equal(table.cpu().numpy(), m.table)
    assert np.array_equal(pool["free"].cpu().numpy(), m.free)
    assert pool["state"].cpu().tolist() == [m.count, 0, 0, 0]


# B, page size, max_pages, longest prefix, most new tokens, spare pages
SHAPES = [(1, 16, 20, 200, 31, 40), (1, 1, 300, 100, 150, 200), (1, 128, 4000, 900, 400000, 4000),
          (2, 64, 8, 400, 60, 8), (7, 16, 40, 300, 100, 60), (64, 16, 64, 900, 31, 300),
          (257, 32, 30, 500, 64, 900), (3000, 16, 12, 100, 40, 9000), (5, 48, 2000, 50, 60000, 4000)]


@pytest.mark.parametrize("B,ps,max_pages,max_len,most,spare", SHAPES)
@pytest.mark.parametrize("scarce", [False, True])
def test_reserve_and_release_match_the_model(sv, B, ps, max_pages, max_len, most, spare, scarce):
    rng, lens, table, free, n = world(B + ps, B, ps, max_pages, max_len, spare)
    new = np.minimum(rng.integers(0, most + 1, B), max_pages * ps - lens).astype(np.int32)
    new[rng.random(B) < 0.1] = 0
    m = Model(table, free, spare, ps, n)
    if scarce:
        need = sum(up(int(a + b), ps) - up(int(a), ps) for a, b in zip(lens, new))
        m.count = min(spare, need * 2 // 3)
    rows = int(new.sum()) + (0 if scarce else 37)
    depth = rng.integers(0, 9, rows).astype(np.int32) if scarce else None
    before = (m.table.copy(), m.free.copy(), m.count)
    pool, dtable = run_reserve(sv, m, lens, new, rows, depth)
    if not scarce and B < 3000:
        # keep some of the new tokens: the rest goes back
        keep = (lens + rng.integers(0, 1 << 30, B) % (new + 1)).astype(np.int32)
        run_release(sv, m, pool, dtable, lens + new, keep)
        # then everything
        run_release(sv, m, pool, dtable, keep, np.zeros(B, np.int32))
        assert m.count == spare + sum(up(int(x), ps) for x in lens)
    elif not scarce:
        # exactly what was taken: the stack is as before
        run_release(sv, m, pool, dtable, lens + new, lens)
        assert np.array_equal(m.free, before[1]) and m.count == before[2]
    else:
        run_release(sv, m, pool, dtable, lens + new, lens)  # unserved sequences are flagged


def test_bad_lengths_leave_the_others_alone(sv):
    ps, mp = 16, 6
    _, _, table, free, n = world(3, 6, ps, mp, 40, 30)
    lens = np.array([10, -1, 33, 96, 5, 2 ** 31 - 1], np.int32)
    for b, L in enumerate(lens):
        if 0 <= L <= mp * ps:
            table[b, :up(int(L), ps)] = np.arange(up(int(L), ps)) % n
    new = np.array([7, 5, -3, 1, 20, 2 ** 31 - 1], np.int32)   # the last sum passes 31 bits
    m = Model(table, free, 30, ps, n)
    pool, dtable = run_reserve(sv, m, lens, np.where(new > 100, 0, new).astype(np.int32), 50)
    m2 = Model(table, free, 30, ps, n)
    run_reserve(sv, m2, lens, new, 50)                         # too many rows: nothing is taken
    old = np.array([17, 20, 33, 97, -5, 2 ** 31 - 1], np.int32)
    keep = np.array([18, -1, 33, 3, -6, 0], np.int32)
    run_release(sv, m, pool, dtable, old, keep)


def test_zero_rows_and_zero_new_tokens(sv):
    _, lens, table, free, n = world(4, 5, 16, 8, 60, 9)
    m = Model(table, free, 9, 16, n)
    run_reserve(sv, m, lens, np.zeros(5, np.int32), 0)
    run_reserve(sv, m, lens, np.zeros(5, np.int32), 11)
    empty = Model(table, free, 0, 16, n)
    # an empty pool still serves whoever fits into the page it holds
    lens = np.array([1, 16, 15, 30, 0], np.int32)
    empty.table[:, :2] = np.arange(10).reshape(5, 2) % n
    run_reserve(sv, empty, lens, np.array([15, 1, 1, 2, 1], np.int32), 20)


def test_bad_page_ids(sv):
    """A bad id in the partly filled page, or on the stack: that sequence is
    flagged and its rows in that page have no slot."""
    ps = 16
    _, _, table, free, n = world(5, 4, ps, 8, 0, 12)
    lens = np.array([20, 20, 20, 20], np.int32)
    table[:, :2] = np.arange(8).reshape(4, 2) % n
    table[1, 1] = n          # just past the cache
    free[12 - 1 - 4] = -2    # handed out to sequence 2 (two pages each)
    new = np.full(4, 40, np.int32)
    m = Model(table, free, 12, ps, n)
    pool, dtable = run_reserve(sv, m, lens, new, 160)
    # sequence 1's bad page is outside what goes back, sequence 2's is inside
    run_release(sv, m, pool, dtable, lens + new, lens)


def test_giving_back_twice_is_refused(sv):
    rng, lens, table, free, n = world(6, 9, 16, 20, 200, 25)
    m = Model(table, free, 25, 16, n)
    lens[lens < 20] = 20
    for b in range(9):
        m.table[b, :up(int(lens[b]), 16)] %= n
    full = Model(m.table, np.arange(n, dtype=np.int32), n, 16, n)  # every page is free already
    pool = {"free": dev(full.free), "state": dev(np.array([n, 0, 0, 0], np.int32))}
    full.table = np.abs(full.table) % n
    t = dev(full.table)
    run_release(sv, full, pool, t, lens, np.zeros(9, np.int32))
    one = Model(full.table[:1], full.free, n, 16, n)
    run_release(sv, one, {"free": dev(one.free), "state": dev(np.array([n, 0, 0, 0], np.int32))},
                dev(one.table), lens[:1], np.zeros(1, np.int32))


# more pages than the threads of one CTA, or of the cluster, hold at once; the largest batch
@pytest.mark.parametrize("B,max_pages,least", [(1, 9001, 9000), (3, 3001, 2990), (6, 12000, 9000),
                                               (8192, 9, 0)])
@pytest.mark.parametrize("bad", [0, 1, 2])
def test_large_releases(sv, B, max_pages, least, bad):
    """All pages good, one bad id in one sequence, bad ids all over two others."""
    ps = 4
    rng = np.random.default_rng(B + bad)
    held = rng.integers(least, max_pages + 1, B)
    lens = np.maximum(held * ps - rng.integers(0, ps, B), 0).astype(np.int32)
    n = int(held.sum()) + 17
    perm = rng.permutation(n).astype(np.int32)
    table = np.full((B, max_pages), -5, np.int32)
    at = 17
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    keep = np.minimum(rng.integers(0, 3 * ps, B), lens).astype(np.int32)
    if bad == 1:
        table[B // 2, held[B // 2] - 1] = n
    elif bad == 2:
        table[0, 3:held[0]] = -1
        table[B - 1, 3:held[B - 1]] = -1
    free = np.full(n, -9, np.int32)
    free[:17] = perm[:17]
    m = Model(table, free, 17, ps, n)
    pool = {"free": dev(free), "state": dev(np.array([17, 0, 0, 0], np.int32))}
    run_release(sv, m, pool, dev(table), lens, keep)


def test_release_of_more_than_the_cache(sv):
    """The ranges add up to more pages than there are: without the sequence that
    holds a bad id the rest goes back, without that id nothing does."""
    ps, mp, n = 2, 40, 50
    for bad in (True, False):
        table = np.tile(np.arange(mp, dtype=np.int32), (4, 1))
        table[0] = 40 + np.arange(mp) % 10
        if bad:
            table[1, 39] = table[2, 0] = -1
        lens = np.array([10, 80, 80, 60], np.int32)
        keep = np.array([2, 0, 0, 3], np.int32)
        free = np.full(n, -9, np.int32)
        m = Model(table, free, 0, ps, n)
        pool = {"free": dev(free), "state": dev(np.zeros(4, np.int32))}
        run_release(sv, m, pool, dev(table), lens, keep)
        assert (m.count > 0) == bad


@pytest.mark.parametrize("n", [1, 255, 256, 100003])
def test_pool_init(sv, n):
    pool = sv.page_pool(n)
    assert np.array_equal(pool["free"].cpu().numpy(), np.arange(n)[::-1])
    assert pool["state"].cpu().tolist() == [n, 0, 0, 0]


def test_captured_steps_replay(sv):
    """Reserve and release of a growing batch in one graph, replayed: every
    replay continues from the state that the last one left."""
    B, ps, mp, N = 8, 16, 40, 31
    pool = sv.page_pool(B * mp)
    table = torch.full((B, mp), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    new = torch.full((B,), N, dtype=torch.int32, device="cuda")
    keep = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")
    o, r = {}, {}
    end, kept = torch.empty_like(lens), torch.empty_like(lens)

    def step():
        sv.page_reserve(pool, table, lens, new, ps, B * N, outputs=o)
        torch.add(lens, new, out=end)
        torch.add(lens, keep, out=kept)
        sv.page_release(pool, table, end, kept, ps, outputs=r)
        lens.copy_(kept)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    m = Model(np.full((B, mp), -1, np.int32), np.arange(B * mp, dtype=np.int32)[::-1], B * mp, ps,
              B * mp)
    L = np.zeros(B, np.int32)
    k = np.arange(1, B + 1, dtype=np.int32)
    for i in range(40):
        if i > 0:
            g.replay()
        slots, _, _, status = m.reserve(L, np.full(B, N, np.int32), B * N)
        n_rel, _ = m.release(L + N, L + k)
        L = L + k
        if i in (0, 1, 2, 39):
            torch.cuda.synchronize()
            assert np.array_equal(o["slots"].cpu().numpy(), slots)
            assert np.array_equal(o["status"].cpu().numpy(), status) and not status.any()
            assert np.array_equal(r["n_released"].cpu().numpy(), n_rel)
            assert np.array_equal(table.cpu().numpy(), m.table)
            assert np.array_equal(lens.cpu().numpy(), L)
            assert pool["state"].cpu().tolist() == [m.count, 0, 0, 0]


def test_binding_refusals(sv):
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    pool = sv.page_pool(8)
    table = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    for bad in (lambda: sv.page_reserve(pool, table.long(), i, i, 16, 4),
                lambda: sv.page_reserve(pool, table, i[:2], i, 16, 4),
                lambda: sv.page_reserve(pool, table, i, i.long(), 16, 4),
                lambda: sv.page_reserve(pool, table.T, i, i, 16, 4),
                lambda: sv.page_reserve(pool, table, i, i, 0, 4),
                lambda: sv.page_reserve(pool, table, i, i, 16, 4, depth=i),
                lambda: sv.page_reserve(pool, table, i, i, 16, 4, outputs={"slots": i}),
                lambda: sv.page_reserve({"free": pool["free"], "state": i}, table, i, i, 16, 4),
                lambda: sv.page_release(pool, table, i, i[:1], 16),
                lambda: sv.page_release(pool, table[0], i, i, 16)):
        with pytest.raises(sv.SpecVerifyError):
            bad()
