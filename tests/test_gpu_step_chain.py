"""One layer of serving steps made of the library's calls alone: pages and slots
for the step's trees, the q/k/v projection with each request's adapter, the
rotary K/V write, tree attention, the output projection, acceptance, commit and
release, several steps on end, eager and as one captured graph.

The K/V rows that the calls leave in the cache are followed by a plain list per
request: bit for bit after every commit, and as the prefix of an attention in 64
bits (the attention's own parity bar, 2e-2 on values of order 1)."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

HQ, HKV, D, PS = 8, 2, 128, 16
H = HQ * D
B, N, MAX_PAGES, V = 5, 15, 12, 64


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_tree_03_gb300 import build as _b
    _b.build()
    import speculative_decoding_tree_03_gb300 as m
    return m


def randn(g, sigma, *shape):
    return (torch.randn(*shape, generator=g, device="cuda") * sigma).bfloat16()


class Layer:
    def __init__(self, sv, seed, num_pages):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.sv, self.g = sv, g
        O = (HQ + 2 * HKV) * D
        self.wqkv, self.wo = randn(g, H ** -0.5, O, H), randn(g, H ** -0.5, H, H)
        self.a = [randn(g, H ** -0.5, 3, 16, H) for _ in range(2)]
        self.b = [randn(g, 0.25, 3, O, 16), randn(g, 0.25, 3, H, 16)]
        self.ids = torch.tensor([2, -1, 0, 2, 1], **i32)
        self.kc = randn(g, 1.0, num_pages, PS, HKV, D)
        self.vc = randn(g, 1.0, num_pages, PS, HKV, D)
        t = torch.arange(512, dtype=torch.float64, device="cuda")[:, None] * \
            10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
        self.rope = torch.cat([t.cos(), t.sin()], 1).float()
        self.pool = sv.page_pool(num_pages)
        self.table = torch.full((B, MAX_PAGES), -1, **i32)
        self.lens = torch.zeros(B, **i32)
        p = (np.arange(N) - 1) // 2
        p[0] = -1
        self.parent = torch.from_numpy(np.tile(p.astype(np.int32), (B, 1))).cuda()
        self.depth = sv.tree_mask_build(self.parent)[1]
        self.new = torch.full((B,), N, **i32)
        self.bufs = {}

    def rows(self, x, ids, depth, new, rows):
        """Reserve, project, rotate and write the rows of ``x`` [rows, H]."""
        sv, o = self.sv, self.bufs.setdefault(("r", rows), {})
        sv.page_reserve(self.pool, self.table, self.lens, new, PS, rows, depth=depth, outputs=o)
        qkv, _ = sv.lora_proj(x, self.wqkv, self.a[0], self.b[0], ids)
        q, k, v = (t.unflatten(1, (-1, D))
                   for t in qkv.split([HQ * D, HKV * D, HKV * D], 1))
        q, st = sv.rope_kv_write(q, k, v, self.rope, o["positions"], o["slots"], self.kc, self.vc)
        return o, q, k, v, st

    def step(self, x, logits, tokens):
        """One verify step; ``x`` [B, N, H]."""
        sv = self.sv
        o, q, k, v, st = self.rows(x.view(B * N, H), self.ids, self.depth, self.new, B * N)
        att, lse, ast, _, _, _ = sv.tree_mask_attn(self.parent, q.view(B, N, HQ, D), self.kc,
                                                   self.vc, self.table, self.lens)
        y, _ = sv.lora_proj(att.view(B, N, H), self.wo, self.a[1], self.b[1], self.ids)
        acc = sv.spec_accept_greedy(logits, tokens, self.parent)
        com = sv.kv_commit(self.kc, self.vc, self.table, self.lens, acc["path"], acc["accept_len"])
        rel = sv.page_release(self.pool, self.table, self.lens + N, com["new_seq_lens"], PS)
        old = self.lens.clone()
        self.lens.copy_(com["new_seq_lens"])
        return dict(o=o, q=q, k=k, v=v, st=st, att=att, ast=ast, y=y, acc=acc, com=com, rel=rel,
                    old=old)

    def held(self):
        table, lens = self.table.cpu().numpy(), self.lens.cpu().numpy()
        return [table[b, :-(-int(lens[b]) // PS)] for b in range(B)]

    def rows_of(self, cache, b, n):
        pages = torch.from_numpy(self.held()[b].astype(np.int64)).cuda()
        return cache[pages].flatten(0, 1)[:n]


def inputs(g, n):
    out = []
    for _ in range(n):
        x = randn(g, 1.0, B, N, H)
        logits = torch.randn(B, N, V, generator=g, device="cuda")
        # tokens that follow the argmax for a few levels, so that paths are accepted
        tokens = torch.randint(0, V, (B, N), generator=g, device="cuda").int()
        best = logits.argmax(-1).int()
        for c in range(1, N):
            hit = torch.rand(B, generator=g, device="cuda") < 0.6
            tokens[:, c] = torch.where(hit, best[:, (c - 1) // 2], tokens[:, c])
        out.append((x, logits, tokens))
    return out


def attention64(q, k, v, visible):
    """q [HQ, D], k / v [t, HKV, D], visible [t] in 64 bits."""
    k, v = (t.double().repeat_interleave(HQ // HKV, 1) for t in (k, v))
    s = torch.einsum("hd,thd->ht", q.double(), k) / D ** 0.5
    s = s.masked_fill(~visible, float("-inf"))
    return torch.einsum("ht,thd->hd", s.softmax(1), v)


def test_steps_on_end(sv):
    pages = B * 9
    L = Layer(sv, 1, pages)
    # prompts of ragged lengths, one of them empty; rows behind the last are padding
    n = np.array([37, 16, 0, 5, 70], np.int32)
    new = torch.from_numpy(n).cuda()
    rows = int(n.sum()) + 6
    x = randn(L.g, 1.0, rows, H)
    x[int(n.sum()):] = float("nan")
    ids = torch.cat([L.ids.repeat_interleave(new.long()), torch.full((6,), -1, device="cuda").int()])
    o, q, k, v, st = L.rows(x, ids, None, new, rows)
    assert not bool(o["status"].any()) and not bool(st.any())
    L.lens.copy_(new)
    at = o["row_offsets"].tolist()
    store = []
    for b in range(B):
        s = o["slots"][at[b]:at[b + 1]].long()
        store.append([L.kc.flatten(0, 1)[s].clone(), L.vc.flatten(0, 1)[s].clone()])
        assert torch.equal(store[b][1], v[at[b]:at[b + 1]])
    accepted = 0
    for x, logits, tokens in inputs(L.g, 8):
        r = L.step(x, logits, tokens)
        torch.cuda.synchronize()
        for s in (r["o"]["status"], r["st"], r["ast"], r["acc"]["status"], r["com"]["status"],
                  r["rel"]["status"]):
            assert not bool(s.any())
        slots, path = r["o"]["slots"].view(B, N).long(), r["acc"]["path"].cpu().numpy()
        old = r["old"].tolist()
        assert torch.equal(r["o"]["positions"].view(B, N), r["old"][:, None] + L.depth)
        anc = [{j} for j in range(N)]
        for j in range(1, N):
            anc[j] |= anc[(j - 1) // 2]
        for b in range(B):
            # the commit moved rows of the cache: the tree's rows from their definition
            kept = path[b][path[b] >= 0]
            accepted += len(kept) - 1
            k_tree = rotated(r["k"].view(B, N, HKV, D)[b], L.rope[(r["old"][b] + L.depth[b]).long()])
            v_tree = r["v"].reshape(B, N, HKV, D)[b]
            k_all, v_all = torch.cat([store[b][0], k_tree]), torch.cat([store[b][1], v_tree])
            for j in (0, 1, 6, N - 1):
                see = torch.zeros(old[b] + N, dtype=torch.bool, device="cuda")
                see[:old[b]] = True
                see[[old[b] + i for i in anc[j]]] = True
                ref = attention64(r["q"].view(B, N, HQ, D)[b, j], k_all, v_all, see)
                assert float((r["att"][b, j].double() - ref).abs().max()) < 2e-2
            n_now = old[b] + len(kept)
            assert int(L.lens[b]) == n_now
            # the cache now holds the old prefix as it was, then the accepted path
            k_now, v_now = L.rows_of(L.kc, b, n_now), L.rows_of(L.vc, b, n_now)
            assert torch.equal(k_now[:old[b]], store[b][0]) and torch.equal(v_now[:old[b]], store[b][1])
            assert torch.equal(v_now[old[b]:], v_tree[kept])
            # half a step of bf16 and the fp32 roundings of two terms
            d = (k_now[old[b]:].double() - k_tree[kept]).abs()
            assert bool((d <= 2.0 ** -8 * 1.02 * k_tree[kept].abs() + 1e-6).all())
            store[b] = [k_now.clone(), v_now.clone()]
        # every page is held once or free once
        held = np.concatenate(L.held())
        free = L.pool["free"].cpu().numpy()[:int(L.pool["state"][0])]
        assert sorted(np.concatenate([held, free]).tolist()) == list(range(pages))
    assert accepted > B          # paths were accepted, so commits moved rows
    # finished requests give everything back
    sv.page_release(L.pool, L.table, L.lens, torch.zeros_like(L.lens), PS)
    assert int(L.pool["state"][0]) == pages


def rotated(x, cs):
    x, c, s = x.double(), cs.double()[:, None, :D // 2], cs.double()[:, None, D // 2:]
    a, b = x[..., :D // 2], x[..., D // 2:]
    return torch.cat([a * c - b * s, b * c + a * s], -1)


def test_a_request_without_pages_leaves_the_others_alone(sv):
    """The pool runs dry for the last request of the batch: it is flagged by
    every call, writes nothing, and takes nothing from the others."""
    L, full = Layer(sv, 2, B - 1), Layer(sv, 2, 3 * B)
    full.kc[:B - 1], full.vc[:B - 1] = L.kc, L.vc
    (x, logits, tokens), = inputs(L.g, 1)
    r, want = L.step(x, logits, tokens), full.step(x, logits, tokens)
    torch.cuda.synchronize()
    assert r["o"]["status"].tolist() == [0] * (B - 1) + [sv.SVF_DEV_NO_PAGES]
    assert r["ast"].tolist()[B - 1] == sv.SVF_DEV_BAD_PAGE
    assert bool((r["att"][B - 1] == 0).all())
    assert r["com"]["status"].tolist()[B - 1] == sv.SVF_DEV_BAD_PAGE
    assert r["rel"]["status"].tolist()[B - 1] == sv.SVF_DEV_BAD_PAGE
    assert int(L.lens[B - 1]) == 0
    # pages are handed out in the same order: the others' results are the same bits
    for key in ("att", "y"):
        assert torch.equal(r[key][:B - 1], want[key][:B - 1])
    assert torch.equal(L.lens[:B - 1], full.lens[:B - 1])


def test_captured_steps_repeat_eager_ones(sv):
    data = inputs(torch.Generator(device="cuda").manual_seed(9), 6)
    eager, graph = Layer(sv, 3, B * 8), Layer(sv, 3, B * 8)
    graph.kc.copy_(eager.kc)
    graph.vc.copy_(eager.vc)
    x, logits, tokens = (t.clone() for t in data[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.step(x, logits, tokens)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = graph.step(x, logits, tokens)
    want = eager.step(*data[0])
    for i in range(1, 6):
        for t, new in zip((x, logits, tokens), data[i]):
            t.copy_(new)
        g.replay()
        want = eager.step(*data[i])
        torch.cuda.synchronize()
        for key in ("att", "y", "q"):
            assert torch.equal(out[key], want[key]), (i, key)
        assert torch.equal(graph.lens, eager.lens) and torch.equal(graph.table, eager.table)
        assert torch.equal(graph.kc, eager.kc) and torch.equal(graph.vc, eager.vc)
        assert torch.equal(graph.pool["state"], eager.pool["state"])
