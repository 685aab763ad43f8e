"""A prompt's way into the cache and out of it again, made of the library's calls: pages for
chunks of prompts, their normed and rotated K/V, chunk attention, forks of the prompts into
samples, decoded tokens of all samples, one tree-verify step on the samples, commit and release.

The K/V that each sequence should hold is followed as a plain list of rows; the rows that the
cache holds in a sequence's pages equal them bit for bit, and every attention output is compared
with a softmax over them in 64 bits: within 2^-8 sum w |v| for the rounding of the weights and
2^-8 |o| for that of the result, one and a quarter times as much for the fp32 sums besides."""

import pytest
import torch

pytestmark = pytest.mark.gpu

HQ, HKV, D, PS, B, MP = 8, 2, 128, 16, 9, 14


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_tree_03_gb300 import build as _b
    _b.build()
    import speculative_decoding_tree_03_gb300 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Layer:
    def __init__(self, sv, seed):
        self.sv, self.g = sv, torch.Generator(device="cuda").manual_seed(seed)
        self.pool = sv.page_pool(80, shared=True)
        self.table = torch.full((B, MP), -1, dtype=torch.int32, device="cuda")
        self.lens = i32([0] * B)
        self.kc = torch.full((1, 80, PS, HKV, D), float("nan"), device="cuda").bfloat16()
        self.vc = self.kc.clone()
        t = torch.arange(400, dtype=torch.float64, device="cuda")[:, None] * \
            10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)
        self.rope = torch.cat([t.cos(), t.sin()], 1).float()
        self.norms = [(1 + 0.2 * self.randn(D)).bfloat16() for _ in range(2)]
        self.axis = (torch.arange(D // 2, device="cuda") % 3).int()
        self.held = [([], []) for _ in range(B)]  # K and V rows that each sequence should hold

    def randn(self, *s):
        return torch.randn(*s, generator=self.g, device="cuda")

    def write(self, new, depth=None, rows=None):
        """``new[b]`` more tokens of every sequence: reserve, norm, rotate, write."""
        sv, rows = self.sv, rows or sum(new)
        o = sv.page_reserve(self.pool, self.table, self.lens, i32(new), PS, rows, depth=depth)
        f = self.randn(rows, (HQ + 2 * HKV) * D).bfloat16()
        q, k, v = (t.unflatten(1, (-1, D)) for t in f.split([HQ * D, HKV * D, HKV * D], 1))
        pos = torch.stack([o["positions"], o["positions"] // 2, o["positions"] // 3]).contiguous()
        q, st = sv.norm_rope_kv_write(q, k, v, *self.norms, self.rope, pos, o["slots"], self.kc[0],
                                      self.vc[0], pair_axis=self.axis)
        assert not bool(st.any()) and not bool(o["status"].any())
        flat = [c[0].flatten(0, 1) for c in (self.kc, self.vc)]
        at = 0
        for b, n in enumerate(new):
            for r in range(at, at + n):
                for kept, cache in zip(self.held[b], flat):
                    kept.append(cache[int(o["slots"][r])].clone())
            at += n
        assert torch.equal(torch.stack([x for b, n in enumerate(new) if n for x in
                                        self.held[b][1][-n:]]), v[:sum(new)])
        return o, q

    def same_cache(self):
        table, lens = self.table.tolist(), self.lens.tolist()
        for b in range(B):
            assert len(self.held[b][0]) == lens[b]
            for kept, cache in zip(self.held[b], (self.kc, self.vc)):
                for t, row in enumerate(kept):
                    assert torch.equal(cache[0, table[b][t // PS], t % PS], row), (b, t)

    def compare(self, got, q, b, seen):
        """got, q [HQ, D] of one row of sequence b that sees the tokens ``seen``."""
        k, v = (torch.stack([x[t] for t in seen]).double().repeat_interleave(HQ // HKV, 1)
                for x in self.held[b])
        w = (torch.einsum("hd,thd->ht", q.double(), k) / D ** 0.5).softmax(1)
        ref, mag = torch.einsum("ht,thd->hd", w, v), torch.einsum("ht,thd->hd", w, v.abs())
        assert bool(((got.double() - ref).abs() <= 1.25 * 2.0 ** -8 * (mag + ref.abs())).all())

    def chunk(self, new):
        o, q = self.write(new)
        out, _, st = self.sv.chunk_attn(q, self.kc[0], self.vc[0], self.table, self.lens,
                                        o["row_offsets"])
        assert not bool(st.any())
        at = 0
        for b, n in enumerate(new):
            L = int(self.lens[b])
            for i in sorted({0, 1, n // 2, n - 1} & set(range(n))):
                self.compare(out[at + i], q[at + i], b, range(L + i + 1))
            at += n
        self.lens += i32(new)

    def fork(self, src, dst):
        f = self.sv.page_fork(self.pool, self.table, self.lens, i32(src), i32(dst), PS)
        st = self.sv.page_copy(self.kc, self.vc, f["copy_src"], f["copy_dst"], f["copy_len"])
        assert not bool(f["status"].any()) and not bool(st.any())
        for s, d in zip(src, dst):
            self.held[d] = tuple(list(x) for x in self.held[s])


def test_prompts_samples_and_a_tree(sv):
    L = Layer(sv, 7)
    L.chunk([70, 33, 0, 0, 0, 0, 0, 0, 0])       # two prompts
    L.same_cache()
    L.chunk([5, 31, 0, 0, 0, 0, 0, 0, 0])        # the rest of them: 75 and 64 tokens
    L.fork([0, 0, 1, 1], [2, 3, 4, 5])           # samples: a shared tail, and none
    L.same_cache()
    assert int(L.pool["shares"].sum()) == 2 * 4 + 2 * 4
    for _ in range(3):                            # decoding all of them, token by token
        L.chunk([1, 1, 1, 1, 1, 1, 0, 0, 0])
    L.same_cache()
    L.fork([2, 5], [6, 7])                        # samples of samples
    L.chunk([1, 0, 2, 0, 17, 1, 1, 4, 0])         # mixed chunks
    L.same_cache()
    # one verify step of a draft tree on every sequence that is there
    N = 7
    parent = i32([[-1, 0, 0, 1, 1, 2, 2]] * B)
    depth = sv.tree_mask_build(parent)[1]
    live = [b for b in range(B) if int(L.lens[b]) > 0]
    before = L.lens.clone()
    new = [N] * B
    o, q = L.write(new, depth=depth, rows=N * B)
    out, _, st, _, _, _ = sv.tree_mask_attn(parent, q.view(B, N, HQ, D), L.kc[0], L.vc[0], L.table,
                                            before)
    assert not bool(st.any())
    path_of = {0: [0], 1: [0, 1], 3: [0, 1, 3], 6: [0, 2, 6]}
    for b in live:
        for node, path in path_of.items():
            seen = list(range(int(before[b]))) + [int(before[b]) + j for j in path]
            L.compare(out[b, node], q.view(B, N, HQ, D)[b, node], b, seen)
    path = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = 0
    path[:, 1], path[:, 2] = 2, 6
    com = sv.kv_commit(L.kc, L.vc, L.table, before, path, i32([2] * B))
    rel = sv.page_release(L.pool, L.table, before + N, com["new_seq_lens"], PS)
    assert not bool(com["status"].any()) and not bool(rel["status"].any())
    for b in range(B):
        n = int(before[b])
        L.held[b] = tuple(x[:n] + [x[n], x[n + 2], x[n + 6]] for x in L.held[b])
    L.lens.copy_(com["new_seq_lens"])
    L.same_cache()                                # nobody's shared pages were touched
    # the requests end, the prompts first: what they shared stays with the samples
    keep = L.lens.clone()
    keep[:2] = 0
    sv.page_release(L.pool, L.table, L.lens, keep, PS)
    L.lens.copy_(keep)
    for b in (0, 1):
        L.held[b] = ([], [])
    L.same_cache()
    L.chunk([0, 0, 1, 1, 1, 1, 1, 1, 1])
    L.same_cache()
    sv.page_release(L.pool, L.table, L.lens, torch.zeros_like(L.lens), PS)
    torch.cuda.synchronize()
    assert int(L.pool["state"][0]) == 80 and not bool(L.pool["shares"].any())
    assert sorted(L.pool["free"].tolist()) == list(range(80)) and bool((L.table == -1).all())


def test_a_captured_decode_step(sv):
    """Reserve, write and chunk attention of one token each as one graph, step after step."""
    L = Layer(sv, 8)
    L.chunk([40, 7, 1, 0, 16, 63, 15, 2, 100])
    one = i32([1] * B)
    f = torch.zeros(B, (HQ + 2 * HKV) * D, device="cuda").bfloat16()
    q, k, v = (t.unflatten(1, (-1, D)) for t in f.split([HQ * D, HKV * D, HKV * D], 1))
    res = {n: torch.zeros(s, dtype=torch.int32, device="cuda") for n, s in
           dict(slots=B, positions=B, row_offsets=B + 1, status=B).items()}
    q_out, st = torch.zeros(B, HQ, D, device="cuda").bfloat16(), i32([0] * B)
    out, ast = torch.zeros_like(q_out), i32([0] * B)
    ws = torch.zeros(sv.chunk_attn_workspace_size(B, B, HQ, HKV, D, out.dtype), dtype=torch.uint8,
                     device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.page_reserve(L.pool, L.table, L.lens, one, PS, B, outputs=res)
        sv.norm_rope_kv_write(q, k, v, *L.norms, L.rope, res["positions"], res["slots"], L.kc[0],
                              L.vc[0], q_out=q_out, status=st)
        sv.chunk_attn(q_out, L.kc[0], L.vc[0], L.table, L.lens, res["row_offsets"], out=out,
                      workspace=ws, status=ast, want_lse=False)
        L.lens += one
    for _ in range(20):
        f.copy_(L.randn(*f.shape))
        g.replay()
        torch.cuda.synchronize()
        assert not bool(st.any()) and not bool(ast.any())
        for b in range(B):
            for kept, c in zip(L.held[b], (L.kc, L.vc)):
                kept.append(c[0].flatten(0, 1)[int(res["slots"][b])].clone())
            L.compare(out[b], q_out[b], b, range(int(L.lens[b])))
    L.same_cache()
