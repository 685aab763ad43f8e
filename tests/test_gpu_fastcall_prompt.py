"""The compiled checks of the fork, copy, norm-and-rotary and chunk-attention calls: taken for
calls that are all in order, with the results of the checks in Python, and left for others."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from speculative_decoding_tree_03_gb300 import build as _b
    _b.build()
    import speculative_decoding_tree_03_gb300 as m
    m.load_library()
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def calls(sv):
    """Functions of a stream that return what their call wrote, from the same inputs each time."""
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    qkv, rope = r(33, 6 * 64), torch.rand(100, 64, generator=g, device="cuda")
    q, k, v = (t.unflatten(1, (-1, 64)) for t in qkv.split([256, 64, 64], 1))
    pos = torch.randint(0, 100, (3, 33), generator=g, device="cuda").int()
    axis, slots = (torch.arange(32, device="cuda") % 3).int(), torch.arange(33, device="cuda").int()
    w = [r(64), r(64)]
    cq, ck, cv = r(20, 8, 128), r(9, 16, 2, 128), r(9, 16, 2, 128)

    def pages(stream=None):
        pool = sv.page_pool(20, shared=True)
        table, lens = torch.full((4, 5), -1, dtype=torch.int32, device="cuda"), i32([0, 0, 0, 0])
        torch.cuda.synchronize()
        sv.page_reserve(pool, table, lens, i32([20, 3, 0, 0]), 8, 23)
        lens.copy_(i32([20, 3, 0, 0]))
        o = {n: i32([0, 0]) for n in ("copy_src", "copy_dst", "copy_len", "status")}
        kc, vc = r(3, 20, 8, 1, 64), r(3, 20, 8, 1, 64)
        kc, vc = torch.arange(kc.numel(), device="cuda").view_as(kc).float(), torch.ones_like(vc).float()
        rel, st = {"n_released": i32([0] * 4), "status": i32([0] * 4)}, i32([0, 0])
        torch.cuda.synchronize()
        sv.page_fork(pool, table, lens, i32([0, 1]), i32([2, 3]), 8, outputs=o, stream=stream)
        sv.page_copy(kc, vc, o["copy_src"], o["copy_dst"], o["copy_len"], status=st, stream=stream)
        kept = [table.clone(), lens.clone(), pool["shares"].clone()] if stream is None else []
        sv.page_release(pool, table, lens, i32([20, 3, 0, 0]), 8, outputs=rel, stream=stream)
        torch.cuda.synchronize()
        return [*o.values(), *rel.values(), kc, vc, st, table, pool["state"], pool["shares"],
                pool["free"][:int(pool["state"][0])]], kept

    def write(stream=None, several=True, normed=True):
        kc, vc = torch.zeros(3, 16, 1, 64, device="cuda").bfloat16(), torch.zeros(3, 16, 1, 64, device="cuda").bfloat16()
        out, st = torch.empty(33, 4, 64, device="cuda").bfloat16(), torch.empty(33, device="cuda").int()
        torch.cuda.synchronize()
        sv.norm_rope_kv_write(q, k, v, *(w if normed else (None, None)), rope,
                              pos if several else pos[0], slots, kc, vc, eps=1e-5,
                              pair_axis=axis if several else None, q_out=out, status=st,
                              interleaved=not several, stream=stream)
        torch.cuda.synchronize()
        return [kc, vc, out, st], []

    def attn(stream=None, want_lse=True):
        out, st = torch.zeros_like(cq), i32([0, 0])
        lse = torch.zeros(20, 8, device="cuda") if want_lse else None
        ws = torch.zeros(sv.chunk_attn_workspace_size(20, 2, 8, 2, 128, cq.dtype), dtype=torch.uint8,
                         device="cuda")
        torch.cuda.synchronize()
        sv.chunk_attn(cq, ck, cv, i32([[0, 1, 2, 3], [4, 5, 6, 7]]), i32([40, 9]), i32([0, 3, 20]),
                      sm_scale=0.1, out=out, lse=lse, workspace=ws, status=st, want_lse=want_lse,
                      stream=stream)
        torch.cuda.synchronize()
        return [out, st] + ([lse] if want_lse else []), []

    return [pages, write, lambda stream=None: write(stream, False, False), attn,
            lambda stream=None: attn(stream, False)]


def test_the_same_results_with_and_without(sv, monkeypatch):
    assert sv._fast is not None, "fastcall.cpp is built where the library is"
    fns, side = calls(sv), torch.cuda.Stream()
    names, real = [], sv._fast

    class Spy:
        def __getattr__(self, name):
            def call(*a):
                rc = getattr(real, name)(*a)
                names.append((name, rc))
                return rc
            return call

    monkeypatch.setattr(sv, "_fast", Spy())
    fast = [f() for f in fns]
    on_side = [f(stream=side) for f in fns]
    took = {n for n, rc in names if rc == 0}
    assert {"page_fork", "page_copy", "page_release_shared", "norm_rope_kv_write",
            "chunk_attn"} <= took
    assert all(rc == 0 for n, rc in names if n != "page_reserve")
    monkeypatch.setattr(sv, "_fast", None)
    slow = [f() for f in fns]
    for a, b, c in zip(fast, on_side, slow):
        for x, y, z in zip(a[0], b[0], c[0]):
            assert torch.equal(x, z) and torch.equal(y, z)
        assert all(torch.equal(x, z) for x, z in zip(a[1], c[1]))


def test_what_is_not_in_order_is_left_to_the_binding(sv):
    f = sv._fast
    q, kc = torch.zeros(3, 8, 128, device="cuda"), torch.zeros(4, 16, 2, 128, device="cuda")
    t, l, o = i32([[0, 1]]), i32([0]), i32([0, 3])
    ws, st, out = torch.zeros(10, dtype=torch.uint8, device="cuda"), i32([0]), torch.zeros_like(q)
    good = (q, kc, kc, t, l, o, 0.0, out, None, ws, st, None)
    for i, bad in ((0, q.cpu()), (0, q[:2]), (1, kc.bfloat16()), (2, kc[:3]), (3, t.long()),
                   (4, i32([0, 0])), (5, l), (6, -1.0), (6, float("nan")), (7, None), (8, out),
                   (9, None), (10, None), (11, 5)):
        a = list(good)
        a[i] = bad
        assert f.chunk_attn(*a) is None, i
    assert f.chunk_attn(*good[:11]) is None
    with pytest.raises(sv.SpecVerifyError):   # a workspace that is too small: the library says so
        sv.chunk_attn(q, kc, kc, t, l, o, out=out, workspace=ws, status=st, want_lse=False)
    assert f.page_copy(kc, kc, l, l, l, None, None) is None
    assert f.page_copy(kc, kc[:3], l, l, l, st, None) is None
    pool = {"free": i32([0]), "state": i32([0] * 4)}
    assert f.page_fork(pool, t, l, l, l, 16, {}, None) is None
    assert f.page_release_shared(pool, t, l, l, 16, {}, None) is None
    with pytest.raises(sv.SpecVerifyError):
        sv.chunk_attn(q, kc, kc, t, l, o, lse=torch.zeros(2, 8, device="cuda"), out=out)
