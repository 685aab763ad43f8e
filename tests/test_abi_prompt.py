"""Host-side refusals of the fork, copy, norm-and-rotary and chunk-attention calls: argument
checks return their codes before any CUDA call, and the binding raises before it asks the
library to launch anything."""

import ctypes

import pytest
import torch

P = ctypes.c_void_p(256)   # never dereferenced: every call below returns before using it
Q = ctypes.c_void_p(264)   # not 16-byte aligned

OK, ARG, UNSUPPORTED, WORKSPACE = 0, -1, -2, -4


@pytest.fixture(scope="module")
def sv():
    from speculative_decoding_tree_03_gb300 import build as b
    b.build()
    import speculative_decoding_tree_03_gb300 as m
    m.load_library()
    return m


@pytest.fixture(scope="module")
def lib(sv):
    return sv.load_library()


BAD_POOL = [(dict(B=-1), ARG), (dict(table=None), ARG), (dict(free=None), ARG),
            (dict(state=None), ARG), (dict(shares=None), ARG), (dict(lens=None), ARG),
            (dict(B=8193), UNSUPPORTED), (dict(max_pages=0), UNSUPPORTED),
            (dict(ps=0), UNSUPPORTED), (dict(num_pages=0), UNSUPPORTED),
            (dict(num_pages=1 << 30, ps=1), UNSUPPORTED),
            (dict(num_pages=1 << 27), UNSUPPORTED), (dict(max_pages=1 << 27), UNSUPPORTED)]


def test_page_fork_argument_checks(lib):
    def call(table=P, max_pages=8, ps=16, free=P, state=P, num_pages=64, shares=P, lens=P, B=2,
             src=P, dst=P, F=1, cs=P, cd=P, cl=P, st=P):
        return lib.svf_page_fork(table, max_pages, ps, free, state, num_pages, shares, lens, B, src,
                                 dst, F, cs, cd, cl, st, None)
    for kw, rc in BAD_POOL:
        assert call(**kw) == rc, kw
    for name in ("src", "dst", "cs", "cd", "cl", "st"):
        assert call(**{name: None}) == ARG, name
    assert call(F=-1) == ARG and call(F=8193) == UNSUPPORTED
    assert call(F=0, table=None) == OK


def test_page_release_shared_argument_checks(lib):
    def call(table=P, max_pages=8, ps=16, free=P, state=P, num_pages=64, shares=P, lens=P, keep=P,
             B=2, n=P, st=P):
        return lib.svf_page_release_shared(table, max_pages, ps, free, state, num_pages, shares,
                                           lens, keep, B, n, st, None)
    for kw, rc in BAD_POOL:
        assert call(**kw) == rc, kw
    assert call(keep=None) == ARG and call(n=None) == ARG and call(st=None) == ARG
    assert call(B=0, table=None) == OK


def test_page_copy_argument_checks(lib):
    def call(k=P, v=P, layers=1, stride=0, pages=8, ps=16, src=P, dst=P, lens=None, n=2, Hkv=2,
             D=64, dtype=1, st=P):
        return lib.svf_page_copy(k, v, layers, stride, pages, ps, src, dst, lens, n, Hkv, D, dtype,
                                 st, None)
    for name in ("k", "v", "src", "dst", "st"):
        assert call(**{name: None}) == ARG, name
    assert call(k=Q) == ARG and call(v=Q) == ARG
    for name in ("pages", "ps", "Hkv", "D"):
        assert call(**{name: 0}) == ARG, name
    assert call(n=-1) == ARG and call(layers=-1) == ARG and call(stride=-1) == ARG
    assert call(n=0, k=None) == OK
    assert call(layers=0) == UNSUPPORTED and call(layers=65536, stride=1 << 20) == UNSUPPORTED
    assert call(dtype=2) == UNSUPPORTED
    assert call(Hkv=1, D=4) == UNSUPPORTED          # 8 bytes to a row
    assert call(pages=1 << 27) == UNSUPPORTED
    assert call(layers=2, stride=8 * 16 * 2 * 64 - 8) == ARG   # layers overlap
    assert call(layers=2, stride=8 * 16 * 2 * 64 + 4) == ARG   # not a multiple of 16 bytes


def test_norm_rope_kv_write_argument_checks(lib):
    def call(q=P, k=P, v=P, qs=None, ks=None, vs=None, T=3, Hq=8, Hkv=2, D=128, dtype=1, wq=P, wk=P,
             eps=1e-6, rope=P, rot=128, max_pos=100, pos=P, axes=1, axis=None, slots=P, out=P, kc=P,
             vc=P, ns=64):
        qs = Hq * D if qs is None else qs
        ks = Hkv * D if ks is None else ks
        vs = Hkv * D if vs is None else vs
        return lib.svf_norm_rope_kv_write(q, k, v, qs, ks, vs, T, Hq, Hkv, D, dtype, wq, wk, eps,
                                          rope, rot, max_pos, 0, pos, axes, axis, slots, out, kc, vc,
                                          ns, None, None)
    assert call(T=-1) == ARG
    assert call(T=0, q=None) == OK
    for name in ("q", "k", "v", "rope", "pos", "slots", "out", "kc", "vc"):
        assert call(**{name: None}) == ARG, name
    for name in ("q", "k", "v", "rope", "out", "kc", "vc", "wq", "wk"):
        assert call(**{name: Q}) == ARG, name
    assert call(ns=-1) == ARG and call(max_pos=-1) == ARG
    assert call(eps=-1.0) == ARG and call(eps=float("nan")) == ARG
    assert call(axes=0) == ARG and call(axes=2) == ARG
    assert call(axes=5, axis=P) == UNSUPPORTED
    assert call(dtype=2) == UNSUPPORTED and call(D=264, rot=128) == UNSUPPORTED
    assert call(Hkv=0) == UNSUPPORTED and call(Hq=1025) == UNSUPPORTED
    assert call(rot=8) == UNSUPPORTED and call(rot=144) == UNSUPPORTED
    assert call(qs=8 * 128 - 8) == ARG and call(ks=2 * 128 + 4) == ARG


def test_chunk_attn_argument_checks(lib):
    def call(q=P, k=P, v=P, pages=8, ps=16, table=P, max_pages=4, lens=P, offs=P, B=2, rows=5, Hq=8,
             Hkv=2, D=128, dtype=1, out=P, ws=None, wsb=0, st=P):
        return lib.svf_chunk_attn(q, k, v, pages, ps, table, max_pages, lens, offs, B, rows, Hq, Hkv,
                                  D, dtype, 0.0, out, None, ws, wsb, st, None)
    assert call(B=-1) == ARG and call(rows=-1) == ARG
    assert call(B=0, q=None) == OK
    for name in ("q", "k", "v", "table", "lens", "offs", "out", "st"):
        assert call(**{name: None}) == ARG, name
    for name in ("q", "k", "v", "out", "ws"):
        assert call(**{name: Q}) == ARG, name
    assert call(dtype=2) == UNSUPPORTED and call(D=64) == UNSUPPORTED
    assert call(D=96, dtype=0) == UNSUPPORTED
    assert call(Hq=6, Hkv=4) == UNSUPPORTED and call(Hkv=0) == UNSUPPORTED
    assert call(Hq=130, Hkv=2) == UNSUPPORTED      # 65 heads to one
    assert call(Hq=1025, Hkv=1025) == UNSUPPORTED
    assert call(ps=48) == UNSUPPORTED and call(ps=0) == UNSUPPORTED
    assert call(rows=(1 << 24) + 1) == UNSUPPORTED and call(B=(1 << 20) + 1) == UNSUPPORTED
    assert call(pages=1 << 27) == UNSUPPORTED and call(max_pages=1 << 27) == UNSUPPORTED
    assert call() == WORKSPACE
    need = lib.svf_chunk_attn_workspace_size(5, 2, 8, 2, 128, 1)
    assert need > 0 and call(ws=P, wsb=need - 1) == WORKSPACE
    assert call(dtype=0, ps=7, ws=P, wsb=1) == WORKSPACE   # fp32 takes any page size


def test_chunk_attn_workspace_size(lib):
    size = lib.svf_chunk_attn_workspace_size
    assert size(-1, 1, 8, 2, 128, 1) == 0 and size(4, 1, 8, 2, 64, 1) == 0
    assert size(4, 1, 7, 2, 128, 1) == 0
    assert 0 < size(0, 1, 8, 2, 128, 1) <= size(1, 1, 8, 2, 128, 1) < size(1000, 1, 8, 2, 128, 1)
    assert size(1000, 1, 8, 2, 128, 1) == size(100000, 9, 8, 2, 128, 1)


def test_binding_refuses_cpu_tensors(sv):
    z = torch.zeros
    i = lambda *s: z(*s, dtype=torch.int32)  # noqa: E731
    q, kc = z(3, 8, 128, dtype=torch.bfloat16), z(4, 16, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(sv.SpecVerifyError):
        sv.chunk_attn(q, kc, kc, i(1, 4), i(1), i(2))
    with pytest.raises(sv.SpecVerifyError):
        sv.norm_rope_kv_write(q, q[:, :2], q[:, :2], None, None, z(9, 128), i(3), i(3), kc, kc)
    with pytest.raises(sv.SpecVerifyError):
        sv.page_copy(kc, kc, i(1), i(1))
    with pytest.raises(sv.SpecVerifyError):
        sv.page_fork({"free": i(4), "state": i(4), "shares": i(4)}, i(2, 4), i(2), i(1), i(1), 16)


def test_row_status_has_a_name(sv):
    assert "row" in sv.status_string(sv.SVF_DEV_BAD_ROW)
