"""Host-side refusals of the page, rotary-write and adapter-projection calls:
argument checks return their codes before any CUDA call, and the binding
raises before it asks the library to launch anything."""

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


def _pool_args(**kw):
    a = dict(table=P, max_pages=8, ps=16, free=P, state=P, num_pages=64, l0=P, l1=P, B=2)
    a.update(kw)
    return [a[k] for k in ("table", "max_pages", "ps", "free", "state", "num_pages", "l0", "l1",
                           "B")]


BAD_POOL = [(dict(B=-1), ARG), (dict(table=None), ARG), (dict(free=None), ARG),
            (dict(state=None), ARG), (dict(l0=None), ARG), (dict(l1=None), ARG),
            (dict(B=8193), UNSUPPORTED), (dict(max_pages=0), UNSUPPORTED),
            (dict(ps=0), UNSUPPORTED), (dict(num_pages=0), UNSUPPORTED),
            (dict(num_pages=1 << 30, ps=1), UNSUPPORTED),
            (dict(num_pages=1 << 27, ps=16), UNSUPPORTED),   # slots pass 31 bits
            (dict(max_pages=1 << 27), UNSUPPORTED)]


def test_page_reserve_argument_checks(lib):
    def call(rows=10, slots=P, pos=P, off=P, st=P, **kw):
        return lib.svf_page_reserve(*_pool_args(**kw), rows, None, slots, pos, off, st, None)
    for kw, rc in BAD_POOL:
        assert call(**kw) == rc, kw
    assert call(B=0, table=None) == OK
    assert call(rows=-1) == ARG
    assert call(slots=None) == ARG and call(off=None) == ARG and call(st=None) == ARG
    assert call(rows=(1 << 30)) == UNSUPPORTED


def test_page_release_argument_checks(lib):
    def call(n=P, st=P, **kw):
        return lib.svf_page_release(*_pool_args(**kw), n, st, None)
    for kw, rc in BAD_POOL:
        assert call(**kw) == rc, kw
    assert call(B=0, table=None) == OK
    assert call(n=None) == ARG and call(st=None) == ARG


def test_page_pool_init_argument_checks(lib):
    assert lib.svf_page_pool_init(None, P, 4, None) == ARG
    assert lib.svf_page_pool_init(P, None, 4, None) == ARG
    assert lib.svf_page_pool_init(P, P, -1, None) == ARG
    assert lib.svf_page_pool_init(P, P, 0, None) == UNSUPPORTED
    assert lib.svf_page_pool_init(P, P, 1 << 30, None) == UNSUPPORTED


def test_rope_kv_write_argument_checks(lib):
    def call(q=P, k=P, v=P, qs=None, ks=None, vs=None, T=3, Hq=8, Hkv=2, D=128, dtype=1, rope=P,
             rot=128, max_pos=100, pos=P, slots=P, out=P, kc=P, vc=P, ns=64):
        qs = Hq * D if qs is None else qs
        ks = Hkv * D if ks is None else ks
        vs = Hkv * D if vs is None else vs
        return lib.svf_rope_kv_write(q, k, v, qs, ks, vs, T, Hq, Hkv, D, dtype, rope, rot, max_pos,
                                     0, pos, slots, out, kc, vc, ns, None, None)
    assert call(T=-1) == ARG
    assert call(T=0, q=None) == OK
    for name in ("q", "k", "v", "rope", "pos", "slots", "out", "kc", "vc"):
        assert call(**{name: None}) == ARG, name
    for name in ("q", "k", "v", "rope", "out", "kc", "vc"):
        assert call(**{name: Q}) == ARG, name
    assert call(ns=-1) == ARG and call(max_pos=-1) == ARG
    assert call(dtype=2) == UNSUPPORTED
    assert call(Hkv=0) == UNSUPPORTED and call(Hq=1025) == UNSUPPORTED
    assert call(D=100, rot=96) == UNSUPPORTED           # rows of 200 bytes
    assert call(D=520, rot=128) == UNSUPPORTED
    assert call(rot=24) == UNSUPPORTED                  # bf16: multiples of 16
    assert call(rot=0) == UNSUPPORTED
    assert call(rot=144) == UNSUPPORTED                 # more than D
    assert call(dtype=0, rot=12) == UNSUPPORTED         # fp32: multiples of 8
    assert call(qs=1016) == ARG and call(ks=248) == ARG and call(vs=248) == ARG  # rows overlap
    assert call(qs=1028) == ARG                         # not a multiple of 16 bytes
    assert call(T=(1 << 24) + 1) == UNSUPPORTED


def test_lora_proj_argument_checks(lib):
    def call(x=P, xs=None, w=P, a=P, b=P, ids=P, per=2, R=4, H=64, O=100, n=3, rank=16, y=P,
             ys=None, ws=P, wsb=1 << 20, st=P):
        return lib.svf_lora_proj(x, H if xs is None else xs, w, a, b, None, ids, per, R, H, O, n,
                                 rank, y, O if ys is None else ys, ws, wsb, st, None)
    for kw in (dict(R=-1), dict(x=None), dict(w=None), dict(a=None), dict(b=None), dict(ids=None),
               dict(y=None), dict(st=None), dict(per=0), dict(per=3), dict(x=Q), dict(w=Q),
               dict(a=Q), dict(b=Q), dict(xs=56), dict(xs=68), dict(ys=99)):
        assert call(**kw) == ARG, kw
    assert call(R=0, x=None) == OK
    for kw in (dict(H=60), dict(H=0), dict(H=65544), dict(O=0), dict(n=0), dict(n=65537),
               dict(rank=0), dict(rank=12), dict(rank=136), dict(R=(1 << 17) + 2)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(ws=None), dict(wsb=4 * 16 * 4 - 1), dict(ws=Q)):
        assert call(**kw) == WORKSPACE, kw
    assert lib.svf_lora_proj_workspace_size(4, 16) == 256
    assert lib.svf_lora_proj_workspace_size(0, 16) == 0
    assert lib.svf_lora_proj_workspace_size(1 << 17, 128) == 1 << 26


def test_status_strings(sv):
    assert "pages" in sv.status_string(sv.SVF_DEV_NO_PAGES)
    assert "adapter" in sv.status_string(sv.SVF_DEV_BAD_ADAPTER)


def test_binding_refuses_cpu_tensors(sv):
    i = torch.zeros((2,), dtype=torch.int32)
    f = torch.zeros((2, 4, 8))
    pool = {"free": torch.zeros(8, dtype=torch.int32), "state": torch.zeros(4, dtype=torch.int32)}
    with pytest.raises(sv.SpecVerifyError):
        sv.page_reserve(pool, torch.zeros((2, 4), dtype=torch.int32), i, i, 16, 8)
    with pytest.raises(sv.SpecVerifyError):
        sv.page_release(pool, torch.zeros((2, 4), dtype=torch.int32), i, i, 16)
    with pytest.raises(sv.SpecVerifyError):
        sv.rope_kv_write(f, f, f, torch.zeros((4, 8)), i, i, f[None], f[None])
    with pytest.raises(sv.SpecVerifyError):
        sv.lora_proj(f[0], f[0], f, f, i)
    with pytest.raises(sv.SpecVerifyError):
        sv.page_pool(0)
