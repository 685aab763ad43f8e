"""The compiled checks of the short calls: taken for calls that are all in
order, with the results of the checks in Python, and left for all others."""

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


def cases(sv):
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    fresh = lambda: (sv.page_pool(40), torch.full((3, 8), -1, **i32))
    lens, new = torch.tensor([0, 0, 0], **i32), torch.tensor([20, 1, 33], **i32)
    out = lambda **kw: {k: torch.empty(n, **i32) for k, n in kw.items()}
    res = dict(slots=60, positions=60, row_offsets=4, status=3)
    depth = torch.arange(60, **i32)
    qkv, rope = r(54, 6 * 64), torch.rand(100, 64, generator=g, device="cuda")
    q, k, v = (t.unflatten(1, (-1, 64)) for t in qkv.split([256, 64, 64], 1))
    slots, pos = torch.randperm(64, generator=g, device="cuda")[:54].int(), torch.arange(54, **i32)
    x, w, a, b = r(6, 4, 128), r(100, 128), r(2, 8, 128), r(2, 100, 8)
    ids, scales = torch.tensor([0, 1, -1, 1, 0, 0], **i32), torch.rand(2, device="cuda")
    ws = torch.empty(sv.lora_proj_workspace_size(24, 8), dtype=torch.uint8, device="cuda")

    def pages(stream=None, with_depth=False):
        pool, table = fresh()
        o, rel = out(**res), out(n_released=3, status=3)
        sv.page_reserve(pool, table, lens, new, 16, 60, depth=depth if with_depth else None,
                        outputs=o, stream=stream)
        kept = table.clone()
        sv.page_release(pool, table, new, torch.tensor([16, 0, 1], **i32), 16, outputs=rel,
                        stream=stream)
        return [*o.values(), kept, *rel.values(), table, pool["state"]]

    def write(stream=None, interleaved=False):
        kc, vc = torch.zeros(4, 16, 1, 64, device="cuda").bfloat16(), torch.zeros(4, 16, 1, 64, device="cuda").bfloat16()
        qo, st = torch.empty(54, 4, 64, device="cuda").bfloat16(), torch.empty(54, **i32)
        sv.rope_kv_write(q, k, v, rope, pos, slots, kc, vc, q_out=qo, interleaved=interleaved,
                         status=st, stream=stream)
        return [kc, vc, qo, st]

    def proj(stream=None, scaled=True, flat=False):
        xx = x.view(24, 128)[:, :] if flat else x
        y, st = torch.empty(*xx.shape[:-1], 100, device="cuda").bfloat16(), torch.empty(6, **i32)
        sv.lora_proj(xx, w, a, b, ids, scales=scales if scaled else None, out=y, workspace=ws,
                     status=st, stream=stream)
        return [y, st]

    return [pages, lambda stream=None: pages(stream, True), write,
            lambda stream=None: write(stream, True), proj,
            lambda stream=None: proj(stream, False), lambda stream=None: proj(stream, True, True)]


def test_the_same_results_with_and_without(sv, monkeypatch):
    assert sv._fast is not None, "fastcall.cpp is built where the library is"
    fns = cases(sv)
    side = torch.cuda.Stream()
    fast = [f() for f in fns]
    torch.cuda.synchronize()
    on_side = []
    for f in fns:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            on_side.append(f(stream=side))
    torch.cuda.synchronize()
    calls = []

    class Spy:
        def __getattr__(self, name):
            return lambda *a: calls.append((name, getattr(real, name)(*a))) or calls[-1][1]

    real = sv._fast
    monkeypatch.setattr(sv, "_fast", Spy())
    for f in fns:
        f()
    assert len(calls) == 9 and all(rc == 0 for _, rc in calls)   # every call was taken
    monkeypatch.setattr(sv, "_fast", None)
    for f, a, b in zip(fns, fast, on_side):
        slow = f()
        torch.cuda.synchronize()
        for x, y, z in zip(slow, a, b):
            assert torch.equal(x, y) and torch.equal(x, z)


def test_what_is_not_in_order_is_left_to_the_binding(sv):
    f = sv._fast
    i = torch.zeros(3, dtype=torch.int32, device="cuda")
    pool = sv.page_pool(4)
    table = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    o = dict(slots=i[:2].clone(), positions=i[:2].clone(), status=i.clone(),
             row_offsets=torch.zeros(4, dtype=torch.int32, device="cuda"))
    good = [pool, table, i, i, 16, 2, None, o, None]
    assert f.page_reserve(*good) == 0
    for at, bad in ((0, {}), (0, {**pool, "state": i}), (0, None), (1, table.long()),
                    (1, table.cpu()), (1, table[0]), (1, table.T), (1, 3), (2, i[:2]), (2, None),
                    (3, i.float()), (4, -16), (4, 1 << 40), (4, 1.5), (5, 3), (6, i), (6, 5),
                    (7, {}), (7, {**o, "status": i[:1]}), (7, None), (8, 7)):
        assert f.page_reserve(*(good[:at] + [bad] + good[at + 1:])) is None, (at, bad)
    assert f.page_reserve(*good[:5]) is None and f.page_reserve() is None
    # errors of the library itself come back as its code
    assert f.page_reserve(*(good[:4] + [0] + good[5:])) == sv.SVF_ERR_UNSUPPORTED


@pytest.mark.parametrize("fast", [True, False])
def test_what_a_call_allocates_belongs_to_its_stream(sv, monkeypatch, fast):
    """A workspace that the call allocates is not handed out on the current
    stream while the call's own stream still works with it."""
    if not fast:
        monkeypatch.setattr(sv, "_fast", None)
    g = torch.Generator(device="cuda").manual_seed(9)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    x, w, a, b = r(64, 512), r(256, 512), r(3, 16, 512), r(3, 256, 16)
    ids = torch.arange(64, device="cuda", dtype=torch.int32) % 3
    want, _ = sv.lora_proj(x, w, a, b, ids)
    side, need = torch.cuda.Stream(), sv.lora_proj_workspace_size(64, 16)
    outs = [torch.empty_like(want) for _ in range(50)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)   # about 10 ms, in which the calls queue up
    for y in outs:
        sv.lora_proj(x, w, a, b, ids, out=y, stream=side)
    new = sv.lora_proj(x, w, a, b, ids, stream=side)[0]
    mine = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(8)]
    for _ in range(2000):
        for m in mine:
            m.fill_(255)
    torch.cuda.synchronize()
    for y in outs + [new]:
        assert torch.equal(y, want)
    pool = sv.page_pool(20, stream=side)
    side.synchronize()
    assert pool["state"].tolist() == [20, 0, 0, 0]


@pytest.mark.parametrize("fast", [True, False])
def test_no_sequences_and_no_rows(sv, monkeypatch, fast):
    """Calls without sequences or rows leave their outputs as documented."""
    if not fast:
        monkeypatch.setattr(sv, "_fast", None)
    i32 = dict(dtype=torch.int32, device="cuda")
    pool, none = sv.page_pool(4), torch.empty(0, **i32)
    o = {k: torch.full((n,), 77, **i32) for k, n in (("slots", 5), ("positions", 5),
                                                     ("row_offsets", 1), ("status", 0))}
    for given in (o, None):
        got = sv.page_reserve(pool, torch.empty((0, 3), **i32), none, none, 16, 5, outputs=given)
        assert got["slots"].tolist() == [-1] * 5 and got["positions"].tolist() == [0] * 5
        assert got["row_offsets"].tolist() == [0]
    assert sv.page_release(pool, torch.empty((0, 3), **i32), none, none, 16)["status"].numel() == 0
    assert pool["state"].tolist() == [4, 0, 0, 0]
    bf = dict(dtype=torch.bfloat16, device="cuda")
    st = torch.full((4,), 77, **i32)
    y, st = sv.lora_proj(torch.empty(4, 0, 64, **bf), torch.zeros(32, 64, **bf),
                         torch.zeros(2, 8, 64, **bf), torch.zeros(2, 32, 8, **bf),
                         torch.zeros(4, **i32), status=st)
    assert y.shape == (4, 0, 32) and st.tolist() == [0] * 4


@pytest.mark.parametrize("fast", [True, False])
def test_two_threads_at_once(sv, monkeypatch, fast):
    """Two host threads with streams, workspaces and shapes of their own."""
    import threading

    if not fast:
        monkeypatch.setattr(sv, "_fast", None)
    g = torch.Generator(device="cuda").manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
    jobs = []
    for rows, out, rank in ((96, 264, 16), (5, 1000, 72)):
        x, w, a, b = r(rows, 512), r(out, 512), r(3, rank, 512), r(3, out, rank)
        ids = torch.arange(rows, device="cuda", dtype=torch.int32) % 4 - 1
        jobs.append((x, w, a, b, ids, sv.lora_proj(x, w, a, b, ids)[0], torch.cuda.Stream(), []))
    torch.cuda.synchronize()

    def work(x, w, a, b, ids, want, stream, got):
        with torch.cuda.stream(stream):
            ws = torch.empty(sv.lora_proj_workspace_size(x.shape[0], a.shape[1]),
                             dtype=torch.uint8, device="cuda")
            st = torch.empty(ids.shape, dtype=torch.int32, device="cuda")
            for _ in range(60):
                y = torch.empty_like(want)
                sv.lora_proj(x, w, a, b, ids, out=y, workspace=ws, status=st)
                got.append(y)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for *_, want, _, got in jobs:
        assert len(got) == 60 and all(torch.equal(y, want) for y in got)
