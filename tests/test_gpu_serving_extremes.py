"""The serving calls at the largest sizes that they document, and with rows
further apart than 31 bits reach."""

import numpy as np
import pytest
import torch

from test_gpu_lora_proj import case, check, reference, sv  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def leave_the_memory_to_others():
    yield
    torch.cuda.empty_cache()


# rows, rows per id, H, O, rank, adapters
@pytest.mark.parametrize("R,per,H,O,rank,adapters", [
    (1, 1, 65536, 40, 128, 2), (3, 1, 8, 1 << 20, 8, 2), (70, 7, 8, 1 << 20, 16, 5),
    (1 << 17, 1 << 10, 64, 40, 8, 3), (1 << 17, 1, 8, 130, 16, 300), (200, 1, 65536, 8, 16, 9),
    (300, 1, 8, 8, 8, 65536), (1, 1, 8, 1, 8, 1)])
def test_projection(sv, R, per, H, O, rank, adapters):  # noqa: F811
    ids = np.random.default_rng(R).integers(-1, adapters, R // per)
    ids[0] = adapters - 1
    check(sv, case(O, R, H, O, rank, adapters, ids))


@pytest.mark.parametrize("R", [2, 3])
def test_projection_of_rows_far_apart(sv, R):  # noqa: F811
    far = (1 << 31) + 64
    c = case(3, R, 136, 50, 16, 2, [1] * (R - 1) + [0])
    x = torch.empty((R - 1) * far + 136, dtype=torch.bfloat16, device="cuda")
    x = x.as_strided((R, 136), (far, 1))
    x.copy_(c["x"])
    y = torch.empty((R - 1) * far + 50, dtype=torch.bfloat16, device="cuda")
    y = y.as_strided((R, 50), (far, 1))
    want, bound = reference(c)
    got, status = sv.lora_proj(**dict(c, x=x), out=y)
    assert got.data_ptr() == y.data_ptr() and not bool(status.any())
    assert bool(((y.double() - want).abs() <= bound).all())


def test_rotary_write_of_rows_far_apart_into_the_last_slots(sv):  # noqa: F811
    """A quarter turn: (a, b) becomes (-b, a)."""
    far, T, D, slots = (1 << 31) + 8, 3, 16, (1 << 31) - 16
    g = torch.Generator(device="cuda").manual_seed(1)
    base = torch.empty((T - 1) * far + 4 * D, dtype=torch.bfloat16, device="cuda")
    qkv = base.as_strided((T, 4, D), (far, D, 1))
    qkv.copy_(torch.randn(T, 4, D, generator=g, device="cuda").bfloat16())
    q, k, v = qkv[:, :2], qkv[:, 2:3], qkv[:, 3:]
    rope = torch.cat([torch.zeros(5, D // 2, device="cuda"), torch.ones(5, D // 2, device="cuda")], 1)
    kc, vc = (torch.empty((slots // 16, 16, 1, D), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    at = torch.tensor([slots - 1, 0, slots - 2], dtype=torch.int32, device="cuda")
    pos = torch.tensor([4, 0, 1], dtype=torch.int32, device="cuda")
    out, status = sv.rope_kv_write(q, k, v, rope, pos, at, kc, vc)
    turned = lambda x: torch.cat([-x[..., D // 2:], x[..., :D // 2]], -1)  # noqa: E731
    assert not bool(status.any())
    assert torch.equal(out, turned(q))
    assert torch.equal(kc.view(-1, 1, D)[at.long()], turned(k))
    assert torch.equal(vc.view(-1, 1, D)[at.long()], v)


def test_the_most_rows_of_a_rotary_write(sv):  # noqa: F811
    T, D = 1 << 24, 16
    g = torch.Generator(device="cuda").manual_seed(2)
    k = torch.randint(-9, 9, (T, 1, D), generator=g, device="cuda").bfloat16()
    rope = torch.cat([torch.zeros(2, D // 2, device="cuda"), torch.ones(2, D // 2, device="cuda")], 1)
    kc, vc = (torch.zeros((T // 16, 16, 1, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    at = (T - 1 - torch.arange(T, device="cuda")).int()
    pos = (torch.arange(T, device="cuda") % 2).int()
    _, status = sv.rope_kv_write(k[:, :0], k, k, rope, pos, at, kc, vc)
    assert not bool(status.any())
    assert torch.equal(vc.view(T, 1, D).flip(0), k)
    assert torch.equal(kc.view(T, 1, D).flip(0), torch.cat([-k[..., D // 2:], k[..., :D // 2]], -1))


def test_the_most_rows_of_a_reserve(sv):  # noqa: F811
    i32 = dict(dtype=torch.int32, device="cuda")
    ps, rows = 1 << 20, (1 << 30) - 2
    pool, table = sv.page_pool(1025), torch.full((2, 1024), -1, **i32)
    lens, new = torch.tensor([3, 5], **i32), torch.tensor([rows - 7, 4], **i32)
    table[0, 0], table[1, 0] = 1024, 1023     # held; the stack below them is free
    pool["state"][0] = 1023
    pool["free"][:1023] = torch.arange(1022, -1, -1, **i32)
    o = sv.page_reserve(pool, table, lens, new, ps, rows)
    n = rows - 7
    assert o["status"].tolist() == [0, 0] and o["row_offsets"].tolist() == [0, n, rows - 3]
    assert pool["state"].tolist() == [1023 - (-(-(n + 3) // ps) - 1), 0, 0, 0]
    for b in range(0, n, 1 << 26):            # slot = page * ps + offset, page by page
        t = torch.arange(b, min(n, b + (1 << 26)), device="cuda") + 3
        page = table[0, t // ps].long()
        assert torch.equal(o["slots"][b:b + len(t)].long(), page * ps + t % ps)
        assert torch.equal(o["positions"][b:b + len(t)].long(), t)
    assert o["slots"][n:].tolist() == [1023 * ps + 5 + i for i in range(4)] + [-1] * 3
    assert o["positions"][n:].tolist() == [5, 6, 7, 8, 0, 0, 0]
    r = sv.page_release(pool, table, lens + new, lens, ps)
    assert r["status"].tolist() == [0, 0] and pool["state"].tolist() == [1023, 0, 0, 0]
    assert torch.equal(pool["free"][:1023], torch.arange(1022, -1, -1, **i32))
