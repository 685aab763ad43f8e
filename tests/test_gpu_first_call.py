"""The first calls of a process, made inside a graph capture."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

CODE = """
import torch
import speculative_decoding_tree_03_gb300 as sv
i32 = dict(dtype=torch.int32, device="cuda")
g = torch.Generator(device="cuda").manual_seed(2)
r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()
B, N, ps, mp, H = 4, 31, 16, 8, 256
free, state = torch.arange(64, **i32), torch.tensor([64, 0, 0, 0], **i32)
table, lens = torch.full((B, mp), -1, **i32), torch.zeros(B, **i32)
new, keep = torch.full((B,), N, **i32), torch.full((B,), 3, **i32)
x, w, a, b = r(B * N, H), r(6 * 64, H), r(3, 16, H), r(3, 6 * 64, 16)
ids = torch.tensor([0, -1, 2, 1], **i32)
kc, vc = torch.zeros(64, ps, 1, 64, device="cuda").bfloat16(), torch.zeros(64, ps, 1, 64, device="cuda").bfloat16()
rope = torch.rand(100, 64, generator=g, device="cuda")
pool = {"free": free, "state": state}

def step():
    p = sv.page_reserve(pool, table, lens, new, ps, B * N)
    y, st = sv.lora_proj(x, w, a, b, ids)
    q, k, v = (t.unflatten(1, (-1, 64)) for t in y.split([256, 64, 64], 1))
    qo, st2 = sv.rope_kv_write(q, k, v, rope, p["positions"], p["slots"], kc, vc)
    rel = sv.page_release(pool, table, new, keep, ps)
    return [p["slots"], p["positions"], p["status"], y, st, qo, st2, rel["n_released"], rel["status"]]

first = (table.clone(), free.clone(), state.clone(), kc.clone(), vc.clone())
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    outs = step()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in outs + [table, free, state, kc, vc]]
for t, f in zip((table, free, state, kc, vc), first):
    t.copy_(f)
want = step() + [table, free, state, kc, vc]
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(got, want))
assert want[8].tolist() == [0] * B and bool(want[3].isfinite().all())
"""


def test_first_calls_inside_a_capture():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CODE], capture_output=True, text=True, timeout=300,
                       cwd=root)
    assert r.returncode == 0, r.stderr[-2000:]
