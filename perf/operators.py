"""Measured cases of the operators around the tree-verification step: page bookkeeping of the
paged KV cache on the device, the rotary K/V write of a step's rows, and projections with
per-request low-rank adapters.

Where ``own`` is false, ``run`` computes them in elementary torch operations; where it is true,
it makes the library's calls. Every case names its operator in "op".
"""

import math

import numpy as np
import torch

own = False

DEV_BAD_PAGE, DEV_BAD_LENGTH, DEV_NO_PAGES = 4, 8, 128


def listed():
    return [
        # One request's 31-node binary tree takes its pages before the pass and gives them back:
        # a call whose latency is all that counts.
        {"name": "pages_tree_1x31", "op": "pages", "B": 1, "tokens": 31, "page_size": 16,
         "prefix": 2048, "max_pages": 160, "ragged": False, "depth": True, "short": False},
        # The same for the 70B-shaped serving batch: 64 trees of 31 nodes over 32768-token prefixes.
        {"name": "pages_tree_64x31", "op": "pages", "B": 64, "tokens": 1984, "page_size": 16,
         "prefix": 32768, "max_pages": 2051, "ragged": False, "depth": True, "short": False},
        # Prompts of ragged lengths admitted together, a few of which no longer fit the pool.
        {"name": "pages_prefill_200", "op": "pages", "B": 200, "tokens": 262147, "page_size": 16,
         "prefix": 600, "max_pages": 2051, "ragged": True, "depth": False, "short": True},
        # One token of one request, 8B-shaped heads: the smallest decode step.
        {"name": "rope_token_8b", "op": "rope", "rows": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "rot": 128, "dtype": "bf16", "interleaved": False, "fused": True, "pad": 0,
         "page_size": 16, "max_pos": 8192},
        # fp32 heads of 64 (the small chain's shapes) over a batch, a padded tail behind it.
        {"name": "rope_chain_fp32", "op": "rope", "rows": 500, "Hq": 4, "Hkv": 4, "D": 64,
         "rot": 64, "dtype": "fp32", "interleaved": True, "fused": False, "pad": 12,
         "page_size": 16, "max_pos": 4096},
        # The 70B-shaped batch of trees, rows cut from one fused projection.
        {"name": "rope_tree_70b", "op": "rope", "rows": 1984, "Hq": 64, "Hkv": 8, "D": 128,
         "rot": 128, "dtype": "bf16", "interleaved": False, "fused": True, "pad": 0,
         "page_size": 16, "max_pos": 33024},
        # A chunk of prompt tokens with a partly rotated head.
        {"name": "rope_prefill_8b", "op": "rope", "rows": 16391, "Hq": 32, "Hkv": 8, "D": 128,
         "rot": 64, "dtype": "bf16", "interleaved": False, "fused": True, "pad": 0,
         "page_size": 64, "max_pos": 16896},
        # Decoding one token of one request with its adapter through the 8B-shaped q/k/v projection.
        {"name": "lora_token_8b", "op": "lora", "groups": 1, "per": 1, "H": 4096, "O": 6144,
         "rank": 16, "adapters": 1, "base": 0},
        # 64 requests, one token each, nearly every one with an adapter of its own.
        {"name": "lora_decode_64", "op": "lora", "groups": 64, "per": 1, "H": 4096, "O": 4096,
         "rank": 16, "adapters": 56, "base": 5},
        # Four 60-node EAGLE-2 trees, one request without an adapter.
        {"name": "lora_eagle2_8b", "op": "lora", "groups": 4, "per": 60, "H": 4096, "O": 6144,
         "rank": 64, "adapters": 3, "base": 1},
        # The paged block chains (16 x 16 rows) through an odd-sized output.
        {"name": "lora_chain_odd", "op": "lora", "groups": 16, "per": 16, "H": 4104, "O": 4099,
         "rank": 24, "adapters": 9, "base": 2},
        # The 70B-shaped batch of trees through its q/k/v projection.
        {"name": "lora_tree_70b", "op": "lora", "groups": 64, "per": 31, "H": 8192, "O": 10240,
         "rank": 16, "adapters": 24, "base": 6},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "rope", "lora"])
    if op == "pages":
        ragged = rng.random() < 0.5
        ps = rng.choice([16, 32, 64, 128])
        if ragged:
            B = _log(rng, 2, 256)
            tokens = max(B, _log(rng, 64, 200000))
        else:
            B = _log(rng, 1, 256)
            tokens = B * rng.randint(1, 64)
        prefix = _log(rng, 1, 32768)
        return {"op": op, "B": B, "tokens": tokens, "page_size": ps, "prefix": prefix,
                "max_pages": (prefix + tokens) // ps + 3 if B < 8 else
                             (prefix + 8 * (tokens // B + 1)) // ps + 3,
                "ragged": ragged, "depth": not ragged, "short": rng.random() < 0.3}
    if op == "rope":
        D = rng.choice([64, 128])
        bf = rng.random() < 0.7
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 3, 4, 7, 8])
        rows = max(1, min(_log(rng, 1, 16000), int(3.8e8 // ((Hq + 2 * Hkv) * D * (4 if bf else 8)))))
        return {"op": op, "rows": rows, "Hq": Hq, "Hkv": Hkv, "D": D,
                "rot": rng.choice([D, D, D // 2]), "dtype": "bf16" if bf else "fp32",
                "interleaved": rng.random() < 0.3, "fused": rng.random() < 0.6,
                "pad": rng.randint(0, 9), "page_size": rng.choice([16, 32, 64]),
                "max_pos": _log(rng, 2048, 32768)}
    per = rng.choice([1, 1, rng.randint(2, 64), rng.randint(2, 64)])
    groups = max(1, min(128, _log(rng, 1, 1900) // per))
    base = rng.randint(0, groups // 4)
    return {"op": op, "groups": groups, "per": per, "H": 8 * _log(rng, 32, 1024),
            "O": _log(rng, 256, 10240), "rank": rng.choice([8, 16, 16, 32, 40, 64]),
            "adapters": max(1, rng.randint(1, groups - base) if rng.random() < 0.7 else
                            min(2, groups - base)), "base": base}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _prepare_pages(c, seed):
    rng = np.random.default_rng([int(seed) & 0x7FFFFFFF, 11])
    B, T, ps, mp = c["B"], c["tokens"], c["page_size"], c["max_pages"]
    lens = rng.integers(max(0, c["prefix"] // 2), c["prefix"] + 1, B)
    if c["ragged"]:  # prompts, about one in ten of the requests gets nothing this step
        w = rng.gamma(1.0, 1.0, B) * (rng.random(B) > 0.1)
        new = np.floor(w / max(w.sum(), 1e-9) * (T - T // 50)).astype(np.int64)
    else:
        new = np.full(B, T // B)
    new = np.clip(new, 0, np.maximum(0, mp * ps - lens))
    held = -(-lens // ps)
    need = -(-(lens + new) // ps) - held
    spare = int(need.sum()) * 9 // 10 if c["short"] else int(need.sum()) + 7
    # the cache's size goes by the case; pages of other requests are neither held here nor free
    num_pages = B * (-(-c["prefix"] // ps) + 2) + -(-T // ps) + 8
    perm = rng.permutation(num_pages).astype(np.int32)
    table = np.full((B, mp), -1, np.int32)
    own_pages, at = perm[spare:], 0
    for b in range(B):
        table[b, :held[b]] = own_pages[at:at + held[b]]
        at += held[b]
    free = np.full(num_pages, -1, np.int32)
    free[:spare] = perm[:spare]
    state = np.zeros(4, np.int32)
    state[0] = spare
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    depth = None
    if c["depth"]:  # binary trees: node i at depth floor(log2(i + 1))
        n = T // B
        depth = d(np.tile(np.floor(np.log2(np.arange(n) + 1)).astype(np.int32), B))
    lens, new = lens.astype(np.int32), new.astype(np.int32)
    return {"c": c, "num_pages": num_pages, "pool": {"free": d(free), "state": d(state)},
            "table": d(table), "lens": d(lens), "new": d(new), "ends": d(lens + new),
            "depth": depth, "out": {}, "rel": {}}


def rope_table(max_pos, rot):
    """cos in the first half of a row, sin in the second; angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _prepare_rope(c, seed):
    g = _gen(seed)
    T, Hq, Hkv, D, ps = c["rows"], c["Hq"], c["Hkv"], c["D"], c["page_size"]
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    n = T + c["pad"]
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    if c["fused"]:
        f = r(n, (Hq + 2 * Hkv) * D)
        q, k, v = (x.unflatten(1, (-1, D)) for x in f.split([Hq * D, Hkv * D, Hkv * D], 1))
    else:
        q, k, v = r(n, Hq, D), r(n, Hkv, D), r(n, Hkv, D)
    pages = -(-T // ps) + 3
    perm = torch.randperm(pages, generator=g, device="cuda")
    t = torch.arange(n, device="cuda")
    slots = (perm[t.clamp(max=T - 1) // ps] * ps + t % ps).to(torch.int32)
    pos = torch.randint(0, c["max_pos"], (n,), generator=g, device="cuda").to(torch.int32)
    slots[T:] = -1  # rows behind the last sequence
    pos[T:] = 0
    return {"c": c, "q": q, "k": k, "v": v, "rope": rope_table(c["max_pos"], c["rot"]),
            "pos": pos, "slots": slots, "k_cache": r(pages, ps, Hkv, D),
            "v_cache": r(pages, ps, Hkv, D), "q_out": torch.zeros(n, Hq, D, dtype=dt, device="cuda"),
            "status": torch.zeros(n, dtype=torch.int32, device="cuda")}


def _prepare_lora(c, seed):
    g = _gen(seed)
    G, H, O, r, A = c["groups"], c["H"], c["O"], c["rank"], c["adapters"]

    def n(sigma, *s):
        return (torch.randn(*s, generator=g, device="cuda") * sigma).to(torch.bfloat16)

    # requests take the adapters in turn, in an order of their own; `base` of them have none
    ids = torch.arange(G, device="cuda") % A
    if c["base"]:
        ids[G - c["base"]:] = -1
    ids = ids[torch.randperm(G, generator=g, device="cuda")].to(torch.int32)
    return {"c": c, "x": n(1.0, G * c["per"], H), "w": n(H ** -0.5, O, H),
            "a": n(H ** -0.5, A, r, H), "b": n(0.3 * r ** -0.5, A, O, r), "ids": ids,
            "scales": 0.5 + 1.5 * torch.rand(A, generator=g, device="cuda"), "ws": None,
            "y": torch.empty(G * c["per"], O, dtype=torch.bfloat16, device="cuda"),
            "status": torch.zeros(G, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    return {"pages": _prepare_pages, "rope": _prepare_rope, "lora": _prepare_lora}[case["op"]](
        case, seed)


# ------------------------------------------------------------------ plain forms

def _ceil(x, ps):
    return (x + ps - 1) // ps


def _plain_reserve(s):
    """Pages for every sequence's new tokens from the top of the free stack, and their slots."""
    c, table, free, state = s["c"], s["table"], s["pool"]["free"], s["pool"]["state"]
    ps, T = c["page_size"], c["tokens"]
    L, n = s["lens"].long(), s["new"].long()
    held = _ceil(L, ps)
    need = _ceil(L + n, ps) - held
    incl = need.cumsum(0)
    F = state[0].long()
    served = (need == 0) | (incl <= F)
    ends = n.cumsum(0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends]).int()
    status = torch.where(served, 0, DEV_NO_PAGES).int()
    col = torch.arange(table.shape[1], device=table.device)
    rank = (incl - need - held)[:, None] + col
    fresh = (col >= held[:, None]) & (col < (held + need)[:, None])
    pages = free.long()[(F - 1 - rank).clamp(0, free.numel() - 1)]
    pages = torch.where(served[:, None], pages, -1).int()
    table.copy_(torch.where(fresh, pages, table))
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(ends, t, right=True).clamp(max=len(n) - 1)
    at = L[b] + t - offsets[b]
    live = t < ends[-1]
    page = table[b, torch.where(live, at // ps, 0)].long()
    slots = torch.where(live & served[b], page * ps + at % ps, -1).int()
    pos = L[b] + s["depth"] if s["depth"] is not None else at
    pos = torch.where(live, pos, 0).int()
    state[0] -= torch.where(incl <= F, incl, 0).amax().int()
    return {"slots": slots, "positions": pos, "row_offsets": offsets, "status": status}


def _plain_release(s):
    """The pages of the tokens past each sequence's kept length go back onto the stack."""
    c, table, free, state = s["c"], s["table"], s["pool"]["free"], s["pool"]["state"]
    ps = c["page_size"]
    lo, hi = _ceil(s["lens"].long(), ps), _ceil(s["ends"].long(), ps)
    col = torch.arange(table.shape[1], device=table.device)
    cut = (col >= lo[:, None]) & (col < hi[:, None])
    bad = (cut & ((table < 0) | (table >= s["num_pages"]))).any(1)
    cut &= ~bad[:, None]
    n = cut.sum(1)
    rank = (n.cumsum(0) - n - lo)[:, None] + col
    total = n.sum()
    to = torch.where(cut, state[0].long() + total - 1 - rank, free.numel()).reshape(-1)
    grown = torch.cat([free, free[:1]])
    grown[to] = table.reshape(-1)
    free.copy_(grown[:-1])
    table.masked_fill_(cut, -1)
    state[0] += total.int()
    return {"n_released": n.int(), "status": torch.where(bad, DEV_BAD_PAGE, 0).int()}


def _rotated(x, cs, rot, interleaved):
    cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    x = x.float()
    y = x.clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (
        slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., first], x[..., second]
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y


def _plain_rope(s):
    c = s["c"]
    keep = s["slots"] >= 0
    slots, cs = s["slots"][keep].long(), s["rope"][s["pos"][keep].long()]
    dt = s["q"].dtype
    s["q_out"][keep] = _rotated(s["q"][keep], cs, c["rot"], c["interleaved"]).to(dt)
    s["k_cache"].flatten(0, 1)[slots] = _rotated(s["k"][keep], cs, c["rot"],
                                                 c["interleaved"]).to(dt)
    s["v_cache"].flatten(0, 1)[slots] = s["v"][keep]
    s["status"].zero_()


def _plain_lora(s):
    x, A, r = s["x"].float(), s["c"]["adapters"], s["c"]["rank"]
    ids = s["ids"].long().repeat_interleave(s["c"]["per"], output_size=x.shape[0])
    t = (x @ s["a"].float().flatten(0, 1).T).unflatten(1, (A, r))  # every adapter's, then its own
    mine = ids[:, None] == torch.arange(A, device=x.device)
    t = (t * (mine * s["scales"])[:, :, None]).flatten(1)
    y = x @ s["w"].float().T + t @ s["b"].float().transpose(1, 2).flatten(0, 1)
    s["y"].copy_(y)
    s["status"].zero_()


def run(state):
    s, op = state, state["c"]["op"]
    if own:
        import speculative_decoding_tree_03_gb300 as sv
    if op == "pages":
        if own:
            res = sv.page_reserve(s["pool"], s["table"], s["lens"], s["new"],
                                  s["c"]["page_size"], s["c"]["tokens"], depth=s["depth"],
                                  outputs=s["out"])
            rel = sv.page_release(s["pool"], s["table"], s["ends"], s["lens"],
                                  s["c"]["page_size"], outputs=s["rel"])
        else:
            res, rel = _plain_reserve(s), _plain_release(s)
        return {"slots": res["slots"], "positions": res["positions"],
                "row_offsets": res["row_offsets"], "status": res["status"],
                "n_released": rel["n_released"], "rel_status": rel["status"],
                "table": s["table"], "free": s["pool"]["free"], "state": s["pool"]["state"]}
    if op == "rope":
        if own:
            sv.rope_kv_write(s["q"], s["k"], s["v"], s["rope"], s["pos"], s["slots"],
                             s["k_cache"], s["v_cache"], q_out=s["q_out"],
                             interleaved=s["c"]["interleaved"], status=s["status"])
        else:
            _plain_rope(s)
        return {"q_out": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"],
                "status": s["status"]}
    if own:
        if s["ws"] is None:  # the workspace that a serving program keeps
            need = sv.lora_proj_workspace_size(s["x"].shape[0], s["c"]["rank"])
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        sv.lora_proj(s["x"], s["w"], s["a"], s["b"], s["ids"], scales=s["scales"], out=s["y"],
                     workspace=s["ws"], status=s["status"])
    else:
        _plain_lora(s)
    return {"y": s["y"], "status": s["status"]}


# ------------------------------------------------------------------ floors

def work(case):
    c = case
    if c["op"] == "pages":
        # lengths, one id per page (out of the stack and into the table, and back), slot and position per row
        pages = c["tokens"] / c["page_size"] + c["B"] / 2
        return {"bytes": 20 * c["B"] + 16 * pages + (12 if c["depth"] else 8) * c["tokens"], "flops": 0}
    if c["op"] == "rope":
        e = 2 if c["dtype"] == "bf16" else 4
        rows = c["rows"]
        return {"bytes": rows * (2 * (c["Hq"] + 2 * c["Hkv"]) * c["D"] * e + 12) +
                         min(rows, c["max_pos"]) * c["rot"] * 4,
                "flops": rows * (c["Hq"] + c["Hkv"]) * c["rot"] * 3}
    R, H, O, r = c["groups"] * c["per"], c["H"], c["O"], c["rank"]
    with_one = c["groups"] - c["base"]
    used = min(c["adapters"], with_one)
    return {"bytes": 2 * (R * H + O * H + used * r * (H + O) + R * O) + 8 * c["groups"] + 4 * used,
            "flops": 2 * R * H * O + 2 * with_one * c["per"] * r * (H + O)}


# ------------------------------------------------------------------ 64 bits

def _exact_pages(c, s):
    """The definition, one sequence and one token after the other."""
    ps, T, B = c["page_size"], c["tokens"], c["B"]
    host = lambda t: t.cpu().numpy().astype(np.int64)  # noqa: E731
    lens, new, table, free = host(s["lens"]), host(s["new"]), host(s["table"]), host(s["pool"]["free"])
    depth = host(s["depth"]) if s["depth"] is not None else None
    F = int(s["pool"]["state"][0])
    slots, pos = np.full(T, -1, np.int64), np.zeros(T, np.int64)
    off, status, rel_status, n_rel = [0], np.zeros(B, np.int64), np.zeros(B, np.int64), np.zeros(B, np.int64)
    asked, top = 0, F
    for b in range(B):
        L, n, at = int(lens[b]), int(new[b]), off[-1]
        first, end = -(-L // ps), -(-(L + n) // ps)
        asked += end - first
        if end > first and asked > F:
            status[b] = DEV_NO_PAGES
        else:
            for i in range(first, end):
                top -= 1
                table[b, i] = free[top]
            i = np.arange(L, L + n)
            slots[at:at + n] = table[b, i // ps] * ps + i % ps
        pos[at:at + n] = L + (depth[at:at + n] if depth is not None else np.arange(n))
        off.append(at + n)
    for b in reversed(range(B)):  # the stack gets back what was taken last first
        first, end = -(-int(lens[b]) // ps), -(-int(lens[b] + new[b]) // ps)
        if status[b]:  # it holds no pages there
            rel_status[b] = DEV_BAD_PAGE
            continue
        n_rel[b] = end - first
        for i in reversed(range(first, end)):
            free[top] = table[b, i]
            table[b, i] = -1
            top += 1
    as_int = lambda v: torch.from_numpy(np.asarray(v).astype(np.int32))  # noqa: E731
    return {"slots": as_int(slots), "positions": as_int(pos), "row_offsets": as_int(off),
            "status": as_int(status), "n_released": as_int(n_rel), "rel_status": as_int(rel_status),
            "table": as_int(table), "free": as_int(free), "state": as_int([top, 0, 0, 0])}


def _exact_rope(c, s):
    """Each pair of a head as a complex number, turned by the table's angle."""
    T, rot = c["rows"], c["rot"]
    turn = torch.complex(*s["rope"][s["pos"][:T].long()].double().chunk(2, 1))[:, None]

    def turned(x):
        x = x[:T].double()
        head = x[..., :rot]
        pairs = head.unflatten(-1, (rot // 2, 2)) if c["interleaved"] else \
            head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, x[..., rot:]], -1)

    q, k, v = (s[n].double() for n in ("q_out", "k_cache", "v_cache"))
    q[:T] = turned(s["q"])
    at = s["slots"][:T].long()
    k.view(-1, c["Hkv"], c["D"]).index_copy_(0, at, turned(s["k"]))
    v.view(-1, c["Hkv"], c["D"]).index_copy_(0, at, s["v"][:T].double())
    return {"q_out": q, "k_cache": k, "v_cache": v, "status": s["status"]}


def _exact_lora(c, s):
    """Request by request, with its own adapter's matrices."""
    x, per = s["x"].double(), c["per"]
    y = torch.empty(x.shape[0], c["O"], dtype=torch.float64, device="cuda")
    for o in range(0, c["O"], 1024):
        y[:, o:o + 1024] = x @ s["w"][o:o + 1024].double().T
    scales = s["scales"].double()
    for g, a in enumerate(s["ids"].tolist()):
        if a >= 0:
            rows = slice(g * per, (g + 1) * per)
            y[rows] += scales[a] * (s["b"][a].double() @ (s["a"][a].double() @ x[rows].T)).T
    return {"y": y, "status": torch.zeros_like(s["ids"])}


def exact(case, seed):
    s = prepare(case, seed)
    return {"pages": _exact_pages, "rope": _exact_rope, "lora": _exact_lora}[case["op"]](case, s)
