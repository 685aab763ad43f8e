"""Measured cases of the operators around a prompt's way into the paged KV cache: attention of
chunks of new tokens over it, per-head norms of queries and keys with their rotary positions and
the write into it in one pass, and forks of sequences that share its pages.

Where ``own`` is false, ``run`` computes them in elementary torch operations; where it is true,
it makes the library's calls. Every case names its operator in "op".
"""

import math

import numpy as np
import torch

own = False

DEV_NO_PAGES = 128


def listed():
    return [
        # One token of one request, 8B-shaped heads: the smallest decode step.
        {"name": "chunk_token_8b", "op": "chunk", "B": 1, "rows": 1, "prefix": 2048, "Hq": 32,
         "Hkv": 8, "D": 128, "page_size": 16, "dtype": "bf16", "mix": "even", "pad": 0},
        # fp32 chains of ragged lengths (the small chain's heads), a padded tail behind them.
        {"name": "chunk_chain_fp32", "op": "chunk", "B": 5, "rows": 333, "prefix": 1000, "Hq": 4,
         "Hkv": 4, "D": 64, "page_size": 16, "dtype": "fp32", "mix": "ragged", "pad": 11},
        # 64 requests of the 70B-shaped layer, one token each, over long ragged contexts.
        {"name": "chunk_decode_64", "op": "chunk", "B": 64, "rows": 64, "prefix": 32768, "Hq": 64,
         "Hkv": 8, "D": 128, "page_size": 16, "dtype": "bf16", "mix": "even", "pad": 0},
        # A step that mixes decoding requests with ragged chunks of prompts; seven heads to a KV head.
        {"name": "chunk_mixed_odd", "op": "chunk", "B": 37, "rows": 5003, "prefix": 4096, "Hq": 28,
         "Hkv": 4, "D": 128, "page_size": 32, "dtype": "bf16", "mix": "decode", "pad": 5},
        # A whole prompt of an 8B-shaped layer, nothing cached before it.
        {"name": "chunk_prompt_8b", "op": "chunk", "B": 1, "rows": 8192, "prefix": 0, "Hq": 32,
         "Hkv": 8, "D": 128, "page_size": 16, "dtype": "bf16", "mix": "even", "pad": 0},
        # A chunk in the middle of a long prompt, 70B-shaped layer.
        {"name": "chunk_long_70b", "op": "chunk", "B": 1, "rows": 8185, "prefix": 24576, "Hq": 64,
         "Hkv": 8, "D": 128, "page_size": 64, "dtype": "bf16", "mix": "even", "pad": 0},
        # One token of one request: the smallest write.
        {"name": "nrope_token_8b", "op": "nrope", "rows": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "rot": 128, "dtype": "bf16", "interleaved": False, "fused": True, "pad": 0, "axes": 1,
         "page_size": 16, "max_pos": 8192},
        # fp32 heads of 64 over a batch, neighbouring pairs, a padded tail behind it.
        {"name": "nrope_chain_fp32", "op": "nrope", "rows": 501, "Hq": 4, "Hkv": 4, "D": 64,
         "rot": 32, "dtype": "fp32", "interleaved": True, "fused": False, "pad": 11, "axes": 1,
         "page_size": 16, "max_pos": 4096},
        # A prompt with images: time, height and width turn interleaved shares of the pairs.
        {"name": "nrope_image_8b", "op": "nrope", "rows": 16391, "Hq": 32, "Hkv": 8, "D": 128,
         "rot": 128, "dtype": "bf16", "interleaved": False, "fused": True, "pad": 0, "axes": 3,
         "page_size": 64, "max_pos": 16896},
        # One more sample of one prompt: its full pages are shared, the last one is copied.
        {"name": "fork_sample_8b", "op": "fork", "prompts": 1, "forks": 1, "prefix": 2048,
         "page_size": 16, "layers": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "short": False},
        # Beams over long prompts: thousands of shared pages each, a single layer's cache.
        {"name": "fork_beams_long", "op": "fork", "prompts": 8, "forks": 56, "prefix": 32768,
         "page_size": 16, "layers": 1, "Hkv": 8, "D": 128, "dtype": "bf16", "short": True},
        # Samples of many prompts, all layers' pages: the copies are the work.
        {"name": "fork_samples_8b", "op": "fork", "prompts": 16, "forks": 112, "prefix": 600,
         "page_size": 64, "layers": 32, "Hkv": 8, "D": 128, "dtype": "bf16", "short": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "nrope", "fork"])
    if op == "chunk":
        bf = rng.random() < 0.8
        D = 128 if bf else rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 5, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 7, 8])
        mix = rng.choice(["even", "ragged", "decode"])
        B = _log(rng, 1, 64)
        prefix = _log(rng, 1, 30000)
        # the products of one pass, and the cache, stay below the largest listed case's
        top = min(8000, int((1.8e12 if bf else 4.0e10) // (Hq * D * (prefix + 4000))))
        rows = max(B, _log(rng, 1, max(2, top)))
        B = max(1, min(B, 1800000 // (prefix + rows)))
        if mix == "even":
            rows = max(1, rows // B) * B
        return {"op": op, "B": B, "rows": rows, "prefix": prefix, "Hq": Hq, "Hkv": Hkv, "D": D,
                "page_size": rng.choice([16, 32, 64, 128]), "dtype": "bf16" if bf else "fp32",
                "mix": mix, "pad": rng.randint(0, 9)}
    if op == "nrope":
        D = rng.choice([64, 80, 128, 128, 256])
        bf = rng.random() < 0.7
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 3, 4, 7, 8])
        top = int(3.8e8 // ((Hq + 2 * Hkv) * D * (4 if bf else 8)))
        return {"op": op, "rows": max(1, min(_log(rng, 1, 16000), top)), "Hq": Hq, "Hkv": Hkv,
                "D": D, "rot": rng.choice([D, D, D // 2 // 16 * 16]),
                "dtype": "bf16" if bf else "fp32", "interleaved": rng.random() < 0.3,
                "fused": rng.random() < 0.6, "pad": rng.randint(0, 9),
                "axes": rng.choice([1, 1, 2, 3, 4]), "page_size": rng.choice([16, 32, 64]),
                "max_pos": _log(rng, 2048, 32768)}
    prompts, prefix, ps = _log(rng, 1, 24), _log(rng, 1, 32768), rng.choice([16, 32, 64, 128])
    forks = max(1, prompts * rng.randint(1, 8) - rng.randint(0, prompts - 1 if prompts > 1 else 0))
    Hkv, D, bf = rng.choice([1, 4, 8]), rng.choice([64, 128]), rng.random() < 0.7
    page = ps * Hkv * D * (4 if bf else 8)
    pages = prompts * (prefix // ps + 1) + 2 * forks + 8
    return {"op": op, "prompts": prompts, "forks": forks, "prefix": prefix, "page_size": ps,
            "layers": max(1, min(_log(rng, 1, 40), int(2.0e9 // (page * pages)))), "Hkv": Hkv,
            "D": D, "dtype": "bf16" if bf else "fp32", "short": rng.random() < 0.3}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _d(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _prepare_chunk(c, seed):
    g, rng = _gen(seed), np.random.default_rng([int(seed) & 0x7FFFFFFF, 21])
    B, T, ps, dt = c["B"], c["rows"], c["page_size"], _dtype(c)
    lens = rng.integers(c["prefix"] // 2, c["prefix"] + 1, B)
    if B == 1:
        lens[:] = c["prefix"]
    if c["mix"] == "even":
        new = np.full(B, T // B)
    else:  # chunks of ragged lengths; in "decode" three of four requests have one token
        w = rng.gamma(1.0, 1.0, B) + 1e-3
        if c["mix"] == "ragged" and B > 2:
            w[rng.random(B) < 0.15] = 0.0  # nothing this step
            w[rng.integers(B)] += 0.5
        new = np.floor(w / w.sum() * T).astype(np.int64)
        if c["mix"] == "decode" and B > 3:
            new[rng.random(B) < 0.75] = 1
        new[new.argmax()] += T - new.sum()
    held = -(-(lens + new) // ps)
    pages = int(held.sum()) + 3
    perm = rng.permutation(pages).astype(np.int32)
    table = np.full((B, int(held.max()) + 2), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    n = T + c["pad"]  # rows behind the last sequence
    r = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=dt)  # noqa: E731
    # some heads look at few tokens, some at nearly all
    sharp = torch.linspace(0.5, 3.0, c["Hq"], device="cuda")[:, None]
    q = (torch.randn(n, c["Hq"], c["D"], generator=g, device="cuda") * sharp).to(dt)
    offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return {"c": c, "q": q, "k_cache": r(pages, ps, c["Hkv"], c["D"]),
            "v_cache": r(pages, ps, c["Hkv"], c["D"]), "table": _d(table),
            "lens": _d(lens.astype(np.int32)), "offsets": _d(offsets),
            "host": (lens.tolist(), new.tolist()), "out": torch.zeros_like(q), "ws": None,
            "lse": torch.zeros(n, c["Hq"], device="cuda"),
            "status": torch.zeros(B, dtype=torch.int32, device="cuda")}


def _rope_table(max_pos, rot):
    """cos in the first half of a row, sin in the second; angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _prepare_nrope(c, seed):
    g = _gen(seed)
    T, Hq, Hkv, D, ps, A = c["rows"], c["Hq"], c["Hkv"], c["D"], c["page_size"], c["axes"]
    dt = _dtype(c)
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
    shape = (n,) if A == 1 else (A, n)
    pos = torch.randint(0, c["max_pos"], shape, generator=g, device="cuda").to(torch.int32)
    slots[T:] = -1  # rows behind the last sequence
    pos[..., T:] = 0
    axis = None
    if A > 1:  # the axes take the pairs in turn, the last pairs go to the first axis
        i = torch.arange(c["rot"] // 2, device="cuda")
        axis = torch.where(i < c["rot"] // 2 * 7 // 8, i % A, 0).to(torch.int32)
    return {"c": c, "q": q, "k": k, "v": v, "rope": _rope_table(c["max_pos"], c["rot"]),
            "q_norm": (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt),
            "k_norm": (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt),
            "pos": pos, "axis": axis, "slots": slots, "k_cache": r(pages, ps, Hkv, D),
            "v_cache": r(pages, ps, Hkv, D), "q_out": torch.zeros(n, Hq, D, dtype=dt, device="cuda"),
            "status": torch.zeros(n, dtype=torch.int32, device="cuda")}


def _prepare_fork(c, seed):
    """Prompts in the first rows; the other rows hold forks of the step before, which the pass
    gives back before it forks anew."""
    g, rng = _gen(seed), np.random.default_rng([int(seed) & 0x7FFFFFFF, 31])
    P, F, ps, dt = c["prompts"], c["forks"], c["page_size"], _dtype(c)
    lens = rng.integers(max(1, c["prefix"] // 2), c["prefix"] + 1, P)
    lens[::5] = np.maximum(1, lens[::5] // ps) * ps  # some end with their page
    old, src = rng.integers(0, P, F), rng.integers(0, P, F)
    dst = P + rng.permutation(F)
    lens = np.concatenate([lens, lens[old]])
    held = -(-lens // ps)
    # the cache's size goes by the case; pages of other requests are neither held here nor free
    most = -(-max(c["prefix"], ps) // ps)
    num_pages = P * most + 2 * F + 8
    perm = rng.permutation(num_pages).astype(np.int32)
    table = np.full((P + F, most + 2), -1, np.int32)
    shares = np.zeros(num_pages, np.int32)
    at = 0
    for b in range(P):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    for b in range(P, P + F):
        full = lens[b] // ps
        table[b, :full] = table[old[b - P], :full]
        shares[table[b, :full]] += 1
        if lens[b] % ps:
            table[b, full] = perm[at]
            at += 1
    need = int((lens[src] % ps > 0).sum())
    given_back = int((lens[P:] % ps > 0).sum())
    spare = max(0, need * 9 // 10 - given_back) if c["short"] else min(num_pages - at, 2 * F + 8)
    free = np.full(num_pages, -1, np.int32)
    free[:spare] = perm[at:at + spare]
    keep = lens.copy()
    keep[P:] = 0
    r = lambda: torch.randn(c["layers"], num_pages, ps, c["Hkv"], c["D"], generator=g,  # noqa: E731
                            device="cuda", dtype=dt)
    i32 = lambda x: _d(np.asarray(x).astype(np.int32))  # noqa: E731
    return {"c": c, "pool": {"free": i32(free), "state": i32([spare, 0, 0, 0]),
                             "shares": i32(shares)},
            "table": i32(table), "lens": i32(lens), "keep": i32(keep), "src": i32(src),
            "dst": i32(dst), "k_cache": r(), "v_cache": r(), "rel": {}, "out": {},
            "cstat": torch.zeros(F, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    return {"chunk": _prepare_chunk, "nrope": _prepare_nrope, "fork": _prepare_fork}[case["op"]](
        case, seed)


# ------------------------------------------------------------------ plain forms

def _plain_chunk(s):
    """Sequence by sequence, a block of rows against all of its keys at once."""
    c = s["c"]
    Hkv, D, ps = c["Hkv"], c["D"], c["page_size"]
    G, at = c["Hq"] // Hkv, 0
    for b, (L, n) in enumerate(zip(*s["host"])):
        if n == 0:
            continue
        end = L + n
        pages = s["table"][b, :-(-end // ps)].long()
        k = s["k_cache"][pages].flatten(0, 1)[:end].float().permute(1, 2, 0)  # [Hkv, D, end]
        v = s["v_cache"][pages].flatten(0, 1)[:end].float().transpose(0, 1)
        step = max(1, int(1.5e9 // (c["Hq"] * end)))
        t = torch.arange(end, device=k.device)
        for i in range(0, n, step):
            m = min(step, n - i)
            rows = slice(at + i, at + i + m)
            q = s["q"][rows].float().unflatten(1, (Hkv, G)).permute(1, 0, 2, 3).reshape(Hkv, m * G, D)
            x = (q @ k).mul_(D ** -0.5).unflatten(1, (m, G))
            x.masked_fill_(t > (L + i + torch.arange(m, device=k.device))[:, None, None], -math.inf)
            top = x.amax(-1, keepdim=True)
            x = x.sub_(top).exp_()
            total = x.sum(-1, keepdim=True)
            o = (x.flatten(1, 2) @ v).unflatten(1, (m, G)) / total
            s["out"][rows] = o.transpose(0, 1).flatten(1, 2).to(s["out"].dtype)
            s["lse"][rows] = (top + total.log())[..., 0].transpose(0, 1).flatten(1, 2)
        at += n
    s["status"].zero_()


def _normed(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()


def _rotated(x, cs, rot, interleaved):
    cos, sin = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    y = x.clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (
        slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., first], x[..., second]
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y


def _plain_nrope(s):
    c = s["c"]
    keep = s["slots"] >= 0
    slots, rot, dt = s["slots"][keep].long(), c["rot"], s["q"].dtype
    if c["axes"] == 1:
        cs = s["rope"][s["pos"][keep].long()]
    else:  # each pair's angle by its own axis
        pair = torch.arange(rot // 2, device=slots.device)
        pos = s["pos"][:, keep].long()[s["axis"].long()].T  # [rows, pairs]
        cs = torch.cat([s["rope"][pos, pair], s["rope"][pos, pair + rot // 2]], 1)
    turn = lambda x, w: _rotated(_normed(x[keep], w), cs, rot, c["interleaved"]).to(dt)  # noqa: E731
    s["q_out"][keep] = turn(s["q"], s["q_norm"])
    s["k_cache"].flatten(0, 1)[slots] = turn(s["k"], s["k_norm"])
    s["v_cache"].flatten(0, 1)[slots] = s["v"][keep]
    s["status"].zero_()


def _plain_release(s):
    """Every holder that leaves lowers a page's count; the last one puts it back on the stack."""
    c, table, pool = s["c"], s["table"], s["pool"]
    free, state, shares, ps = pool["free"], pool["state"], pool["shares"], c["page_size"]
    lo, hi = ((s[n].long() + ps - 1) // ps for n in ("keep", "lens"))
    col = torch.arange(table.shape[1], device=table.device)
    cut = (col >= lo[:, None]) & (col < hi[:, None])
    row = torch.arange(table.shape[0], device=table.device)[:, None].expand_as(table)
    page = torch.where(cut, table.long(), shares.numel()).reshape(-1)  # the last entry: nobody's
    left = torch.zeros(shares.numel() + 1, dtype=torch.long, device=table.device)
    left.index_add_(0, page, torch.ones_like(page))
    last = torch.full_like(left, -1).scatter_reduce_(0, page, row.reshape(-1), "amax")
    gone = left[:-1] > shares
    back = cut & torch.cat([gone, gone[:1] & False])[page].view_as(cut) & (
        last[page].view_as(cut) == row)
    shares.copy_(torch.where(gone, 0, shares - left[:-1]))
    n = back.sum(1)
    rank = back.reshape(-1).cumsum(0).view_as(cut) - 1
    total = n.sum()
    to = torch.where(back, state[0].long() + total - 1 - rank, free.numel()).reshape(-1)
    grown = torch.cat([free, free[:1]])
    grown[to] = table.reshape(-1)
    free.copy_(grown[:-1])
    table.masked_fill_(cut, -1)
    state[0] += total.int()
    return {"n_released": n.int(), "status": torch.zeros_like(n).int()}


def _plain_fork(s):
    """Rows dst take rows src: full pages shared, a page of its own for the tokens behind them;
    without a free page for these the row is empty."""
    c, table, pool = s["c"], s["table"], s["pool"]
    free, state, shares, ps = pool["free"], pool["state"], pool["shares"], c["page_size"]
    src, dst = s["src"].long(), s["dst"].long()
    L = s["lens"][src].long()
    full, part = L // ps, L % ps
    need = (part > 0).long()
    incl = need.cumsum(0)
    F = state[0].long()
    served = (need == 0) | (incl <= F)
    col = torch.arange(table.shape[1], device=table.device)
    fresh = free.long()[(F - incl).clamp(min=0)]
    rows = torch.where(col < full[:, None], table[src].long(), -1)
    own_page = (col == full[:, None]) & (need > 0)[:, None]
    rows = torch.where(own_page, fresh[:, None], rows)
    ok = served[:, None]
    shared = ok & (col < full[:, None])
    shares += torch.zeros(shares.numel() + 1, dtype=torch.int32, device=table.device).index_add_(
        0, torch.where(shared, rows, shares.numel()).reshape(-1),
        torch.ones(rows.numel(), dtype=torch.int32, device=table.device))[:-1]
    taken = torch.where(served & (need > 0), 1, 0).sum()
    old = table[src, full.clamp(max=table.shape[1] - 1)]
    table[dst] = torch.where(ok, rows, -1).int()
    s["lens"][dst] = torch.where(served, L, 0).int()
    state[0] -= taken.int()
    copies = served & (need > 0)
    return {"copy_src": torch.where(copies, old, -1).int(),
            "copy_dst": torch.where(copies, fresh, -1).int(),
            "copy_len": torch.where(copies, part, 0).int(),
            "status": torch.where(served, 0, DEV_NO_PAGES).int()}


def _plain_copy(s, f):
    src, dst, n = f["copy_src"].long(), f["copy_dst"].long(), f["copy_len"]
    live = src >= 0
    src, dst, n = src[live], dst[live], n[live]
    here = (torch.arange(s["c"]["page_size"], device=n.device) < n[:, None])[:, :, None, None]
    for cache in (s["k_cache"], s["v_cache"]):
        for layer in cache:
            layer[dst] = torch.where(here, layer[src], layer[dst])


def run(state):
    s, c = state, state["c"]
    if own:
        import speculative_decoding_tree_03_gb300 as sv
    if c["op"] == "chunk":
        if own:
            if s["ws"] is None:  # the workspace that a serving program keeps
                need = sv.chunk_attn_workspace_size(s["q"].shape[0], c["B"], c["Hq"], c["Hkv"],
                                                    c["D"], s["q"].dtype)
                s["ws"] = torch.zeros(max(need, 1), dtype=torch.uint8, device="cuda")
            sv.chunk_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["offsets"],
                          out=s["out"], lse=s["lse"], workspace=s["ws"], status=s["status"])
        else:
            _plain_chunk(s)
        return {"out": s["out"], "lse": s["lse"], "status": s["status"]}
    if c["op"] == "nrope":
        if own:
            sv.norm_rope_kv_write(s["q"], s["k"], s["v"], s["q_norm"], s["k_norm"], s["rope"],
                                  s["pos"], s["slots"], s["k_cache"], s["v_cache"], eps=1e-6,
                                  pair_axis=s["axis"], interleaved=c["interleaved"],
                                  q_out=s["q_out"], status=s["status"])
        else:
            _plain_nrope(s)
        return {"q_out": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"],
                "status": s["status"]}
    if own:
        rel = sv.page_release(s["pool"], s["table"], s["lens"], s["keep"], c["page_size"],
                              outputs=s["rel"])
        f = sv.page_fork(s["pool"], s["table"], s["lens"], s["src"], s["dst"], c["page_size"],
                         outputs=s["out"])
        sv.page_copy(s["k_cache"], s["v_cache"], f["copy_src"], f["copy_dst"], f["copy_len"],
                     status=s["cstat"])
    else:
        rel, f = _plain_release(s), _plain_fork(s)
        _plain_copy(s, f)
    return {"n_released": rel["n_released"], "rel_status": rel["status"], "status": f["status"],
            "copy_src": f["copy_src"], "copy_dst": f["copy_dst"], "copy_len": f["copy_len"],
            "table": s["table"], "lens": s["lens"], "free": s["pool"]["free"],
            "state": s["pool"]["state"], "shares": s["pool"]["shares"], "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


# ------------------------------------------------------------------ floors

def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "chunk":
        # requests of about the mean length; a row sees the prefix and, on average, half its chunk
        B, T = c["B"], c["rows"]
        ctx = c["prefix"] if B == 1 else 0.75 * c["prefix"]
        if c["mix"] == "even":
            pairs = T * (ctx + (T / B + 1) / 2)
        elif c["mix"] == "decode" and B > 3:  # a quarter of the requests shares the rows
            pairs = T * (ctx + 2 * T / (B / 4 + 1) / 2)
        else:
            pairs = T * (ctx + 2 * T / (B + 1) / 2)
        kv = (B * ctx + T) * 2 * c["Hkv"] * c["D"] * e
        return {"bytes": int(kv + T * c["Hq"] * (2 * c["D"] * e + 4) +
                             4 * ((B * ctx + T) / c["page_size"] + 3 * B)),
                "flops": int(4 * pairs * c["Hq"] * c["D"])}
    if c["op"] == "nrope":
        rows = c["rows"]
        return {"bytes": rows * (2 * (c["Hq"] + 2 * c["Hkv"]) * c["D"] * e + 8 + 4 * c["axes"]) +
                         min(rows, c["max_pos"]) * c["rot"] * 4 + 2 * c["D"] * e,
                "flops": rows * (c["Hq"] + c["Hkv"]) * (4 * c["D"] + 3 * c["rot"])}
    # per fork: its row out of and into the table, a count per page down and up, half a page of
    # every layer's keys and values read and written
    F, ps = c["forks"], c["page_size"]
    pages = 0.75 * c["prefix"] / ps
    copied = 4 / 5 * F * 0.5 * ps * 2 * c["layers"] * c["Hkv"] * c["D"] * e
    return {"bytes": int(2 * copied + F * (pages * 4 * 6 + 40)), "flops": 0}


# ------------------------------------------------------------------ 64 bits

def _exact_chunk(c, s):
    """KV head by KV head, every row's softmax over the tokens it sees."""
    G, D, ps = c["Hq"] // c["Hkv"], c["D"], c["page_size"]
    if work(c)["flops"] > 1.2e13:
        return None
    out, lse, at = s["out"].double(), s["lse"].double(), 0
    for b, (L, n) in enumerate(zip(*s["host"])):
        tok = torch.arange(L + n, device="cuda")
        where = s["table"][b].long()[tok // ps] * ps + tok % ps
        for h in range(c["Hkv"]):
            k, v = (s[m].flatten(0, 1)[where, h].double() for m in ("k_cache", "v_cache"))
            for i in range(0, n, 512):
                m = min(512, n - i)
                seen = tok[None] <= (L + i + torch.arange(m, device="cuda"))[:, None]
                for j in range(G):
                    x = s["q"][at + i:at + i + m, h * G + j].double() @ k.T / math.sqrt(D)
                    x = torch.where(seen, x, -math.inf)
                    z = torch.logsumexp(x, 1)
                    out[at + i:at + i + m, h * G + j] = (x - z[:, None]).exp() @ v
                    lse[at + i:at + i + m, h * G + j] = z
        at += n
    return {"out": out, "lse": lse, "status": torch.zeros_like(s["status"])}


def _exact_nrope(c, s):
    """Each pair of a normed head as a complex number, turned by the angle of its axis."""
    T, rot = c["rows"], c["rot"]
    pos = s["pos"].view(c["axes"], -1)[:, :T].long()
    axis = s["axis"].long() if s["axis"] is not None else torch.zeros(rot // 2, dtype=torch.long,
                                                                      device="cuda")
    turn = torch.empty(T, 1, rot // 2, dtype=torch.complex128, device="cuda")
    for i, a in enumerate(axis.tolist()):
        turn[:, 0, i] = torch.complex(s["rope"][pos[a], i].double(),
                                      s["rope"][pos[a], rot // 2 + i].double())

    def turned(x, w):
        x = x[:T].double()
        x = w.double() * x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["D"] + 1e-6)
        head = x[..., :rot]
        pairs = head.unflatten(-1, (rot // 2, 2)) if c["interleaved"] else \
            head.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return torch.cat([z, x[..., rot:]], -1)

    q, k, v = (s[n].double() for n in ("q_out", "k_cache", "v_cache"))
    q[:T] = turned(s["q"], s["q_norm"])
    at = s["slots"][:T].long()
    k.view(-1, c["Hkv"], c["D"]).index_copy_(0, at, turned(s["k"], s["k_norm"]))
    v.view(-1, c["Hkv"], c["D"]).index_copy_(0, at, s["v"][:T].double())
    return {"q_out": q, "k_cache": k, "v_cache": v, "status": s["status"]}


def _exact_fork(c, s):
    """The definition, one sequence and one page after the other."""
    ps, P, F = c["page_size"], c["prompts"], c["forks"]
    host = lambda t: t.cpu().numpy().astype(np.int64)  # noqa: E731
    table, lens, keep = host(s["table"]), host(s["lens"]), host(s["keep"])
    src, dst = host(s["src"]), host(s["dst"])
    free, shares = host(s["pool"]["free"]), host(s["pool"]["shares"])
    top = int(s["pool"]["state"][0])
    holders, back, n_rel = shares + 1, [], np.zeros(P + F, np.int64)
    for b in range(P + F):
        for i in range(-(-int(keep[b]) // ps), -(-int(lens[b]) // ps)):
            p = table[b, i]
            table[b, i] = -1
            holders[p] -= 1
            if holders[p] == 0:  # the last one that held it
                back.append(p)
                n_rel[b] += 1
    for p in reversed(back):
        free[top] = p
        top += 1
    for p in back:
        holders[p] = 1  # a page on the stack counts no other holder
    shares = holders - 1
    out = {n: np.full(F, -1, np.int64) for n in ("copy_src", "copy_dst")}
    out["copy_len"], out["status"] = np.zeros(F, np.int64), np.zeros(F, np.int64)
    kc, vc = s["k_cache"], s["v_cache"]
    asked, stack = 0, top
    for f in range(F):
        L, a, d = int(lens[src[f]]), int(src[f]), int(dst[f])
        asked += L % ps > 0
        table[d] = -1
        if L % ps and asked > stack:  # the row stays empty
            out["status"][f], lens[d] = DEV_NO_PAGES, 0
            continue
        table[d, :L // ps] = table[a, :L // ps]
        shares[table[a, :L // ps]] += 1
        lens[d] = L
        if L % ps:
            top -= 1
            old, new = int(table[a, L // ps]), int(free[top])
            table[d, L // ps] = new
            out["copy_src"][f], out["copy_dst"][f], out["copy_len"][f] = old, new, L % ps
            kc[:, new, :L % ps] = kc[:, old, :L % ps]
            vc[:, new, :L % ps] = vc[:, old, :L % ps]
    i32 = lambda x: torch.from_numpy(np.asarray(x).astype(np.int32))  # noqa: E731
    res = {n: i32(x) for n, x in out.items()}
    res.update({"n_released": i32(n_rel), "rel_status": i32(np.zeros(P + F)), "table": i32(table),
                "lens": i32(lens), "free": i32(free), "state": i32([top, 0, 0, 0]),
                "shares": i32(shares), "k_cache": kc, "v_cache": vc})
    names = ("n_released", "rel_status", "status", "copy_src", "copy_dst", "copy_len", "table",
             "lens", "free", "state", "shares", "k_cache", "v_cache")
    return {n: res[n] for n in names}


def exact(case, seed):
    s = prepare(case, seed)
    return {"chunk": _exact_chunk, "nrope": _exact_nrope, "fork": _exact_fork}[case["op"]](case, s)
