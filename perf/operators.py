"""Serving attention, measured: whole prompts, drafted trees over a paged cache, and the cache's own work.

Five operators that one serving step uses together:

- ``prompt``: causal attention of whole prompts packed back to back, grouped heads, token-major rows;
- ``tree``: attention of drafted tokens (a tree, a chain or one token) over a cache in pages and over each other;
- ``append``: the keys and values of new or accepted tokens, written into their pages;
- ``update``: every slot of the cache becomes a prefix of some slot (fork, beam reordering, trimming, freeing,
  growing), sharing full pages and copying the page that is written next;
- ``compact``: the pages in use move to the lowest ids.

Where ``own`` is false, ``run`` computes them in elementary torch operations, in 32 bits and rounded once.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a handful of short chat turns at the GPT-2 head layout (12 heads of 64): latency counts
        dict(name="prompt_chat", op="prompt", dtype="bf16", d=64, hq=12, hkv=12, seqs=4, longest=200, fused=False,
             shape_seed=1),
        # a batch of ordinary prompts of very different lengths, q, k, v views of one projection, 2 heads a group
        dict(name="prompt_batch", op="prompt", dtype="fp16", d=128, hq=16, hkv=8, seqs=16, longest=2048, fused=True,
             shape_seed=2),
        # long documents, 8 heads a group: bound by the tensor cores
        dict(name="prompt_long", op="prompt", dtype="bf16", d=128, hq=16, hkv=2, seqs=3, longest=8192, fused=True,
             shape_seed=3),
        # a small draft on short contexts, 16-token pages, one head a group: latency counts
        dict(name="tree_small", op="tree", dtype="fp16", d=64, hq=12, hkv=12, seqs=8, ctx=700, nodes=7, tree=True,
             page=16, shape_seed=4),
        # plain decoding: one token a sequence over contexts of very different lengths: bound by memory
        dict(name="decode_batch", op="tree", dtype="bf16", d=128, hq=32, hkv=8, seqs=64, ctx=8192, nodes=1,
             tree=False, page=64, shape_seed=5),
        # long contexts verified with full trees: as much tensor work as memory traffic
        dict(name="tree_long", op="tree", dtype="bf16", d=128, hq=32, hkv=8, seqs=64, ctx=32768, nodes=64, tree=True,
             page=64, shape_seed=6),
        # the accepted path of each sequence's draft, picked by row out of the draft's keys and values
        dict(name="append_accepted", op="append", dtype="bf16", d=128, hkv=8, seqs=64, ctx=4096, tokens=5, pick=True,
             page=64, shape_seed=7),
        # the keys and values of whole prompts
        dict(name="append_prompt", op="append", dtype="fp16", d=128, hkv=8, seqs=8, ctx=1, tokens=8192, pick=False,
             page=16, shape_seed=8),
        # one step of beam search: four beams each, 12 layers of 12 heads of 64 (the GPT-2 layout)
        dict(name="update_beams", op="update", dtype="bf16", d=64, hkv=12, layers=12, what="beams", slots=16, beams=4,
             ctx=500, page=16, shape_seed=9),
        # a busy server's step: slots freed, forked, trimmed and grown
        dict(name="update_mixed", op="update", dtype="bf16", d=128, hkv=8, layers=16, what="mixed", slots=256, beams=1,
             ctx=2000, page=32, shape_seed=10),
        # a small pool after some requests have ended
        dict(name="compact_small", op="compact", dtype="fp16", d=64, hkv=12, layers=12, slots=8, ctx=500, page=16,
             used=0.7, shape_seed=11),
        # a large pool half empty, before part of it is given back
        dict(name="compact_large", op="compact", dtype="bf16", d=128, hkv=8, layers=32, slots=64, ctx=4096, page=64,
             used=0.6, shape_seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "tree", "append", "update", "compact"])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), d=rng.choice([64, 128]), shape_seed=rng.randrange(1, 1 << 20))
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 12])
    if op in ("prompt", "tree"):
        group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if g * hkv <= 32])
        c.update(hq=group * hkv, hkv=hkv, seqs=_log(rng, 1, 64 if op == "tree" else 24))
    if op == "prompt":
        most = math.sqrt(3 * 16 * 8192 ** 2 / (c["seqs"] * c["hq"]))
        c.update(longest=_log(rng, 1, min(8192, most)), fused=rng.random() < 0.5)
    elif op == "tree":
        c.update(nodes=rng.choice([1, 1, _log(rng, 2, 128), rng.randrange(2, 65)]), page=rng.choice([16, 32, 64, 128]))
        most = min(32768.0, 32 * 64 * 64 * 32768 / (c["seqs"] * c["hq"] * c["nodes"]),
                   8 * 64 * 32768 * 128 / (c["seqs"] * hkv * c["d"]))
        c.update(ctx=_log(rng, 1, most), tree=c["nodes"] > 1 and rng.random() < 0.7)
    elif op == "append":
        tokens = rng.choice([1, _log(rng, 1, 16), _log(rng, 1, 8192)])
        c.update(hkv=hkv, seqs=_log(rng, 1, max(1, min(256, 8 * 8192 // tokens))), tokens=tokens,
                 ctx=_log(rng, 1, 4096), pick=tokens > 1 and rng.random() < 0.5, page=rng.choice([16, 32, 64, 128]))
    elif op == "update":
        c.update(hkv=hkv, layers=rng.choice([1, 2, 7, 12, 16]), what=rng.choice(["beams", "mixed"]),
                 beams=rng.choice([2, 3, 4, 8]), slots=_log(rng, 8, 256), ctx=_log(rng, 1, 2000),
                 page=rng.choice([16, 32, 64]))
    else:
        c.update(hkv=hkv, layers=rng.choice([1, 2, 7, 12, 16]), slots=_log(rng, 1, 64), ctx=_log(rng, 1, 4096),
                 page=rng.choice([16, 32, 64]), used=rng.choice([0.2, 0.5, 0.9, 1.0]))
    return c


def _lengths(r, count, longest):
    """Lengths up to `longest`, the first of them that long, spread over their logarithm; a few empty."""
    x = np.exp(r.uniform(0.0, math.log(longest + 0.999), count)).astype(np.int64).clip(1, longest)
    if count > 4:
        x[r.uniform(size=count) < 0.04] = 0
    x[0] = longest
    return x


def _offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def _plan(case):
    """What the case's sizes are, from the case alone: lengths, pages, trees and what becomes of the slots."""
    r = np.random.RandomState(case["shape_seed"])
    op, s = case["op"], {}
    if op == "prompt":
        s["lens"] = _lengths(r, case["seqs"], case["longest"])
        return s
    page = case["page"]
    if op == "tree":
        s["lens"] = r.randint(max(1, case["ctx"] // 8), case["ctx"] + 1, case["seqs"])
        s["lens"][0] = case["ctx"]
        n = r.randint(max(1, case["nodes"] // 2), case["nodes"] + 1, case["seqs"])
        n[0] = case["nodes"]
        if case["seqs"] > 4:
            n[r.randint(1, case["seqs"])] = 0  # a slot that sits this step out
            s["lens"][r.randint(1, case["seqs"])] = 0
        s["n"] = n
        s["parents"] = np.concatenate([[-1 if i == 0 else r.randint(max(0, i // 2 - 2), i) for i in range(k)]
                                       for k in n]).astype(np.int64)
        pages = -(-s["lens"] // page)
        width, pool = int(pages.max()) + 1, int(pages.sum()) + 3
    elif op == "append":
        s["lens"] = r.randint(0, case["ctx"] + 1, case["seqs"])
        s["n"] = _lengths(r, case["seqs"], case["tokens"])
        s["drafted"] = 2 * s["n"] + 3 if case["pick"] else s["n"]
        s["pick"] = [np.sort(r.choice(int(m), int(k), replace=False)) for m, k in zip(s["drafted"], s["n"])]
        pages = -(-(s["lens"] + s["n"]) // page)
        width, pool = int(pages.max()) + 1, int(pages.sum()) + 3
    else:
        slots = case["slots"]
        s["lens"] = _lengths(r, slots, case["ctx"])
        if op == "update":
            s["src"], s["new"] = np.arange(slots), s["lens"].copy()
            if case["what"] == "beams":  # the beams of a group are as long as each other; each takes one of them and a token
                group = np.arange(slots) // case["beams"]
                s["lens"] = s["lens"][group * case["beams"]]
                s["src"] = np.minimum(group * case["beams"] + r.randint(0, case["beams"], slots), slots - 1)
                s["new"] = s["lens"] + (s["lens"] > 0)
            else:
                u = r.uniform(size=slots)
                grow = u < 0.4
                s["new"][grow] += r.randint(1, 2 * page, int(grow.sum()))
                cut = (u >= 0.4) & (u < 0.6)
                s["new"][cut] = (s["lens"][cut] * r.uniform(size=int(cut.sum()))).astype(np.int64)
                s["new"][(u >= 0.6) & (u < 0.75)] = 0
                fork = (u >= 0.75) & (u < 0.9)
                s["src"][fork] = r.randint(0, slots, int(fork.sum()))
                s["new"][fork] = s["lens"][s["src"][fork]] + r.randint(0, 3, int(fork.sum()))
        pages = -(-s["lens"] // page)
        width = int(max(pages.max(), (-(-s["new"] // page)).max() if op == "update" else 0)) + 1
        pool = int(pages.sum()) + (int((-(-s["new"] // page)).sum()) if op == "update" else 0) + 3
        if op == "compact":
            pool = max(pool, int(math.ceil(pages.sum() / case["used"])))
    ids = r.permutation(pool)[: int(pages.sum())]
    first = _offsets(pages)
    table = np.full((len(pages), width), -1, np.int64)
    for b, k in enumerate(pages):
        table[b, :k] = ids[first[b]: first[b] + k]
    if op == "update" and case["what"] == "beams":  # the beams of a group share the pages of the prompt's first half
        shared = (s["lens"] // 2) // page
        for b in range(len(pages)):
            table[b, : shared[b]] = table[b // case["beams"] * case["beams"], : shared[b]]
    s.update(table=table, pool=pool, width=width, pages=pages)
    return s


# ------------------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    s = _plan(case)
    dt, d, hkv = DTYPES[case["dtype"]], case["d"], case["hkv"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 11)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    def ints(x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(device="cuda", dtype=torch.int32)

    out = {"case": case, "op": case["op"], "scale": 1.0 / math.sqrt(d), "page": case.get("page")}
    if case["op"] == "prompt":
        t, hq = int(s["lens"].sum()), case["hq"]
        if case["fused"]:  # views of one projection's rows
            rows = normal(t, hq + 2 * hkv, d)
            q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        else:
            q, k, v = normal(t, hq, d), normal(t, hkv, d), normal(t, hkv, d)
        out.update(q=q, k=k, v=v, cu=ints(_offsets(s["lens"])), longest=int(s["lens"].max()))
        return out
    if case["op"] in ("tree", "append"):
        kv = torch.empty((2, s["pool"], hkv, case["page"], d), dtype=dt, device="cuda")
        kv.normal_(generator=g)
        out.update(k_cache=kv[0], v_cache=kv[1], table=ints(s["table"]), lens=ints(s["lens"]), cu=ints(_offsets(s["n"])),
                   longest=int(s["n"].max()))
    if case["op"] == "tree":
        t = int(s["n"].sum())
        out.update(q=normal(t, case["hq"], d), k=normal(t, hkv, d), v=normal(t, hkv, d),
                   parents=ints(s["parents"]) if case["tree"] else None, words=-(-case["nodes"] // 32))
    elif case["op"] == "append":
        t = int(s["drafted"].sum())
        rows = np.concatenate([p + o for p, o in zip(s["pick"], _offsets(s["drafted"]))]) if case["pick"] else None
        out.update(k=normal(t, hkv, d), v=normal(t, hkv, d), rows=None if rows is None else ints(rows))
    elif case["op"] in ("update", "compact"):
        kv = torch.empty((2 * case["layers"], s["pool"], hkv, case["page"], d), dtype=dt, device="cuda")
        kv.normal_(generator=g)
        out.update(kv=kv, table=ints(s["table"]), lens=ints(s["lens"]))
        if case["op"] == "update":
            out.update(src=ints(s["src"]), new=ints(s["new"]))
    return out


# ------------------------------------------------------------------------------------------------ the passes
def run(state):
    if own:
        return {"prompt": _own_prompt, "tree": _own_tree, "append": _own_append, "update": _own_update,
                "compact": _own_compact}[state["op"]](state)
    return {"prompt": _plain_prompt, "tree": _plain_tree, "append": _plain_append, "update": _plain_update,
            "compact": _plain_compact}[state["op"]](state)


def _own_prompt(s):
    from io_aware_exact_04_gb300 import api
    o, lse = api.forward_prompt(s["q"], s["k"], s["v"], s["cu"], scale=s["scale"])
    return {"o": o, "lse": lse}


def _own_tree(s):
    from io_aware_exact_04_gb300 import api
    if s["parents"] is None:
        o, lse = api.forward_tree(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"],
                                  scale=s["scale"])
        return {"o": o, "lse": lse}
    mask = api.tree_mask(s["parents"], s["cu"], s["words"])
    o, lse = api.forward_tree(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"],
                              mask=mask, scale=s["scale"])
    return {"o": o, "lse": lse, "mask": mask}


def _own_append(s):
    from io_aware_exact_04_gb300 import api
    api.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"], rows=s["rows"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_update(s):
    from io_aware_exact_04_gb300 import api
    table, lens = s["table"].clone(), s["lens"].clone()
    info = api.cache_update(s["kv"], table, lens, s["src"], s["new"])
    return {"kv": s["kv"], "table": table, "lens": lens, "info": info}


def _own_compact(s):
    from io_aware_exact_04_gb300 import api
    table = s["table"].clone()
    info = api.cache_compact(s["kv"], table, s["lens"])
    return {"kv": s["kv"], "table": table, "info": info}


def _padded(cu, longest):
    """Rows of each sequence in a padded batch: their places among the packed rows, and which of them exist."""
    i = torch.arange(longest, device=cu.device)
    n = (cu[1:] - cu[:-1]).long()
    there = i[None, :] < n[:, None]
    return torch.where(there, cu[:-1, None].long() + i[None, :], 0), there


def _softmax_rows(q, k, v, scale, seen):
    """O and LSE of padded rows: q [B, H, G, n, d], k and v [B, H, m, d], seen [B or 1, n, m]."""
    scores = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, q.shape[2:4]) * scale
    scores = scores.masked_fill(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, q.shape[2:4]) / torch.where(total > 0, total, 1.0)
    return o, (top + torch.log(total)).squeeze(-1)


def _packed(x, there):
    """[B, H, G, n, ...] of a padded batch -> [T, H * G, ...] of the rows that exist (head h G + g)."""
    return x.permute(0, 3, 1, 2, *range(4, x.dim())).flatten(2, 3)[there]


def _grouped(q, at, hkv):
    """[T, H G, d] -> [B, H, G, n, d] in 32 bits."""
    return q.float()[at].unflatten(2, (hkv, -1)).permute(0, 2, 3, 1, 4)


def _plain_prompt(s):
    at, there = _padded(s["cu"], s["longest"])
    hkv = s["k"].shape[1]
    q = _grouped(s["q"], at, hkv)
    k, v = (_grouped(s[x], at, hkv).squeeze(2) for x in ("k", "v"))
    i = torch.arange(s["longest"], device=at.device)
    o, lse = _softmax_rows(q, k, v, s["scale"], (i[None, :] <= i[:, None]) & there[:, None, :])
    return {"o": _packed(o, there).to(s["q"].dtype), "lse": _packed(lse, there).t().contiguous()}


def _plain_tree(s):
    at, there = _padded(s["cu"], s["longest"])
    hkv, n = s["k"].shape[1], s["longest"]
    q = _grouped(s["q"], at, hkv)
    # keys: the context out of its pages, then the drafted tokens
    table = s["table"].long().clamp(min=0)
    k, v = (torch.cat([s[c][table].permute(0, 2, 1, 3, 4).flatten(2, 3).float(), _grouped(s[x], at, hkv).squeeze(2)], 2)
            for c, x in (("k_cache", "k"), ("v_cache", "v")))
    ctx = k.shape[2] - n
    i = torch.arange(n, device=at.device)
    out = {}
    if s["parents"] is None:
        nodes = (i[None, :] <= i[:, None]) & there[:, None, :]
    else:
        parents = torch.where(there, s["parents"].long()[at], -1)
        edges = (parents[:, :, None] == i[None, None, :]).double() + torch.eye(n, dtype=torch.float64, device=at.device)
        nodes = (torch.linalg.matrix_power(edges, 1 << (n - 1).bit_length()) > 0) & there[:, None, :]
        bits = torch.nn.functional.pad(nodes, (0, 32 * s["words"] - n)).reshape(*nodes.shape[:2], s["words"], 32)
        words = (bits.long() << torch.arange(32, device=at.device)).sum(-1)[there]
        out["mask"] = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    c = torch.arange(ctx, device=at.device) < s["lens"][:, None]
    o, lse = _softmax_rows(q, k, v, s["scale"], torch.cat([c[:, None, :].expand(-1, n, -1), nodes], -1))
    return {"o": _packed(o, there).to(s["q"].dtype), "lse": _packed(lse, there).t().contiguous(), **out}


def _plain_append(s):
    cu, page = s["cu"].long(), s["page"]
    count = s["k"].shape[0] if s["rows"] is None else s["rows"].shape[0]
    t = torch.arange(count, device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    at = s["lens"].long()[b] + t - cu[b]
    ids = s["table"].long()[b, at // page]
    for x, c in (("k", "k_cache"), ("v", "v_cache")):
        s[c][ids, :, at % page] = s[x] if s["rows"] is None else s[x][s["rows"].long()]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _in_use(table, lens, page, pool):
    """How often each page is in use."""
    used = torch.arange(table.shape[1], device=table.device) < ((lens + page - 1) // page)[:, None]
    count = torch.zeros(pool + 1, dtype=torch.int64, device=table.device)
    return count.scatter_add_(0, torch.where(used, table, pool).flatten(), torch.ones_like(table).flatten())[:pool]


def _plain_update(s):
    kv, page = s["kv"], s["page"]
    pool, width = kv.shape[1], s["table"].shape[1]
    table, lens, src, new = (s[x].clone().long() for x in ("table", "lens", "src", "new"))
    slot, col = torch.arange(len(lens), device=lens.device), torch.arange(width, device=lens.device)
    old = table[src]
    keep = torch.minimum(new, lens[src])
    full, part = keep // page, keep % page
    own_part = (part > 0) & (src == slot)
    shares = _in_use(old, (full + own_part) * page, page, pool)
    part_page = old.gather(1, full.clamp(max=width - 1)[:, None])[:, 0].clamp(min=0)
    stays = own_part & (shares[part_page] == 1)
    kept = full + stays
    pages = (new + page - 1) // page
    need = pages - kept
    free = _in_use(table, lens, page, pool) == 0
    info = torch.stack([need.sum(), free.sum()]).to(torch.int32)
    ids = torch.sort((~free).to(torch.int8), stable=True).indices
    fresh = ids[(need.cumsum(0) - need)[:, None].add(col[None, :] - kept[:, None]).clamp(0, pool - 1)]
    made = torch.where(col < kept[:, None], old, torch.where(col < pages[:, None], fresh, -1))
    fits = info[0] <= info[1]
    copied = (part > 0) & ~stays & fits
    to, of, rows = (x[copied] for x in (made.gather(1, full.clamp(max=width - 1)[:, None])[:, 0], part_page, part))
    first = (torch.arange(page, device=lens.device) < rows[:, None])[None, :, None, :, None]
    kv[:, to] = torch.where(first, kv[:, of], kv[:, to])
    return {"kv": kv, "table": torch.where(fits, made, table).to(torch.int32),
            "lens": torch.where(fits, new, lens).to(torch.int32), "info": info}


def _plain_compact(s):
    kv, page = s["kv"], s["page"]
    pool = kv.shape[1]
    table, lens = s["table"].clone().long(), s["lens"].long()
    used = _in_use(table, lens, page, pool) > 0
    count = used.sum()
    ids = torch.arange(pool, device=used.device)
    high, holes = ids[used & (ids >= count)], ids[~used & (ids < count)]
    goes = ids.clone()
    goes[high] = holes
    kv[:, holes] = kv[:, high]
    mine = torch.arange(table.shape[1], device=used.device) < ((lens + page - 1) // page)[:, None]
    moved = torch.where(mine, goes[table.clamp(min=0)], table)
    return {"kv": kv, "table": moved.to(torch.int32), "info": torch.stack([count, (used & (ids >= count)).sum()]).to(torch.int32)}


# ------------------------------------------------------------------------------------------------ floors
def work(case):
    s = _plan(case)
    d, hkv = case["d"], case["hkv"]
    row = 2 * d  # bytes of one head's row
    if case["op"] == "prompt":
        n, hq = s["lens"].astype(np.float64), case["hq"]
        return {"bytes": float(n.sum() * (2 * hq * row + 2 * hkv * row + 4 * hq)),
                "flops": float(4 * d * hq * (n * (n + 1) / 2).sum())}
    if case["op"] == "tree":
        n, hq = s["n"].astype(np.float64), case["hq"]
        ctx = np.where(n > 0, s["lens"], 0).astype(np.float64)
        pages = np.where(n > 0, s["pages"], 0)
        pairs = n * ctx
        if case["tree"]:
            depth = np.zeros(len(s["parents"]), np.int64)
            first = np.repeat(_offsets(s["n"])[:-1], s["n"])
            for i, p in enumerate(s["parents"]):
                depth[i] = 1 if p < 0 else depth[first[i] + p] + 1
            seen = depth.sum()
        else:
            seen = (n * (n + 1) / 2).sum()
        return {"bytes": float(2 * hkv * row * (ctx.sum() + n.sum()) + n.sum() * hq * (2 * row + 4) + 4 * pages.sum()),
                "flops": float(4 * d * hq * (pairs.sum() + seen))}
    if case["op"] == "append":
        return {"bytes": float(s["n"].sum() * 2 * hkv * row * 2)}
    planes, page = 2 * case["layers"], case["page"]
    if case["op"] == "update":
        keep = np.minimum(s["new"], s["lens"][s["src"]])
        copied = np.where(s["src"] != np.arange(len(keep)), keep % page, 0)
        return {"bytes": float(4 * (s["pages"].sum() + s["table"].size) + 16 * len(keep) + 2 * planes * hkv * row * copied.sum())}
    used = np.unique(s["table"][s["table"] >= 0])
    moved = int((used >= len(used)).sum())
    return {"bytes": float(4 * (s["pages"].sum() + moved + len(s["lens"])) + 2.0 * planes * moved * hkv * page * row)}


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "tree": _exact_tree, "append": _exact_append, "update": _exact_update,
            "compact": _exact_compact}[case["op"]](s)


def _exact_head(q, k, v, scale, seen):
    """O and LSE of one head in 64 bits, row by key; seen [n, m]."""
    x = (q.double() @ k.double().t()) * scale
    x[~seen] = -math.inf
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[:, None])
    p[~seen] = 0.0
    return p @ v.double(), lse


def _exact_rows(s, keys, values, sees):
    """Every sequence and head by itself: keys(b, h), values(b, h) [m, d], sees(b) [n, m]."""
    q, cu = s["q"], s["cu"].tolist()
    group = q.shape[1] // s["k"].shape[1]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros((q.shape[1], q.shape[0]), dtype=torch.float64, device=q.device)
    for b in range(len(cu) - 1):
        lo, hi = cu[b], cu[b + 1]
        if lo == hi:
            continue
        seen = sees(b)
        for h in range(q.shape[1]):
            o[lo:hi, h], lse[h, lo:hi] = _exact_head(q[lo:hi, h], keys(b, h // group), values(b, h // group), s["scale"], seen)
    return {"o": o, "lse": lse}


def _exact_prompt(s):
    cu = s["cu"].tolist()
    return _exact_rows(s, lambda b, h: s["k"][cu[b]:cu[b + 1], h], lambda b, h: s["v"][cu[b]:cu[b + 1], h],
                       lambda b: torch.ones((cu[b + 1] - cu[b],) * 2, dtype=torch.bool, device=s["q"].device).tril())


def _exact_tree(s):
    cu, lens, page = s["cu"].tolist(), s["lens"].tolist(), s["page"]
    parents = None if s["parents"] is None else s["parents"].tolist()
    def rows(cache, new, b, h):
        ids = s["table"][b, : -(-lens[b] // page)].long()
        return torch.cat([cache[:, h].index_select(0, ids).flatten(0, 1)[: lens[b]], new[cu[b]:cu[b + 1], h]])

    def nodes(b):
        n = cu[b + 1] - cu[b]
        seen = np.zeros((n, n), bool)
        for i in range(n):
            j = i
            while j >= 0:
                seen[i, j] = True
                j = j - 1 if parents is None else parents[cu[b] + j]
        return seen

    def sees(b):
        seen = torch.from_numpy(nodes(b)).to(s["q"].device)
        return torch.cat([torch.ones((len(seen), lens[b]), dtype=torch.bool, device=seen.device), seen], 1)

    out = _exact_rows(s, lambda b, h: rows(s["k_cache"], s["k"], b, h), lambda b, h: rows(s["v_cache"], s["v"], b, h), sees)
    if parents is not None:
        words = np.zeros((cu[-1], 32 * s["words"]), bool)
        for b in range(len(lens)):
            words[cu[b]:cu[b + 1], : cu[b + 1] - cu[b]] = nodes(b)
        out["mask"] = torch.from_numpy(np.packbits(words, axis=1, bitorder="little").view(np.int32).copy())
    return out


def _exact_append(s):
    cu, lens, table, page = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist(), s["page"]
    rows = list(range(cu[-1])) if s["rows"] is None else s["rows"].tolist()
    to, of = [], []
    for b in range(len(lens)):
        for i in range(cu[b + 1] - cu[b]):
            at = lens[b] + i
            to.append((table[b][at // page], at % page))
            of.append(rows[cu[b] + i])
    ids, places = (torch.tensor(x, device="cuda") for x in zip(*to))
    out = {}
    for x, c in (("k", "k_cache"), ("v", "v_cache")):
        heads = s[c].transpose(1, 2).clone()  # [page, token, head, d]
        heads[ids, places] = s[x][torch.tensor(of, device="cuda")]
        out[c] = heads.transpose(1, 2)
    return out


def _exact_update(s):
    kv, page = s["kv"].clone(), s["page"]
    table, lens, src, new = (s[x].tolist() for x in ("table", "lens", "src", "new"))
    slots, width, pool = len(lens), len(table[0]), kv.shape[1]
    busy = {p for b in range(slots) for p in table[b][: -(-lens[b] // page)]}
    free = [p for p in range(pool) if p not in busy]
    keep = [min(new[b], lens[src[b]]) for b in range(slots)]
    holders = {}
    for b in range(slots):
        for j in range(-(-keep[b] // page) if src[b] == b else keep[b] // page):
            p = table[src[b]][j]
            holders[p] = holders.get(p, 0) + 1
    made, copies, taken = [], [], 0
    for b in range(slots):
        row = table[src[b]][: keep[b] // page]
        if keep[b] % page:
            p = table[src[b]][keep[b] // page]
            if src[b] == b and holders[p] == 1:
                row = row + [p]
            else:
                copies.append((b, len(row), p, keep[b] % page))
        while len(row) < -(-new[b] // page):
            row.append(free[taken] if taken < len(free) else -1)
            taken += 1
        made.append(row + [-1] * (width - len(row)))
    fits = taken <= len(free)
    if fits:
        for b, j, p, rows in copies:
            kv[:, made[b][j], :, :rows] = s["kv"][:, p, :, :rows]
    return {"kv": kv, "table": torch.tensor(made if fits else table, dtype=torch.int32),
            "lens": torch.tensor(new if fits else lens, dtype=torch.int32),
            "info": torch.tensor([taken, len(free)], dtype=torch.int32)}


def _exact_compact(s):
    kv, page = s["kv"].clone(), s["page"]
    table, lens = s["table"].tolist(), s["lens"].tolist()
    busy = sorted({p for b in range(len(lens)) for p in table[b][: -(-lens[b] // page)]})
    high = [p for p in busy if p >= len(busy)]
    there = set(busy)
    goes = dict(zip(high, [p for p in range(len(busy)) if p not in there]))
    for of, to in goes.items():
        kv[:, to] = s["kv"][:, of]
    made = [[goes.get(p, p) if j * page < lens[b] else p for j, p in enumerate(row)] for b, row in enumerate(table)]
    return {"kv": kv, "table": torch.tensor(made, dtype=torch.int32),
            "info": torch.tensor([len(busy), len(high)], dtype=torch.int32)}
