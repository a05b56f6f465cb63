"""Serving over a cache in 8 bits, and the position rotation on the way into the cache, measured.

Three operators of a serving step:

- ``attend``: attention of new tokens (one token, a chain or a drafted tree) over a cache in pages held in 8 bits
  (e4m3) with a scale for each block of tokens and head, and over each other;
- ``rotate``: queries and keys rotated by the angles of their positions, keys and values written into their pages,
  of 16 bits, or of 8 bits with their blocks' scales;
- ``append``: keys and values as they are (the accepted tokens of a draft) into pages of 8 bits.

Where ``own`` is false, ``run`` computes them in elementary torch operations, in 32 bits and rounded once.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
BASE = 10000.0


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a small draft on short contexts, 12 heads of 64, small pages and blocks: latency counts
        dict(name="attend_small", op="attend", dtype="fp16", d=64, hq=12, hkv=12, seqs=8, ctx=700, nodes=7, tree=True,
             page=16, block=16, shape_seed=1),
        # plain decoding of a batch over contexts of very different lengths: bound by memory
        dict(name="attend_decode", op="attend", dtype="bf16", d=128, hq=32, hkv=8, seqs=64, ctx=8192, nodes=1,
             tree=False, page=64, block=64, shape_seed=2),
        # the same with heads of 64, small blocks and no groups
        dict(name="attend_decode_64", op="attend", dtype="fp16", d=64, hq=12, hkv=12, seqs=128, ctx=5000, nodes=1,
             tree=False, page=32, block=16, shape_seed=3),
        # two very long contexts: the work lies along one axis
        dict(name="attend_long", op="attend", dtype="bf16", d=128, hq=32, hkv=4, seqs=2, ctx=131072, nodes=1,
             tree=False, page=128, block=32, shape_seed=4),
        # small trees verified, 5 heads a group
        dict(name="attend_draft", op="attend", dtype="bf16", d=128, hq=40, hkv=8, seqs=32, ctx=8000, nodes=6, tree=True,
             page=64, block=64, shape_seed=5),
        # full trees on long contexts: as much tensor work as memory traffic
        dict(name="attend_verify", op="attend", dtype="bf16", d=128, hq=32, hkv=8, seqs=32, ctx=16384, nodes=64,
             tree=True, page=64, block=64, shape_seed=6),
        # a decoding step's tokens into a 16-bit cache: latency counts
        dict(name="rotate_step", op="rotate", dtype="bf16", d=128, hq=32, hkv=8, seqs=64, ctx=4096, tokens=1, page=64,
             block=0, rot=128, interleaved=False, fused=True, shape_seed=7),
        # whole prompts into a 16-bit cache, half of each head rotated, adjacent pairs
        dict(name="rotate_prompt", op="rotate", dtype="fp16", d=128, hq=32, hkv=8, seqs=8, ctx=1, tokens=8192, page=16,
             block=0, rot=64, interleaved=True, fused=False, shape_seed=8),
        # a decoding step's tokens into an 8-bit cache: blocks grow by a token
        dict(name="rotate_step_8bit", op="rotate", dtype="bf16", d=128, hq=32, hkv=8, seqs=64, ctx=4096, tokens=1,
             page=64, block=64, rot=128, interleaved=False, fused=True, shape_seed=9),
        # whole prompts into an 8-bit cache
        dict(name="rotate_prompt_8bit", op="rotate", dtype="bf16", d=128, hq=32, hkv=8, seqs=8, ctx=1, tokens=8192,
             page=64, block=64, rot=128, interleaved=False, fused=True, shape_seed=10),
        # the accepted path of each sequence's draft into an 8-bit cache
        dict(name="append_accepted_8bit", op="append", dtype="bf16", d=128, hq=8, hkv=8, seqs=64, ctx=4096, tokens=5,
             pick=True, page=64, block=32, shape_seed=11),
        # parts of prompts, rotated before, heads of 64
        dict(name="append_parts_8bit", op="append", dtype="fp16", d=64, hq=12, hkv=12, seqs=16, ctx=3000, tokens=2000,
             pick=False, page=32, block=32, shape_seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "rotate", "rotate", "append"])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), d=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128]),
             shape_seed=rng.randrange(1, 1 << 20))
    blocks = [b for b in (16, 32, 64, 128) if b <= c["page"]]
    hkv = rng.choice([1, 2, 3, 4, 5, 8, 12])
    group = rng.choice([g for g in (1, 2, 3, 4, 5, 7, 8, 16) if g * hkv <= 40])
    c.update(hq=group * hkv, hkv=hkv, block=rng.choice(blocks))
    if op == "attend":
        seqs = _log(rng, 1, 128)
        nodes = rng.choice([1, 1, 1, rng.randrange(2, 9), _log(rng, 2, 100)])
        most = min(131072.0, 32 * 16384 * 64 * 32 / (seqs * c["hq"] * nodes), 64 * 8192 * 8 * 128 / (seqs * hkv * c["d"]))
        c.update(seqs=seqs, nodes=nodes, ctx=_log(rng, 1, max(2.0, most)), tree=nodes > 1 and rng.random() < 0.7)
        return c
    tokens = rng.choice([1, _log(rng, 1, 16), _log(rng, 1, 8192)])
    c.update(seqs=_log(rng, 1, max(1, min(256, 8 * 8192 // tokens))), tokens=tokens, ctx=_log(rng, 1, 4096))
    if op == "append":
        c.update(hq=hkv, pick=tokens > 1 and rng.random() < 0.5)
        return c
    c.update(block=rng.choice([0, c["block"]]), rot=rng.choice([c["d"], c["d"], c["d"] // 2, c["d"] // 2 + 16]),
             interleaved=rng.random() < 0.5, fused=rng.random() < 0.5)
    return c


def _offsets(lens):
    return np.concatenate([[0], np.cumsum(lens)])


def _plan(case):
    """What the case's sizes are, from the case alone: lengths, pages and trees."""
    r = np.random.RandomState(case["shape_seed"])
    seqs, page, s = case["seqs"], case["page"], {}
    if case["op"] == "attend":
        lens = r.randint(max(1, case["ctx"] // 8), case["ctx"] + 1, seqs)
        lens[0] = case["ctx"]
        n = r.randint(max(1, case["nodes"] // 2), case["nodes"] + 1, seqs)
        n[0] = case["nodes"]
        if seqs > 4:
            n[r.randint(1, seqs)] = 0  # a slot that sits this step out
            lens[r.randint(1, seqs)] = 0
        s["parents"] = [[-1 if i == 0 else int(r.randint(max(0, i // 2 - 2), i)) for i in range(k)] for k in n]
        pages = -(-lens // page)
    else:
        lens = r.randint(0, case["ctx"] + 1, seqs)
        n = np.exp(r.uniform(0.0, math.log(case["tokens"] + 0.999), seqs)).astype(np.int64).clip(1, case["tokens"])
        if seqs > 4:
            n[r.uniform(size=seqs) < 0.04] = 0
        n[0] = case["tokens"]
        drafted = 2 * n + 3 if case.get("pick") else n
        s["drafted"] = drafted
        s["rows"] = np.concatenate([np.sort(r.choice(int(m), int(k), replace=False)) + o
                                    for m, k, o in zip(drafted, n, _offsets(drafted))]).astype(np.int64)
        pages = -(-(lens + n) // page)
    ids = r.permutation(int(pages.sum()) + 3)
    first = _offsets(pages)
    table = np.full((seqs, int(pages.max()) + 1), -1, np.int64)
    for b, k in enumerate(pages):
        table[b, :k] = ids[first[b]: first[b] + k]
    s.update(lens=lens, n=n, pages=pages, table=table, pool=len(ids))
    return s


# ------------------------------------------------------------------------------------------------ inputs
def _cache(case, pool, g):
    """K and V of a cache in 8 bits and their blocks' scales: powers of two that bring each block near the type's range,
    heads of different sizes."""
    hkv, page, d, block = case["hkv"], case["page"], case["d"], case["block"]
    size = torch.exp2(torch.randint(-2, 3, (2, 1, hkv, 1, 1), generator=g, device="cuda").float())
    values = torch.empty((2, pool, hkv, page, d), dtype=E4M3, device="cuda")
    scales = torch.empty((2, pool, hkv, page // block), dtype=torch.float32, device="cuda")
    some = max(1, (1 << 26) // (hkv * page * d))
    for p in range(0, pool, some):
        x = torch.randn((2, min(some, pool - p), hkv, page, d), generator=g, device="cuda") * size
        x = x.unflatten(3, (page // block, block))
        scale = torch.exp2(torch.ceil(torch.log2(x.abs().amax((-2, -1)) / 440.0)))
        values[:, p:p + some] = (x / scale[..., None, None]).flatten(3, 4).to(E4M3)
        scales[:, p:p + some] = scale
    return values, scales


def _angles(count, dim):
    """[count, dim]: the cosines of each position's angles, then the sines."""
    at = torch.arange(count, dtype=torch.float64, device="cuda")
    f = BASE ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    x = at[:, None] * f[None, :]
    return torch.cat([torch.cos(x), torch.sin(x)], 1).float()


def prepare(case, seed):
    s = _plan(case)
    dt, d, hq, hkv = DTYPES[case["dtype"]], case["d"], case["hq"], case["hkv"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 6007 + 17)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    def ints(x):
        return torch.from_numpy(np.ascontiguousarray(x)).to(device="cuda", dtype=torch.int32)

    out = {"op": case["op"], "scale": 1.0 / math.sqrt(d), "page": case["page"], "block": case["block"], "longest": int(s["n"].max()),
           "table": ints(s["table"]), "lens": ints(s["lens"]), "cu": ints(_offsets(s["n"]))}
    if case["block"]:
        values, scales = _cache(case, s["pool"], g)
        out.update(k_cache=values[0], v_cache=values[1], k_scale=scales[0], v_scale=scales[1])
    else:
        kv = torch.empty((2, s["pool"], hkv, case["page"], d), dtype=dt, device="cuda").normal_(generator=g)
        out.update(k_cache=kv[0], v_cache=kv[1], k_scale=None, v_scale=None)
    if case["op"] == "append":
        t = int(s["drafted"].sum())
        out.update(k=normal(t, hkv, d), v=normal(t, hkv, d), rows=ints(s["rows"]) if case["pick"] else None)
        return out
    t = int(s["n"].sum())
    if case.get("fused", True):  # views of one projection's rows
        rows = normal(t, hq + 2 * hkv, d)
        out.update(q=rows[:, :hq], k=rows[:, hq:hq + hkv], v=rows[:, hq + hkv:])
    else:
        out.update(q=normal(t, hq, d), k=normal(t, hkv, d), v=normal(t, hkv, d))
    if case["op"] == "attend":
        out["mask"] = ints(_tree_bits(s["parents"], -(-case["nodes"] // 32))) if case["tree"] else None
    else:
        out.update(angles=_angles(int((s["lens"] + s["n"]).max()) + 1, case["rot"]), interleaved=case["interleaved"])
    return out


def _tree_bits(parents, words):
    """int32 [T, words]: the node itself and its ancestors, a bit each (a program makes them once a step for all layers)."""
    rows = []
    for tree in parents:
        bits = []
        for i, p in enumerate(tree):
            bits.append((bits[p] if p >= 0 else 0) | 1 << i)
        rows += [[x >> 32 * w & 0xFFFFFFFF for w in range(words)] for x in bits]
    return np.array(rows, np.uint32).view(np.int32)


# ------------------------------------------------------------------------------------------------ the passes
def run(state):
    if own:
        return {"attend": _own_attend, "rotate": _own_rotate, "append": _own_append}[state["op"]](state)
    return {"attend": _plain_attend, "rotate": _plain_rotate, "append": _plain_append}[state["op"]](state)


def _own_attend(s):
    from io_aware_exact_04_gb300 import api
    o, lse = api.forward_tree(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"],
                              mask=s["mask"], scale=s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return {"o": o, "lse": lse}


def _own_rotate(s):
    from io_aware_exact_04_gb300 import api
    q, k = api.rotary_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"], s["angles"],
                             interleaved=s["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return _cache_outputs(s, q=q, k=k)


def _own_append(s):
    from io_aware_exact_04_gb300 import api
    api.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["cu"], rows=s["rows"],
                     k_scale=s["k_scale"], v_scale=s["v_scale"])
    return _cache_outputs(s)


def _cache_outputs(s, **more):
    out = {"k_cache": s["k_cache"], "v_cache": s["v_cache"], **more}
    if s["block"]:
        out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


def _plain_attend(s):
    cu, q, hkv = s["cu"].long(), s["q"], s["k"].shape[1]
    # a padded batch of the new tokens
    i = torch.arange(s["longest"], device=cu.device)
    there = i[None, :] < (cu[1:] - cu[:-1])[:, None]
    at = torch.where(there, cu[:-1, None] + i[None, :], 0)
    qq = q.float()[at].unflatten(2, (hkv, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [B, Hkv, G n, d]
    # keys and values: the context out of its pages, then the new tokens
    table = s["table"].long().clamp(min=0)
    k, v = (torch.cat([(s[c][table].float().unflatten(3, (-1, s["block"])) * s[z][table][..., None, None])
                       .flatten(3, 4).permute(0, 2, 1, 3, 4).flatten(2, 3), s[x].float()[at].transpose(1, 2)], 2)
            for c, z, x in (("k_cache", "k_scale", "k"), ("v_cache", "v_scale", "v")))
    if s["mask"] is None:
        nodes = (i[None, :] <= i[:, None]) & there[:, None, :]
    else:
        words = s["mask"].long()[at]
        nodes = ((words[:, :, i // 32] >> (i % 32)) & 1).bool() & there[:, None, :]
    c = torch.arange(k.shape[2] - s["longest"], device=cu.device) < s["lens"][:, None]
    seen = torch.cat([c[:, None, :].expand(-1, s["longest"], -1), nodes], -1)
    scores = torch.matmul(qq, k.transpose(-1, -2)).unflatten(2, (-1, s["longest"])) * s["scale"]
    scores = scores.masked_fill(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (-1, s["longest"])) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).squeeze(-1)
    return {"o": o.permute(0, 3, 1, 2, 4).flatten(2, 3)[there].to(q.dtype),
            "lse": lse.permute(0, 3, 1, 2).flatten(2, 3)[there].t().contiguous()}


def _places(s, count):
    """Sequence and position of each of the `count` packed tokens."""
    cu = s["cu"].long()
    t = torch.arange(count, device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, s["lens"].long()[b] + t - cu[b]


def _turned(x, angles, interleaved):
    """x [T, H, d] in 32 bits, its first `dim` elements rotated by the angles [T, dim] (cosines, then sines)."""
    half = angles.shape[1] // 2
    c, n = angles[:, None, :half], angles[:, None, half:]
    x = x.float()
    a, rest = x[..., : 2 * half], x[..., 2 * half:]
    x1, x2 = (a[..., ::2], a[..., 1::2]) if interleaved else (a[..., :half], a[..., half:])
    y1, y2 = x1 * c - x2 * n, x2 * c + x1 * n
    y = torch.stack([y1, y2], -1).flatten(-2) if interleaved else torch.cat([y1, y2], -1)
    return torch.cat([y, rest], -1)


def _store(s, k, v, b, at):
    """Rows k and v in 32 bits into the places `at` of the sequences `b`."""
    page, block = s["page"], s["block"]
    ids = s["table"].long()[b, at // page]
    if not block:
        s["k_cache"][ids, :, at % page] = k.to(s["k_cache"].dtype)
        s["v_cache"][ids, :, at % page] = v.to(s["v_cache"].dtype)
        return
    per = page // block
    of = ids * per + at % page // block  # the block of each token among all blocks
    for x, values, scales in ((k, s["k_cache"], s["k_scale"]), (v, s["v_cache"], s["v_scale"])):
        pool, hkv = scales.shape[:2]
        finite = torch.isfinite(x)
        most = torch.zeros((pool * per, hkv), dtype=torch.float32, device=x.device)
        most.index_reduce_(0, of, torch.where(finite, x.abs(), 0.0).amax(-1), "amax")
        first = torch.full((pool * per,), block, dtype=torch.int64, device=x.device)
        first.index_reduce_(0, of, at % block, "amin")  # the first new token of a block; `block`: none
        old = scales.transpose(1, 2).reshape(pool * per, hkv).double()
        fresh = (first == 0)[:, None] | ~(torch.isfinite(old) & (old > 0))
        old = torch.where(fresh, 1.0, old)
        m, e = torch.frexp(most.double() / old)  # least k with most <= 448 old 2^k
        k2 = torch.where(most > 0, e - 9 + (m > 0.875), -118).clamp(min=-118)
        k2 = torch.where(fresh, k2, k2.clamp(min=0))
        k2 = torch.where((first < block)[:, None], k2, 0)
        new = torch.where((first < block)[:, None], old * torch.exp2(k2.double()), scales.transpose(1, 2).reshape(pool * per, hkv).double())
        scales.copy_(new.float().reshape(pool, per, hkv).transpose(1, 2))
        grown = torch.where(fresh, 0, k2).reshape(pool, per, hkv).transpose(1, 2)
        kept = (torch.arange(block, device=x.device) < first[:, None]).reshape(pool, 1, per, block) & (grown > 0)[..., None]
        b8 = values.unflatten(2, (per, block))
        now = (b8.float() * torch.exp2(-grown.double()).float()[..., None, None]).to(values.dtype)
        values.copy_(torch.where(kept[..., None], now.float(), b8.float()).to(values.dtype).flatten(2, 3))
        values[ids, :, at % page] = torch.where(finite, x / new.float()[of][..., None], float("nan")).to(values.dtype)


def _plain_rotate(s):
    b, at = _places(s, s["k"].shape[0])
    angles = s["angles"][at]
    q, k = _turned(s["q"], angles, s["interleaved"]), _turned(s["k"], angles, s["interleaved"])
    _store(s, k, s["v"].float(), b, at)
    return _cache_outputs(s, q=q.to(s["q"].dtype), k=k.to(s["k"].dtype))


def _plain_append(s):
    rows = s["rows"]
    b, at = _places(s, s["k"].shape[0] if rows is None else rows.shape[0])
    k, v = (s[x].float() if rows is None else s[x].float()[rows.long()] for x in ("k", "v"))
    _store(s, k, v, b, at)
    return _cache_outputs(s)


# ------------------------------------------------------------------------------------------------ floors
def work(case):
    s = _plan(case)
    d, hq, hkv, block = case["d"], case["hq"], case["hkv"], case["block"]
    n, ctx = s["n"].astype(np.float64), s["lens"].astype(np.float64)
    if case["op"] == "attend":
        live = n > 0
        seen = (n * (n + 1) / 2).sum()
        if case["tree"]:
            seen = 0
            for tree in s["parents"]:
                depth = []
                for p in tree:
                    depth.append(1 + (depth[p] if p >= 0 else 0))
                seen += sum(depth)
        cached = 2 * hkv * (d * ctx[live].sum() + 4 * np.ceil(ctx[live] / block).sum())
        return {"bytes": float(cached + n.sum() * (2 * hkv * 2 * d + hq * (4 * d + 4)) + 4 * s["pages"][live].sum()),
                "flops": float(4 * d * hq * ((n * ctx).sum() + seen))}
    t = n.sum()
    if block:  # a block's values and scale are written (and, where it has tokens already, its scale is read)
        blocks = (np.ceil((ctx + n) / block) - np.floor(ctx / block))[n > 0].sum()
        kv = 2 * hkv * (t * 3 * d + 4 * (blocks + ((ctx % block > 0) & (n > 0)).sum()))
    else:
        kv = 2 * hkv * t * 4 * d
    if case["op"] == "append":
        return {"bytes": float(kv), "flops": float(2 * hkv * t * d * 2)}
    places = len(np.unique(np.concatenate([np.arange(a, a + k) for a, k in zip(s["lens"], s["n"])])))
    return {"bytes": float(kv + t * (hq * 4 * d + hkv * 2 * d) + places * 4 * case["rot"]),
            "flops": float(3 * t * (hq + hkv) * case["rot"] + (2 * hkv * t * d * 2 if block else 0))}


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "rotate": _exact_rotate, "append": _exact_append}[case["op"]](s, case)


def _exact_attend(s, case):
    cu, lens, parents = s["cu"].tolist(), s["lens"].tolist(), _plan(case)["parents"]
    q, group = s["q"], s["q"].shape[1] // s["k"].shape[1]
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.zeros((q.shape[1], q.shape[0]), dtype=torch.float64, device=q.device)
    for b, length in enumerate(lens):
        lo, hi = cu[b], cu[b + 1]
        if lo == hi:
            continue
        seen = np.ones((hi - lo, length + hi - lo), bool)
        for i in range(hi - lo):
            line, j = {i}, i
            while j >= 0:
                line.add(j)
                j = parents[b][j] if case["tree"] else j - 1
            seen[i, length:] = [x in line for x in range(hi - lo)]
        seen = torch.from_numpy(seen).to(q.device)
        ids = s["table"][b, : -(-length // case["page"])].long()
        for h in range(s["k"].shape[1]):
            keys, values = (torch.cat([(s[c].index_select(0, ids)[:, h].double()
                                        * s[z].index_select(0, ids)[:, h].double().repeat_interleave(case["block"], 1)[..., None])
                                       .flatten(0, 1)[:length], s[x][lo:hi, h].double()])
                            for c, z, x in (("k_cache", "k_scale", "k"), ("v_cache", "v_scale", "v")))
            for r in range(h * group, (h + 1) * group):
                x = (q[lo:hi, r].double() @ keys.t()) * s["scale"]
                x[~seen] = -math.inf
                lse[r, lo:hi] = torch.logsumexp(x, -1)
                o[lo:hi, r] = torch.exp(x - lse[r, lo:hi, None]) @ values
    return {"o": o, "lse": lse}


def _exact_turn(x, positions, case):
    """Rotation in complex numbers, angles from the positions anew."""
    dim = case["rot"]
    f = BASE ** (-np.arange(0, dim, 2, dtype=np.float64) / dim)
    w = torch.from_numpy(np.exp(1j * np.asarray(positions, np.float64)[:, None] * f[None, :])).to(x.device)[:, None, :]
    y = x.double().clone()
    a = slice(0, dim, 2) if case["interleaved"] else slice(0, dim // 2)
    b = slice(1, dim, 2) if case["interleaved"] else slice(dim // 2, dim)
    z = torch.complex(y[..., a].contiguous(), y[..., b].contiguous()) * w
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_store(s, case, k, v, rows):
    """The pages after rows k and v (in 64 bits) went in, sequence by sequence, block by block."""
    page, block = case["page"], case["block"]
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    out = {}
    for x, c, z in ((k, "k_cache", "k_scale"), (v, "v_cache", "v_scale")):
        values = s[c].double().clone()
        scales = s[z].double().clone() if block else None
        for b, start in enumerate(lens):
            n, i = cu[b + 1] - cu[b], 0
            while i < n:
                at = start + i
                step = min(n - i, (block or page) - at % (block or page))
                p, r = table[b][at // page], at % page
                new = x[torch.tensor([rows[cu[b] + i + j] for j in range(step)], device=x.device)].transpose(0, 1)  # [H, step, d]
                if block:
                    w = r // block
                    for_all = new.abs().amax((1, 2)) / 448.0
                    least = torch.exp2(torch.ceil(torch.log2(for_all)))
                    if at % block:
                        was = scales[p, :, w].clone()
                        least = was * torch.exp2(torch.ceil(torch.log2(for_all / was)).clamp(min=0))
                        kept = values[p, :, w * block: r] * (was / least)[:, None, None]
                        values[p, :, w * block: r] = kept.float().to(E4M3).double()
                    scales[p, :, w] = least
                    new = (new / least[:, None, None]).float().to(E4M3).double()
                values[p, :, r: r + step] = new
                i += step
        out[c] = values
        if block:
            out[z] = scales
    return out


def _exact_rotate(s, case):
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    at = np.concatenate([np.arange(a, a + cu[b + 1] - cu[b]) for b, a in enumerate(lens)])
    q, k = _exact_turn(s["q"], at, case), _exact_turn(s["k"], at, case)
    return {"q": q, "k": k, **_exact_store(s, case, k, s["v"].double(), list(range(cu[-1])))}


def _exact_append(s, case):
    rows = list(range(s["k"].shape[0])) if s["rows"] is None else s["rows"].tolist()
    return _exact_store(s, case, s["k"].double(), s["v"].double(), rows)
