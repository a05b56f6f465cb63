"""Plain 64-bit forms of the serving operators, for their tests: attention row by row from the
definition, and the cache's bookkeeping on Python lists."""

import math

import numpy as np
import torch

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative to the value


def offsets(lens):
    return [0] + list(np.cumsum(lens).tolist())


def attention(q, k, v, seen, scale):
    """O, LSE and the error bounds of both for one head: q [n, d], k and v [m, d], seen [n, m] bool.

    The bounds: the kernels form scores with fp32 sums of d exact products (error at most d 2^-24
    of the sum of magnitudes, doubled for the scaling and the exponential's own error, 2^-20 in all),
    round P to the inputs' type before the product with V (half a step of each p), keep every sum in
    fp32 and round O once. So with delta the relative error of a p,
      |dLSE| <= delta + 2^-22 |LSE|,   |dO| <= (unit + 2 delta) sum p |v| + unit |O|."""
    q, k, v = q.double(), k.double(), v.double()
    unit = UNIT_OF[0]
    k = torch.where(seen.any(0)[:, None], k, 0.0)  # what nobody sees may hold anything
    v = torch.where(seen.any(0)[:, None], v, 0.0)
    s = torch.where(seen, (q @ k.t()) * scale, -math.inf)
    top = s.amax(1, keepdim=True) if s.shape[1] else torch.full((s.shape[0], 1), -math.inf, dtype=s.dtype, device=s.device)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(s - top)
    total = p.sum(1, keepdim=True)
    p = p / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total))[:, 0]
    o = p @ v
    mag = torch.where(seen, (q.abs() @ k.abs().t()) * scale, 0.0)
    mag = mag.amax(1) if mag.shape[1] else torch.zeros(q.shape[0], dtype=q.dtype, device=q.device)
    delta = q.shape[1] * 2.0 ** -23 * mag + 2.0 ** -19
    dl = delta + 2.0 ** -22 * torch.where(torch.isinf(lse), 0.0, lse.abs())
    do = (unit + 2 * delta[:, None]) * (p @ v.abs()) + unit * o.abs()
    return o, lse, do, dl


UNIT_OF = [2.0 ** -8]


def rows_of_cache(cache, table, b, length):
    """[length, Hkv, d] of sequence b out of its pages."""
    page = cache.shape[2]
    ids = table[b, : -(-length // page)].long()
    return cache[ids].transpose(1, 2).flatten(0, 1)[:length]


def forward(q, k, v, lens_new, scale, ctx=None, seen_nodes=None):
    """O [T, Hq, d], LSE [Hq, T] and their bounds over packed sequences. ctx(b): the cached K and V rows
    [L, Hkv, d] of sequence b; seen_nodes(b, n): bool [n, n], a chain by default."""
    UNIT_OF[0] = UNIT[q.dtype]
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    o = torch.zeros((T, Hq, d), dtype=torch.float64, device=q.device)
    lse = torch.zeros((Hq, T), dtype=torch.float64, device=q.device)
    do, dl = torch.zeros_like(o), torch.zeros_like(lse)
    at = offsets(lens_new)
    for b, n in enumerate(lens_new):
        if n == 0:
            continue
        lo, hi = at[b], at[b + 1]
        kk, vv = k[lo:hi], v[lo:hi]
        nodes = torch.ones((n, n), dtype=torch.bool, device=q.device).tril() if seen_nodes is None else seen_nodes(b, n)
        if ctx is not None:
            ck, cv = ctx(b)
            kk, vv = torch.cat([ck, kk]), torch.cat([cv, vv])
            nodes = torch.cat([torch.ones((n, ck.shape[0]), dtype=torch.bool, device=q.device), nodes.to(q.device)], 1)
        for h in range(Hq):
            o[lo:hi, h], lse[h, lo:hi], do[lo:hi, h], dl[h, lo:hi] = attention(q[lo:hi, h], kk[:, h // G], vv[:, h // G],
                                                                              nodes, scale)
    return o, lse, do, dl


def assert_close(o, lse, want, rows):
    """Rows [0, rows) within their bounds; -inf exactly where it belongs."""
    ro, rl, do, dl = want
    assert torch.equal(torch.isneginf(lse[:, :rows]), torch.isneginf(rl[:, :rows])), "LSE -inf pattern differs"
    fin = ~torch.isneginf(rl[:, :rows])
    el = (lse[:, :rows].double() - rl[:, :rows])[fin].abs() - dl[:, :rows][fin]
    assert not torch.isnan(lse[:, :rows]).any()
    assert el.numel() == 0 or float(el.max()) <= 0, f"LSE beyond its bound by {float(el.max())}"
    eo = (o[:rows].double() - ro[:rows]).abs() - do[:rows]
    assert not torch.isnan(o[:rows].float()).any(), "NaN in O"
    assert eo.numel() == 0 or float(eo.max()) <= 1e-12, f"O beyond its bound by {float(eo.max())}"


def ancestors(parents):
    """bool [n, n]: i sees j for j = i, its parent, its parent's parent, ..."""
    n = len(parents)
    seen = torch.zeros((n, n), dtype=torch.bool)
    for i in range(n):
        j = i
        while j >= 0:
            seen[i, j] = True
            j = parents[j] if parents[j] < j else -1
    return seen


def pack_bits(seen, words):
    """bool [n, m] -> int32 [n, words], bit j % 32 of word j / 32."""
    n, m = seen.shape
    bits = np.zeros((n, 32 * words), bool)
    w = min(m, 32 * words)
    bits[:, :w] = seen[:, :w].cpu().numpy()
    return torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy())


def update(kv, table, lens, src, new, page):
    """cache_update on Python lists; kv [planes, pages, H, page, d] is changed in place."""
    slots, width, pool = len(lens), len(table[0]), kv.shape[1]
    busy = {p for s in range(slots) for p in table[s][: -(-lens[s] // page)]}
    free = [p for p in range(pool) if p not in busy]
    keep = [min(new[s], lens[src[s]]) for s in range(slots)]
    holders = {}
    for s in range(slots):
        for j in range(-(-keep[s] // page) if src[s] == s else keep[s] // page):
            holders[table[src[s]][j]] = holders.get(table[src[s]][j], 0) + 1
    made, copies, taken = [], [], 0
    for s in range(slots):
        row = table[src[s]][: keep[s] // page]
        if keep[s] % page:
            p = table[src[s]][keep[s] // page]
            if src[s] == s and holders[p] == 1:
                row = row + [p]
            else:
                copies.append((s, len(row), p, keep[s] % page))
        while len(row) < -(-new[s] // page):
            row = row + [free[taken] if taken < len(free) else -1]
            taken += 1
        made.append(row + [-1] * (width - len(row)))
    info = [taken, len(free)]
    if taken > len(free):
        return table, lens, info
    before = kv.clone()
    for s, j, p, rows in copies:
        kv[:, made[s][j], :, :rows] = before[:, p, :, :rows]
    return made, list(new), info


def compact(kv, table, lens, page):
    busy = sorted({p for s in range(len(lens)) for p in table[s][: -(-lens[s] // page)]})
    there, n = set(busy), len(busy)
    goes = dict(zip([p for p in busy if p >= n], [p for p in range(n) if p not in there]))
    before = kv.clone()
    for of, to in goes.items():
        kv[:, to] = before[:, of]
    made = [[goes.get(p, p) if j * page < lens[s] else p for j, p in enumerate(row)] for s, row in enumerate(table)]
    return made, [n, len(goes)]
