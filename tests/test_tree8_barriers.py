"""The barriers of the few-row attention kernel over a cache in 8 bits (csrc/fa_serve8.cu), stepped on the CPU, and
how its CTAs share the tiles.

A model of one CTA: the scheduler with K's loads, the loaders of V and of the scales, the two warps that split Q, the
issuer of S, the two issuers of P V and the eight softmax warps as coroutines, with the kernel's barriers (counts,
phases, parities), its rings and tensor memory. Copies land and tensor work completes at random times, the latter in
order. Random items, scheduled at random, must run to their end, and the model fails where
- a barrier gets more arrivals than its phase expects;
- a wait by parity would take another use of the barrier for its own;
- a reader finds another tile, score tile, P, O, Q slot, statistics or descriptor than the one it is at;
- nothing can run.
"""

import random

import pytest

from tests.test_serving_barriers import Bar, Fault

NQ = 4


def draw_items(r):
    items = []
    for _ in range(r.randint(1, 12)):
        cnt = r.choice([1, 1, 1, 2, 2, 3, 4, 5, 8, 9])
        dual = r.random() < 0.6
        # the first lane's rows see no more tiles than the second's; none in a cut item's last part
        c = ((cnt + 1) // 2, cnt // 2) if dual else (r.choice([0, cnt, max(0, cnt - 1), r.randint(0, cnt)]), cnt)
        own = [[(k & 1) == t if dual else k < c[t] for k in range(cnt)] for t in range(2)]
        items.append(dict(cnt=cnt, dual=dual, c=c, own=own))
    return items


def simulate(seed, one_p_ready=False, skip_other_q=False, p_unguarded=False, owner_twice=False, own_q_twice=False):
    """one_p_ready, skip_other_q, p_unguarded, owner_twice, own_q_twice: mistakes to plant (a single barrier for both buffers of P; a
    softmax warp that waits for its own lane's Q only; P written without a wait for the product that reads the buffer; a
    tile let go by the issuer that takes it alone, so that the other one may fall two uses of its slot behind; a
    slot of Q let go by the lane whose rows it holds alone, likewise)."""
    r = random.Random(seed)
    NT = r.choice([2, 3, 6, 11])
    FULL = [Bar(10, f"FULL {i}") for i in range(NT)]
    EMPTY = [Bar(2, f"EMPTY {i}") for i in range(NT)]
    Q_FULL = [Bar(2, f"Q_FULL {i}") for i in range(NQ)]
    Q_EMPTY = [Bar(9, f"Q_EMPTY {i}") for i in range(NQ)]
    S_FULL, S_FREE, P_READY, O_DONE = ([[Bar(c, f"{n} {t} {u}") for u in range(2)] for t in range(2)]
                                       for n, c in (("S_FULL", 1), ("S_FREE", 4), ("P_READY", 4), ("O_DONE", 1)))
    O_FREE, GROUP = ([Bar(c, f"{n} {t}") for t in range(2)] for n, c in (("O_FREE", 8), ("GROUP", 4)))
    MERGE = Bar(8, "MERGE")
    D_FULL, D_EMPTY = ([Bar(c, f"{n} {i}") for i in range(4)] for n, c in (("D_FULL", 1), ("D_EMPTY", 15)))
    items = draw_items(r)
    kv = [[None] * NT, [None] * NT, [None] * NT]  # K, V and the scales of the ring's entries
    q_slots, descs = [[None, None] for _ in range(NQ)], [None] * 4
    S, P, O = [[None] * 2, [None] * 2], [[[None] * 4 for _ in range(2)] for _ in range(2)], [None, None]
    s_left = [{}, {}]           # warps that have taken a score tile into registers
    stats = [[None] * 4, [None] * 4]  # the item whose sums a warp has left
    moved = {}
    copies, tensor = [], []

    def wait(bar, n):
        return lambda: bar.ready(n)

    def next_item(i):
        yield wait(D_FULL[i & 3], i >> 2)
        if descs[i & 3] != i:
            raise Fault(f"descriptor of item {descs[i & 3]} read as that of {i}")
        D_EMPTY[i & 3].arrive()

    def load(it, which, e):
        for _ in range(it["cnt"]):
            if e >= NT:
                yield wait(EMPTY[e % NT], e // NT - 1)
            kv[which][e % NT] = None
            FULL[e % NT].expect()
            copies.append((FULL[e % NT], kv[which], e % NT, e))
            e += 1
            yield None

    def scheduler():
        e = 0
        for i, it in enumerate(items + [None]):
            if i >= 4:
                yield wait(D_EMPTY[i & 3], (i >> 2) - 1)
            descs[i & 3] = i
            D_FULL[i & 3].arrive()
            if it is None:
                return
            yield from load(it, 0, e)
            e += it["cnt"]

    def load_v():
        e = 0
        for i, it in enumerate(items + [None]):
            yield from next_item(i)
            if it is None:
                return
            yield from load(it, 1, e)
            e += it["cnt"]

    def scales():
        e = 0
        for i, it in enumerate(items + [None]):
            yield from next_item(i)
            if it is None:
                return
            for _ in range(it["cnt"]):
                if e >= NT:
                    yield wait(EMPTY[e % NT], e // NT - 1)
                kv[2][e % NT] = e
                FULL[e % NT].arrive(8)
                e += 1
                yield None

    def split(half):
        uq = 0
        for i, it in enumerate(items + [None]):
            yield from next_item(i)
            if it is None:
                return
            for _ in range(1 if it["dual"] else 2):
                if uq >= NQ:
                    yield wait(Q_EMPTY[uq % NQ], uq // NQ - 1)
                q_slots[uq % NQ][half] = uq
                yield None
                Q_FULL[uq % NQ].arrive()
                uq += 1

    def s_both():
        e = uq = 0
        g = [0, 0]
        for i, it in enumerate(items + [None]):
            yield from next_item(i)
            if it is None:
                return
            nq = 1 if it["dual"] else 2
            for u in range(uq, uq + nq):
                yield wait(Q_FULL[u % NQ], u // NQ)
            for k in range(it["cnt"]):
                yield wait(FULL[e % NT], e // NT)
                for t in range(2):
                    if not it["own"][t][k]:
                        continue
                    x = g[t]
                    if x > 1:
                        yield wait(S_FREE[t][x & 1], (x >> 1) - 1)
                    tensor.append(("S", t, x, e, uq if it["dual"] else uq + t))
                    tensor.append(("commit", S_FULL[t][x & 1]))
                    g[t] += 1
                    yield None
                e += 1
            for u in range(uq, uq + nq):
                tensor.append(("commit", Q_EMPTY[u % NQ]))
            uq += nq

    def pv(t):
        e = g = used = 0
        for i, it in enumerate(items + [None]):
            yield from next_item(i)
            if it is None:
                return
            first = True
            for k in range(it["cnt"]):
                yield wait(FULL[e % NT], e // NT)
                if kv[1][e % NT] != e:
                    raise Fault(f"V of entry {e} is not there")
                if not it["own"][t][k]:
                    if not (owner_twice and it["dual"]):
                        EMPTY[e % NT].arrive()
                    e += 1
                    yield None
                    continue
                yield wait(P_READY[t][0], g) if one_p_ready else wait(P_READY[t][g & 1], g >> 1)
                if first and used > 0:
                    yield wait(O_FREE[t], used - 1)
                tensor.append(("PV", t, g, e, first))
                tensor.append(("commit", O_DONE[t][g & 1]))
                tensor.append(("commit", EMPTY[e % NT]))
                if owner_twice and it["dual"]:
                    tensor.append(("commit", EMPTY[e % NT]))
                g, first, e = g + 1, False, e + 1
                yield None
            used += it["c"][t] > 0

    def softmax(t, w):
        uq = g = e0 = meets = merges = 0
        for i, it in enumerate(items + [None]):
            yield from next_item(i)
            if it is None:
                return
            dual, steps = it["dual"], it["c"][t]
            slot = uq + (0 if dual else t)
            for u in ([slot] if skip_other_q else range(uq, uq + (1 if dual else 2))):
                yield wait(Q_FULL[u % NQ], u // NQ)
            if q_slots[slot % NQ] != [slot, slot]:
                raise Fault(f"Q of use {slot} is not there")
            if not dual and not own_q_twice:
                Q_EMPTY[(uq + (t ^ 1)) % NQ].arrive()
            mine = [k for k in range(it["cnt"]) if it["own"][t][k]]
            for s, k in enumerate(mine):
                yield wait(S_FULL[t][g & 1], g >> 1)
                if S[t][g & 1] != g or kv[2][(e0 + k) % NT] != e0 + k:
                    raise Fault(f"S or the scales of step {g} are not there")
                if g >= 2 and not p_unguarded:
                    yield wait(O_DONE[t][g & 1], (g - 2) >> 1)
                moves = s == 0
                if not moves:  # the vote
                    GROUP[t].arrive()
                    yield None
                    yield wait(GROUP[t], meets)
                    meets += 1
                    moves = moved.setdefault((t, g), r.random() < 0.3)
                if moves:
                    for _ in range(2):
                        GROUP[t].arrive()
                        yield None
                        yield wait(GROUP[t], meets)
                        meets += 1
                    if s > 0:
                        yield wait(O_DONE[t][(g - 1) & 1], (g - 1) >> 1)
                        if O[t] != g - 1:
                            raise Fault(f"O of step {O[t]} rescaled as that of {g - 1}")
                s_left[t][g] = s_left[t].get(g, 0) + 1
                S_FREE[t][g & 1].arrive()
                yield None
                P[t][g & 1][w] = g
                yield None
                (P_READY[t][0] if one_p_ready else P_READY[t][g & 1]).arrive()
                g += 1
                yield None
            if steps > 0:
                yield wait(O_DONE[t][(g - 1) & 1], (g - 1) >> 1)
                stats[t][w] = i
                yield None
                join = dual and it["c"][1] > 0
                if join:
                    MERGE.arrive()
                    yield None
                    yield wait(MERGE, merges)
                    merges += 1
                else:
                    GROUP[t].arrive()
                    yield None
                    yield wait(GROUP[t], meets)
                    meets += 1
                for x in (0, 1) if join else (t,):
                    if stats[x] != [i] * 4:
                        raise Fault(f"the statistics of items {stats[x]} read as those of {i}")
                if O[t] != g - 1:
                    raise Fault(f"O of step {O[t]} stored as that of {g - 1}")
                yield None
                if any(stats[x] != [i] * 4 for x in ((0, 1) if join else (t,))):
                    raise Fault("statistics written over while they were read")
                O_FREE[t].arrive(1 if join else 2)
                if join:
                    O_FREE[t ^ 1].arrive()
            yield None
            if q_slots[slot % NQ] != [slot, slot]:
                raise Fault(f"Q of use {slot} was written over")
            Q_EMPTY[slot % NQ].arrive(2 if own_q_twice and not dual else 1)
            uq += 1 if dual else 2
            e0 += it["cnt"]

    def complete(x):
        if x[0] == "commit":
            x[1].arrive()
        elif x[0] == "S":
            _, t, g, e, q = x
            if kv[0][e % NT] != e or q_slots[q % NQ] != [q, q]:
                raise Fault(f"S of step {g} reads K or Q that is not there")
            if g > 1 and s_left[t].get(g - 2) != 4:
                raise Fault(f"S of step {g - 2} written over while it was read")
            S[t][g & 1] = g
        else:
            _, t, g, e, first = x
            if kv[1][e % NT] != e:
                raise Fault(f"P V of step {g} reads V that is not there")
            if P[t][g & 1] != [g] * 4:
                raise Fault(f"P of step {g} was written over")
            if not first and O[t] != g - 1:
                raise Fault(f"O of step {O[t]} goes on with step {g}")
            O[t] = g

    roles = {"scheduler": scheduler(), "V": load_v(), "scales": scales(), "S": s_both(), "PV 0": pv(0), "PV 1": pv(1)}
    roles.update({f"split {h}": split(h) for h in range(2)})
    roles.update({f"softmax {t} {w}": softmax(t, w) for t in range(2) for w in range(4)})
    waits = dict.fromkeys(roles)
    weight = {k: r.choice([1, 1, 5, 20]) for k in roles}
    weight["copies"], weight["tensor"] = r.choice([1, 5, 30]), r.choice([1, 5, 30])
    while roles or copies or tensor:
        can = [k for k in roles if waits[k] is None or waits[k]()]
        can += ["copies"] * bool(copies) + ["tensor"] * bool(tensor)
        if not can:
            raise Fault(f"nothing can run: {sorted(roles)}")
        k = r.choices(can, [weight[x] for x in can])[0]
        if k == "copies":
            bar, where, at, what = copies.pop(r.randrange(min(len(copies), 4)))
            where[at] = what
            bar.land()
        elif k == "tensor":
            complete(tensor.pop(0))
        else:
            try:
                waits[k] = next(roles[k])
            except StopIteration:
                del roles[k], waits[k]


@pytest.mark.parametrize("block", range(4))
def test_every_schedule_ends(block):
    for seed in range(60 * block, 60 * block + 60):
        simulate(seed)


@pytest.mark.parametrize("mistake", [dict(one_p_ready=True), dict(skip_other_q=True), dict(p_unguarded=True),
                                     dict(owner_twice=True), dict(own_q_twice=True)],
                         ids=["one_barrier_for_two_buffers", "a_slot_left_out", "p_without_a_wait", "let_go_by_one", "q_let_go_by_one"])
def test_the_model_finds_mistakes(mistake):
    found = 0
    for seed in range(400):
        try:
            simulate(seed, **mistake)
        except Fault:
            found += 1
        if found:
            break
    assert found > 0


def share(sizes, heads, grid, cost, least=2):
    """The parts of items, as the CTAs of a grid take them: (CTA, item, first tile, tiles, slot of its partial result).
    sizes: of each sequence, the tiles of its items, one for each unit of rows (the last has the most)."""
    spans = [max(s) + cost for s in sizes if s]
    total = sum(len(s) * heads * sp for s, sp in zip([s for s in sizes if s], spans))
    ctas = grid if total >= grid * least else max(1, (total + least - 1) // least)
    base, rest = divmod(total, ctas)
    start = [base * c + min(c, rest) for c in range(ctas + 1)]
    starts, at = [], 0
    for s, sp in zip([s for s in sizes if s], spans):
        for most in s:
            for _ in range(heads):
                starts.append((at, most, sp))
                at += sp
    parts, cuts = [], {}
    for c in range(ctas):
        pos, first = start[c], True
        for item, (at, most, sp) in enumerate(starts):
            if pos >= start[c + 1] or at + sp <= pos or at >= start[c + 1]:
                continue
            x0, x1 = pos - at, min(sp, start[c + 1] - at)
            j0, j1 = max(0, x0 - cost), min(max(0, x1 - cost), most)
            n = max(0, j1 - j0)
            tile0 = at + cost
            if j0 > 0 and n > 0 and start[c - 1] <= tile0:
                assert first, "only a CTA's first item may be cut by its start"
                cuts[c] = (item, 1 + sum(start[k] < tile0 + most for k in range(c, ctas)))
            if n:
                parts.append((c, item, j0, n, 2 * c + (j0 == 0), n == most))
            first = False
            pos = at + sp
    return starts, parts, cuts


def test_every_tile_is_taken_once_and_every_part_is_joined():
    r = random.Random(3)
    for trial in range(400):
        grid, heads, cost = r.choice([1, 2, 7, 152]), r.choice([1, 2, 8]), r.choice([4, 8])
        sizes = [sorted(r.choice([1, 2, 5, 40]) + r.randint(0, 2) for _ in range(r.choice([0, 1, 1, 3]))) for _ in range(r.randint(1, 12))]
        if not any(sizes):
            continue
        starts, parts, cuts = share(sizes, heads, grid, cost)
        for item, (_, most, _) in enumerate(starts):
            mine = sorted((j0, n, c, slot, whole) for c, i, j0, n, slot, whole in parts if i == item)
            assert sum(n for _, n, *_ in mine) == most and mine[0][0] == 0
            assert all(a[0] + a[1] == b[0] and b[2] == a[2] + 1 for a, b in zip(mine, mine[1:]))
            joins = [(c, k) for c, (i, k) in cuts.items() if i == item]
            if len(mine) == 1:
                assert mine[0][4] and not joins
            else:  # one CTA boundary joins: its slots are part 0's and then those of the CTAs that follow
                (c, k), = joins
                assert k == len(mine)
                assert [x[3] for x in mine] == [2 * (c - 1) + 1] + [2 * (c - 1 + x) for x in range(1, k)]
        slots = [slot for _, _, _, _, slot, whole in parts if not whole]
        assert len(slots) == len(set(slots))
