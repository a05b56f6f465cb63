"""The barriers of the many-row attention kernel over a cache in 8 bits (csrc/fa_serve.cu with C8), stepped on the CPU.

A model of one CTA: the producer, the four converters, the issuer of S, the two issuers of P V and the eight softmax
warps as coroutines, with the kernel's barriers (counts, phases, parities), both rings (pages of 8 bits; 16-bit tiles, K
and V in slots of their own), the kept scales and factors, the Q slots and tensor memory. Copies land and tensor work
completes at random times, the latter in order. Random items, scheduled at random, must run to their end, and the model
fails where
- a barrier gets more arrivals than its phase expects;
- a wait by parity would take another use of the barrier for its own;
- a reader finds another page, tile, scale, factor, score tile, P, O, Q slot or descriptor than the one it is at;
- nothing can run.

TURN is bf16, whose queries and new tokens the converters bring to fp16. Slots: 10 and 12 at d = 64, 6 and 6 at d = 128.
"""

import random

import pytest

from tests.test_serving_barriers import Bar, Fault


def draw_items(r):
    items = []
    for _ in range(r.randint(1, 12)):
        cnt = r.choice([1, 1, 1, 2, 2, 3, 4, 5, 8, 9, 14, 20])
        dual = r.random() < 0.5
        # the first lane's tokens see no more tiles than the second's; none in a cut item's last part
        c = ((cnt + 1) // 2, cnt // 2) if dual else (r.choice([0, cnt, max(0, cnt - 1), r.randint(0, cnt)]), cnt)
        own = [[(k & 1) == t if dual else k < c[t] for k in range(cnt)] for t in range(2)]
        rows = [[r.random() < 0.6 for _ in range(4)] for _ in range(2)]  # warps with a row
        if dual:
            rows[1] = rows[0]
        items.append(dict(cnt=cnt, dual=dual, c=c, own=own, rows=rows, cached=max(0, cnt - r.choice([0, 1, 1, 2, 8, 20]))))
    return items


def simulate(seed, keep=16, k_alone=False, skip_other_q=False, own_q_twice=False, unwaited_skip=False):
    """keep: tiles whose scales and factors are kept (16). k_alone, skip_other_q, own_q_twice, unwaited_skip: mistakes to
    plant (K's entry of a new tile full without the converters of V; a softmax warp that waits for its own lane's Q
    only; a slot of Q let go by the lane whose rows it holds alone; a tile let go unwaited by the issuer that does not
    take it)."""
    r = random.Random(seed)
    turn = r.random() < 0.6
    NSLOT, NS8 = r.choice([(10, 12), (6, 6)])
    FULL = [Bar(4, f"FULL {i}") for i in range(NSLOT)]
    EMPTY = [Bar(2, f"EMPTY {i}") for i in range(NSLOT)]
    FULL8 = [Bar(1 if i & 1 else 9, f"FULL8 {i}") for i in range(NS8)]
    EMPTY8 = [Bar(2, f"EMPTY8 {i}") for i in range(NS8)]
    NEW_RAW = [Bar(1, f"NEW_RAW {i}") for i in range(NSLOT)]
    Q_RAW = [Bar(1, f"Q_RAW {i}") for i in range(2)]
    Q_FULL = [Bar(4 if turn else 1, f"Q_FULL {i}") for i in range(2)]
    Q_EMPTY = [Bar(9 if turn else 1, f"Q_EMPTY {i}") for i in range(2)]
    S_FULL, P_READY, O_DONE = ([[Bar(c, f"{n} {t} {u}") for u in range(2)] for t in range(2)]
                               for n, c in (("S_FULL", 1), ("P_READY", 4), ("O_DONE", 1)))
    O_FREE = [Bar(8, f"O_FREE {t}") for t in range(2)]
    MERGE = Bar(8, "MERGE")
    D_FULL, D_EMPTY = ([Bar(c, f"{n} {i}") for i in range(4)] for n, c in (("D_FULL", 1), ("D_EMPTY", 15)))
    items = draw_items(r)
    descs = [None] * 4
    pages = [None] * NS8                              # the cached tile whose K or V lies in a slot of 8 bits
    ring = [[None, None] for _ in range(NSLOT)]       # the tile of which a slot holds both halves of the keys
    raw_ring = [None] * NSLOT                         # new tokens as they arrive
    raw_q, q_slots = [None] * 2, [[None] * 4 for _ in range(2)]
    scales, factors = [None] * keep, [[None] * 4 for _ in range(keep)]
    S, P, O = [[None] * 2, [None] * 2], [[None] * 2, [None] * 2], [None, None]
    stats, copies, tensor = [[None] * 4, [None] * 4], [], []

    def wait(bar, n):
        return lambda: bar.ready(n)

    def next_item(i):
        yield wait(D_FULL[i & 3], i >> 2)
        if descs[i & 3] != i:
            raise Fault(f"descriptor of item {descs[i & 3]} read as that of {i}")
        D_EMPTY[i & 3].arrive()

    def copy(bar, where, at, what):
        bar.expect()
        copies.append((bar.land, where, at, what))

    def producer():
        e = uq = 0
        for i, it in enumerate(items + [None]):
            if i >= 4:
                yield wait(D_EMPTY[i & 3], (i >> 2) - 1)
            descs[i & 3] = i
            D_FULL[i & 3].arrive()
            if it is None:
                return
            for _ in range(1 if it["dual"] else 2):
                if uq >= 2:
                    yield wait(Q_EMPTY[uq & 1], (uq >> 1) - 1)
                q_slots[uq & 1] = [None] * 4
                if turn:
                    copy(Q_RAW[uq & 1], raw_q, uq & 1, uq)
                else:
                    copy(Q_FULL[uq & 1], q_slots, uq & 1, [uq] * 4)
                uq += 1
                yield None
            for _ in range(it["cached"]):
                sk = 2 * e % NS8
                if 2 * e >= NS8:
                    yield wait(EMPTY8[sk], 2 * e // NS8 - 1)
                    yield wait(EMPTY8[sk + 1], 2 * e // NS8 - 1)
                pages[sk] = pages[sk + 1] = None
                copy(FULL8[sk], pages, sk, e)
                copy(FULL8[sk + 1], pages, sk + 1, e)
                scales[e % keep] = None
                for _ in range(8):
                    copies.append((FULL8[sk].arrive, scales, e % keep, e))
                e += 1
                yield None

    def converter(kv, half):
        x = uq = news = g = 0  # cached tiles, Q slots, new tiles and all tiles so far
        raws = [0] * NSLOT     # uses of each slot for new tokens
        for i, it in enumerate(items + [None]):
            yield from next_item(i)
            if it is None:
                return
            for _ in range((1 if it["dual"] else 2) if turn else 0):
                yield wait(Q_RAW[uq & 1], uq >> 1)
                if raw_q[uq & 1] != uq:
                    raise Fault(f"Q of use {uq} is not there")
                yield None
                q_slots[uq & 1][2 * kv + half] = uq
                Q_FULL[uq & 1].arrive()
                uq += 1
            for k in range(it["cnt"]):
                slot, use = 2 * (g % (NSLOT // 2)) + kv, g // (NSLOT // 2)
                if k < it["cached"]:
                    s8 = (2 * x + kv) % NS8
                    yield wait(FULL8[s8], (2 * x + kv) // NS8)
                    if use:
                        yield wait(EMPTY[slot], use - 1)
                    if pages[s8] != x:
                        raise Fault(f"the page of tile {x} is not there")
                    ring[slot][half] = None
                    yield None
                    if pages[s8] != x:
                        raise Fault(f"the page of tile {x} was written over")
                    ring[slot][half] = g
                    FULL[slot].arrive(2)
                    EMPTY8[s8].arrive()
                    x += 1
                else:
                    if use:
                        yield wait(EMPTY[slot], use - 1)
                    ring[slot][half] = None
                    if half == 0:
                        copy(NEW_RAW[slot], raw_ring, slot, g)
                    yield None
                    yield wait(NEW_RAW[slot], raws[slot])
                    raws[slot] += 1
                    if raw_ring[slot] != g:
                        raise Fault(f"the new tokens of tile {g} are not there")
                    yield None
                    ring[slot][half] = g
                    factors[news % keep][2 * kv + half] = news
                    if k_alone:
                        FULL[slot].arrive(2)
                    else:
                        FULL[slot].arrive(2 if kv else 1)
                        if kv:
                            FULL[slot - 1].arrive()
                    news += 1
                g += 1
                yield None

    def s_both():
        e = uq = 0
        g = [0, 0]
        for i, it in enumerate(items + [None]):
            yield from next_item(i)
            if it is None:
                return
            nq = 1 if it["dual"] else 2
            for u in range(uq, uq + nq):
                yield wait(Q_FULL[u & 1], u >> 1)
            for k in range(it["cnt"]):
                slot = 2 * (e % (NSLOT // 2))
                yield wait(FULL[slot], e // (NSLOT // 2))
                for t in range(2):
                    if not it["own"][t][k]:
                        continue
                    x = g[t]
                    if x > 1:
                        yield wait(O_DONE[t][x & 1], (x - 2) >> 1)
                    tensor.append(("S", t, x, e, uq if it["dual"] else uq + t))
                    tensor.append(("commit", S_FULL[t][x & 1]))
                    g[t] += 1
                    yield None
                tensor.append(("commit", EMPTY[slot]))
                EMPTY[slot].arrive()
                e += 1
                yield None
            for u in range(uq, uq + nq):
                tensor.append(("commit", Q_EMPTY[u & 1]))
            uq += nq

    def pv(t):
        e = used = g = 0
        for i, it in enumerate(items + [None]):
            yield from next_item(i)
            if it is None:
                return
            first = True
            for k in range(it["cnt"]):
                slot, use, mine = 2 * (e % (NSLOT // 2)) + 1, e // (NSLOT // 2), it["own"][t][k]
                if mine or not unwaited_skip:
                    yield wait(FULL[slot], use)
                    if ring[slot] != [e, e]:
                        raise Fault(f"V of tile {e} is not there")
                if not mine:
                    EMPTY[slot].arrive()
                    e += 1
                    yield None
                    continue
                yield wait(P_READY[t][g & 1], g >> 1)
                if first and used > 0:
                    yield wait(O_FREE[t], used - 1)
                tensor.append(("PV", t, g, e, first))
                tensor.append(("commit", O_DONE[t][g & 1]))
                tensor.append(("commit", EMPTY[slot]))
                g, first, e = g + 1, False, e + 1
                yield None
            used += it["c"][t] > 0

    def softmax(t, w):
        before, merges, uq, tiles8, news = [0, 0], 0, 0, 0, 0

        def pv_done(lane, g):
            return wait(O_DONE[lane][g & 1], g >> 1)

        for i, it in enumerate(items + [None]):
            yield from next_item(i)
            if it is None:
                return
            dual, steps, rows = it["dual"], it["c"][t], it["rows"][t][w]
            slot = uq + (0 if dual else t)
            if turn:
                for u in [slot] if skip_other_q else range(uq, uq + (1 if dual else 2)):
                    yield wait(Q_FULL[u & 1], u >> 1)
                if not dual and not own_q_twice:
                    Q_EMPTY[(slot ^ 1) & 1].arrive()
                read = 2 if own_q_twice and not dual else 1
                if steps == 0:
                    Q_EMPTY[slot & 1].arrive(read)
            mine = [k for k in range(it["cnt"]) if it["own"][t][k]]
            for s, k in enumerate(mine):
                g = before[t] + s
                yield wait(S_FULL[t][g & 1], g >> 1)
                if S[t][g & 1] != g:
                    raise Fault(f"S of step {S[t][g & 1]} read as that of {g}")
                if turn and s == 0:
                    if q_slots[slot & 1] != [slot] * 4:
                        raise Fault(f"the factors of Q of use {slot} are not there")
                    Q_EMPTY[slot & 1].arrive(read)
                yield None
                if rows:
                    if k < it["cached"]:
                        if scales[(tiles8 + k) % keep] != tiles8 + k:
                            raise Fault(f"the scales of tile {tiles8 + k} are not there")
                    elif turn and factors[(news + k - it["cached"]) % keep] != [news + k - it["cached"]] * 4:
                        raise Fault(f"the factors of new tile {news + k - it['cached']} are not there")
                    if s > 0 and r.random() < 0.3:  # the maximum or the scales' reference moved: O is rescaled
                        yield pv_done(t, g - 1)
                        if O[t] != g - 1:
                            raise Fault(f"O of step {O[t]} rescaled as that of {g - 1}")
                    P[t][g & 1] = g
                yield None
                P_READY[t][g & 1].arrive()
                yield None
            if steps > 0:
                yield pv_done(t, before[t] + steps - 1)
            join = dual and it["c"][1] > 0
            if join:
                stats[t][w] = i
                MERGE.arrive()
                yield None
                yield wait(MERGE, merges)
                yield pv_done(t ^ 1, before[t ^ 1] + it["c"][t ^ 1] - 1)
                if stats[t ^ 1] != [i] * 4:
                    raise Fault("the other lane's maxima are not those of this join")
                merges += 1
            before = [before[x] + it["c"][x] for x in range(2)]
            tiles8 += it["cached"]
            news += it["cnt"] - it["cached"]
            uq += 1 if dual else 2
            if (dual and t == 1 and not join) or steps == 0:
                continue
            for lane in (t, t ^ 1) if join else (t,):
                if O[lane] != before[lane] - 1:
                    raise Fault(f"O of step {O[lane]} stored as that of {before[lane] - 1}")
            if join and stats[t ^ 1] != [i] * 4:
                raise Fault("maxima written over while they were read")
            yield None
            O_FREE[t].arrive(1 if join else 2)
            if join:
                O_FREE[t ^ 1].arrive()

    def complete(x):
        if x[0] == "commit":
            x[1].arrive()
        elif x[0] == "S":
            _, t, g, e, q = x
            if ring[2 * (e % (NSLOT // 2))] != [e, e] or q_slots[q & 1] != [q] * 4:
                raise Fault(f"S of step {g} reads K or Q that is not there")
            S[t][g & 1] = g
        else:
            _, t, g, e, first = x
            if ring[2 * (e % (NSLOT // 2)) + 1] != [e, e]:
                raise Fault(f"P V of step {g} reads V that is not there")
            if S[t][g & 1] != g:
                raise Fault(f"P of step {g} was written over")
            if not first and O[t] != g - 1:
                raise Fault(f"O of step {O[t]} goes on with step {g}")
            O[t] = g

    roles = {"producer": producer(), "S": s_both(), "PV 0": pv(0), "PV 1": pv(1)}
    roles.update({f"converter {kv} {h}": converter(kv, h) for kv in range(2) for h in range(2)})
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
            there, where, at, what = copies.pop(r.randrange(min(len(copies), 6)))
            where[at] = what
            there()
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


@pytest.mark.parametrize("mistake", [dict(k_alone=True), dict(skip_other_q=True), dict(own_q_twice=True), dict(unwaited_skip=True),
                                     dict(keep=4)],
                         ids=["k_without_v", "a_slot_left_out", "q_let_go_by_one", "let_go_unwaited", "few_scales"])
def test_the_model_finds_mistakes(mistake):
    for seed in range(400):
        try:
            simulate(seed, **mistake)
        except Fault:
            return
    raise AssertionError("not found")
