"""The barriers of the serving attention kernel, stepped on the CPU.

A model of one CTA: the producer, the issuer of S, the two issuers of P V and the eight softmax warps as
coroutines, with the kernel's barriers (counts, phases, parities), its rings (descriptors, Q slots, K and V
slots) and tensor memory. Copies land and tensor work completes at random times, the latter in order. Random
items, scheduled at random, must run to their end, and the model fails where
- a barrier gets more arrivals than its phase expects;
- a wait by parity would take another use of the barrier for its own;
- a reader finds another key tile, score tile, P, O or descriptor than the one it is at;
- nothing can run.

The names are those of the kernel (csrc/fa_serve.cu). HALF is d = 128: key tiles in two halves, two score buffers
a lane, P over S, five slots. Otherwise d = 64: one step a tile, P apart from S, twelve slots.
"""

import random

import pytest


class Fault(Exception):
    pass


class Bar:
    """An mbarrier: `count` arrivals and the bytes expected complete a phase."""

    def __init__(self, count, name):
        self.count, self.pending, self.tx, self.done, self.name = count, count, 0, 0, name

    def _complete(self):
        if self.pending == 0 and self.tx == 0:
            self.done += 1
            self.pending = self.count

    def arrive(self, n=1):
        if n > self.pending:
            raise Fault(f"{self.name}: an arrival too many")
        self.pending -= n
        self._complete()

    def expect(self):
        self.tx += 1
        self.arrive()

    def land(self):
        self.tx -= 1
        self._complete()

    def ready(self, use):
        """What a wait for use number `use` sees: the parity only."""
        seen = (self.done & 1) != (use & 1)
        if seen != (self.done == use + 1) or self.done > use + 1:
            raise Fault(f"{self.name}: a wait for use {use} at phase {self.done}")
        return seen


def draw_items(r, half):
    items = []
    for _ in range(r.randint(1, 14)):
        cnt = r.choice([1, 1, 1, 2, 2, 3, 4, 5, 8, 9, 14])
        dual = r.random() < 0.6
        if dual:
            c = ((cnt + 1) // 2, cnt // 2)
        else:  # the first lane's tokens see no more tiles than the second's; none in a cut item's last part
            c = (r.choice([0, cnt, max(0, cnt - 1), r.randint(0, cnt)]), cnt)
        own = [[(k & 1) == t if dual else k < c[t] for k in range(cnt)] for t in range(2)]
        last_cached = r.randint(0, cnt)  # the tiles that may have one half: the last cached one and a lane's last
        halves = [[2 if half and not (r.random() < 0.5 and (k == last_cached or k >= (c[t] if not dual else cnt) - 1))
                   else 1 for k in range(cnt)] for t in range(2)]
        rows = [[r.random() < 0.6 for _ in range(4)] for _ in range(2)]  # warps with a row
        if dual:
            rows[1] = rows[0]
        items.append(dict(cnt=cnt, dual=dual, c=c, own=own, halves=halves, rows=rows, pair=dual and cnt >= 8 and r.random() < 0.7,
                          cached=cnt - r.choice([0, 1, 1]),
                          steps=[sum(halves[t][k] for k in range(cnt) if own[t][k]) for t in range(2)]))
    return items


def simulate(seed, half, guard=True, extra_arrival=False, early_free=False):
    """guard, extra_arrival, early_free: mistakes to plant (a wait without the look at `loading`, a slot released
    twice by the lane that computes nothing of it, Q released before the last S that reads it)."""
    r = random.Random(seed)
    NSLOT = 5 if half else 12
    buf = (lambda g: g & 1) if half else (lambda g: 0)
    use = (lambda g: g >> 1) if half else (lambda g: g)
    FULL = [Bar(1, f"FULL {i}") for i in range(NSLOT)]
    EMPTY = [Bar(2, f"EMPTY {i}") for i in range(NSLOT)]
    Q_FULL, Q_EMPTY = ([Bar(1, f"{n} {i}") for i in range(2)] for n in ("Q_FULL", "Q_EMPTY"))
    S_FULL, P_READY, O_DONE = ([[Bar(c, f"{n} {t} {u}") for u in range(2)] for t in range(2)]
                               for n, c in (("S_FULL", 1), ("P_READY", 4), ("O_DONE", 1)))
    S_FREE, O_FREE = ([Bar(c, f"{n} {t}") for t in range(2)] for n, c in (("S_FREE", 4), ("O_FREE", 8)))
    MERGE = Bar(8, "MERGE")
    D_FULL, D_EMPTY = ([Bar(c, f"{n} {i}") for i in range(4)] for n, c in (("D_FULL", 1), ("D_EMPTY", 11)))
    items = draw_items(r, half)
    state = {"loading": 0}
    slots, q_slots, descs = [None] * NSLOT, [None] * 2, [None] * 4
    S, P, O = [[None] * 2, [None] * 2], [[None] * 2, [None] * 2], [None, None]
    copies, tensor = [], []  # copies in flight; tensor work issued, in order

    def wait(bar, n):
        return lambda: bar.ready(n)

    def next_item(i):
        yield wait(D_FULL[i & 3], i >> 2)
        if descs[i & 3] != i:
            raise Fault(f"descriptor of item {descs[i & 3]} read as that of {i}")
        D_EMPTY[i & 3].arrive()

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
                q_slots[uq & 1] = None
                Q_FULL[uq & 1].expect()
                copies.append((Q_FULL[uq & 1], q_slots, uq & 1, uq))
                uq += 1
                yield None
            for k in range(it["cnt"]):
                together = it["pair"] and k < it["cached"]  # K and V of a tile in one go
                for group in ([(e, e + 1)] if together else [(e,), (e + 1,)]):
                    for x in group:
                        if x >= NSLOT:
                            yield wait(EMPTY[x % NSLOT], x // NSLOT - 1)
                    state["loading"] = group[-1] + 1
                    for x in group:
                        FULL[x % NSLOT].expect()
                    yield None
                    for x in group:
                        slots[x % NSLOT] = None
                        copies.append((FULL[x % NSLOT], slots, x % NSLOT, x))
                    yield None
                e += 2

    def landed(e, steady):
        if guard and not steady:
            yield lambda: state["loading"] > e
        yield wait(FULL[e % NSLOT], e // NSLOT)
        if slots[e % NSLOT] != e:
            raise Fault(f"ring entry {e} is not there")

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
            if early_free:
                for u in range(uq, uq + nq):
                    tensor.append(("commit", Q_EMPTY[u & 1]))
            for k in range(it["cnt"]):
                h = [it["halves"][t][k] if it["own"][t][k] else 0 for t in range(2)]
                both = half and k >= 4 and h == [2, 2]  # the ordinary tile of two lanes
                yield from landed(e, k >= 4)
                for hh in range(max(h)):
                    if both:
                        for t in range(2):
                            yield wait(O_DONE[t][buf(g[t])], use(g[t] - 2))
                    for t in range(2):
                        if hh >= h[t]:
                            continue
                        x = g[t]
                        if half and x > 1 and not both:
                            yield wait(O_DONE[t][buf(x)], use(x - 2))
                        if not half and x > 0:
                            yield wait(S_FREE[t], x - 1)
                        tensor.append(("S", t, x, e, uq if it["dual"] else uq + t))
                        tensor.append(("commit", S_FULL[t][buf(x)]))
                        g[t] += 1
                        yield None
                tensor.append(("commit", EMPTY[e % NSLOT]))
                EMPTY[e % NSLOT].arrive()
                e += 2
                yield None
            if not early_free:
                for u in range(uq, uq + nq):
                    tensor.append(("commit", Q_EMPTY[u & 1]))
            uq += nq

    def pv(t):
        e, used, g = 1, 0, 0
        for i, it in enumerate(items + [None]):
            yield from next_item(i)
            if it is None:
                return
            first = True
            for k in range(it["cnt"]):
                yield from landed(e, k >= 4 and (it["dual"] or k < it["c"][t]))
                if not it["own"][t][k]:
                    EMPTY[e % NSLOT].arrive(2 if extra_arrival else 1)
                    e += 2
                    yield None
                    continue
                for _ in range(it["halves"][t][k]):
                    yield wait(P_READY[t][buf(g)], use(g))
                    if first and used > 0:
                        yield wait(O_FREE[t], used - 1)
                    tensor.append(("PV", t, g, e, first))
                    tensor.append(("commit", O_DONE[t][buf(g)]))
                    g, first = g + 1, False
                    yield None
                tensor.append(("commit", EMPTY[e % NSLOT]))
                e += 2
            used += it["c"][t] > 0

    merged = [0, 0]  # warps of a lane that have left their maxima and sums, joins so far taken together

    def softmax(t, warp):
        before, merges = [0, 0], 0

        def pv_done(lane, g):
            return wait(O_DONE[lane][buf(g)], use(g))

        for i, it in enumerate(items + [None]):
            yield from next_item(i)
            if it is None:
                return
            steps, rows = it["steps"][t], it["rows"][t][warp]
            for s in range(steps):
                g = before[t] + s
                yield wait(S_FULL[t][buf(g)], use(g))
                if S[t][buf(g)] != g:
                    raise Fault(f"S of step {S[t][buf(g)]} read as that of {g}")
                yield None
                if not half:
                    S_FREE[t].arrive()
                    if s > 0:
                        yield pv_done(t, g - 1)
                elif rows and s > 0 and r.random() < 0.3:  # the maximum moved: O is rescaled
                    yield pv_done(t, g - 1)
                    if O[t] != g - 1:
                        raise Fault(f"O of step {O[t]} rescaled as that of {g - 1}")
                if rows:
                    P[t][buf(g)] = g
                yield None
                P_READY[t][buf(g)].arrive()
                yield None
            if steps > 0:
                yield pv_done(t, before[t] + steps - 1)
            join = it["dual"] and it["c"][1] > 0
            if join:
                if merged[t] >= 4 * (merges + 1):
                    raise Fault("a join's maxima written over")
                merged[t] += 1
                MERGE.arrive()
                yield None
                yield wait(MERGE, merges)
                o = t ^ 1
                yield pv_done(o, before[o] + it["steps"][o] - 1)
                if merged[o] != 4 * (merges + 1):
                    raise Fault("the other lane's maxima are not those of this join")
                merges += 1
            before = [before[x] + it["steps"][x] for x in range(2)]
            if (it["dual"] and t == 1 and not join) or steps == 0:
                continue
            for lane in (t, t ^ 1) if join else (t,):
                if O[lane] != before[lane] - 1:
                    raise Fault(f"O of step {O[lane]} stored as that of {before[lane] - 1}")
            yield None
            O_FREE[t].arrive(1 if join else 2)
            if join:
                O_FREE[t ^ 1].arrive()

    def complete(x):
        if x[0] == "commit":
            x[1].arrive()
        elif x[0] == "S":
            _, t, g, e, q = x
            if slots[e % NSLOT] != e or q_slots[q & 1] != q:
                raise Fault(f"S of step {g} reads K or Q that is not there")
            S[t][buf(g)] = g
        else:
            _, t, g, e, first = x
            if slots[e % NSLOT] != e:
                raise Fault(f"P V of step {g} reads V that is not there")
            if half and S[t][buf(g)] != g:
                raise Fault(f"P of step {g} was written over")
            if not first and O[t] != g - 1:
                raise Fault(f"O of step {O[t]} goes on with step {g}")
            O[t] = g

    roles = {"producer": producer(), "S": s_both(), "PV 0": pv(0), "PV 1": pv(1)}
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
            bar, where, at, what = copies.pop(r.randrange(min(len(copies), 3)))
            where[at] = what
            bar.land()
        elif k == "tensor":
            complete(tensor.pop(0))
        else:
            try:
                waits[k] = next(roles[k])
            except StopIteration:
                del roles[k], waits[k]


@pytest.mark.parametrize("half", [False, True], ids=["d64", "d128"])
@pytest.mark.parametrize("block", range(4))
def test_every_schedule_ends(half, block):
    for seed in range(60 * block, 60 * block + 60):
        simulate(seed, half)


@pytest.mark.parametrize("mistake", [dict(guard=False), dict(extra_arrival=True), dict(early_free=True)],
                         ids=["wait_by_parity_alone", "arrives_twice", "q_released_early"])
def test_the_model_finds_mistakes(mistake):
    found = 0
    for seed in range(120, 220):  # a wait by parity alone goes wrong in one schedule of 150
        try:
            simulate(seed, True, **mistake)
        except Fault:
            found += 1
    assert found > 0
