"""A model of how the roles of the paged attention's tcgen05 kernels (page_attend_rows.cu, page_attend_tc.cu) hand work to
one another: mbarriers waited for by the parity of a phase, products that a pipe executes in the order of their issue,
and buffers whose contents are followed. Roles are generators that a scheduler advances in any order; nothing here knows
times, so what it allows may be rare on the chip.

A role yields ("wait", barrier, phase) or ("step",). A wait for phase k (the first is 0) is the hardware's: it passes when
the barrier's present phase has another parity than k. It can be relied on only while that phase is k or k + 1; a waiter
that finds another is a fault ("phase"), a role that never goes on is one ("stuck"), and so is a buffer that holds another
unit's or part's contents than its reader's."""
import random


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.left, self.done = name, count, count, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.done = self.count, self.done + 1


class Pipe:
    """The tensor cores as one issuing thread sees them: products and commits, in order, later."""

    def __init__(self):
        self.todo = []

    def role(self):
        while True:
            if self.todo:
                self.todo.pop(0)()
            yield ("step",)


class Cta:
    def __init__(self, parts):
        self.parts, self.faults, self.roles, self.pipes, self.held = parts, set(), [], [], {}

    def bars(self, **counts):
        for name, c in counts.items():
            setattr(self, name, [Bar(name, c[1]) for _ in range(c[0])] if isinstance(c, tuple) else Bar(name, c))

    def put(self, where, what):
        self.held[where] = what

    def look(self, where, what, kind):
        if self.held.get(where) != what:
            self.faults.add(kind)

    def pipe(self):
        p = Pipe()
        self.pipes.append(p.role())
        return p

    def run(self, seed):
        """Every role to its end under one random schedule: roles have speeds, and now and then one rests."""
        rng = random.Random(seed)
        live = [[r, ("step",), rng.choice((1, 1, 4, 20))] for r in self.roles]
        pipes = [[p, ("step",), rng.choice((1, 4, 20))] for p in self.pipes]
        idle = 0
        while live:
            if rng.random() < 0.02:
                rng.choice(live)[2] = rng.choice((0.05, 1, 4, 20))
            x = rng.choices(live + pipes, [y[2] for y in live + pipes])[0]
            if x[1][0] == "wait":
                _, bar, k = x[1]
                if bar.done not in (k, k + 1):
                    self.faults.add("phase")
                if bar.done % 2 == k % 2:  # the present phase has the awaited one's parity: not over
                    idle += 1
                    if idle > 5000:
                        self.faults.add("stuck")
                        return self.faults
                    continue
            if x in live:
                idle = 0
            try:
                x[1] = next(x[0])
            except StopIteration:
                live.remove(x)
        return self.faults


def rows128(parts, pv_waits_for_queries=False, factors=4):
    """attend_rows_kernel, 128 rows: two issuers, S double-buffered. parts: the units of a CTA's parts; factors: the places
    for rows' factors."""
    c = Cta(parts)
    dec, soft = 2, 2  # warps of K and of V, and of each softmax group
    c.bars(k_full=(2, dec), v_full=(2, dec), v_empty=(2, 1), s_full=(2, 1), p_full=(2, 2 * soft), q_full=2 * dec, q_empty=1, merge=2 * soft)

    def queries(seg):
        if seg > 0:
            yield ("wait", c.q_empty, seg - 1)
        yield ("step",)
        c.put("q", seg)
        c.put(("f", seg % factors), seg)
        c.q_full.arrive()

    def decoder(kv, one):
        full, empty, n = (c.v_full, c.v_empty, 0) if kv else (c.k_full, c.s_full, 0)
        for seg, m in enumerate(parts):
            if seg > 0:
                yield from queries(seg)
            for _ in range(m):
                if n > 1:
                    yield ("wait", empty[n & 1], (n >> 1) - 1)
                yield ("step",)
                c.put(("v" if kv else "k", n & 1), n)
                if not kv and one == 0:
                    c.put(("ok", n & 3), n)
                full[n & 1].arrive()
                n += 1

    def qk_issuer(pipe):
        n = 0
        for seg, m in enumerate(parts):
            yield ("wait", c.q_full, seg)
            for i in range(m):
                t = n & 1
                yield ("wait", c.k_full[t], n >> 1)
                if n > 1:
                    yield ("wait", c.v_empty[t], (n >> 1) - 1)

                def product(n=n, t=t, seg=seg):
                    c.look(("k", t), n, "k tile")
                    c.look("q", seg, "queries")
                    c.put(("s", t), n)
                pipe.todo += [product, c.s_full[t].arrive] + ([c.q_empty.arrive] if i == m - 1 else [])
                yield ("step",)
                n += 1

    def pv_issuer(pipe):
        n = 0
        for seg, m in enumerate(parts):
            if pv_waits_for_queries:
                yield ("wait", c.q_full, seg)
            for i in range(m):
                t = n & 1
                yield ("wait", c.v_full[t], n >> 1)
                yield ("wait", c.p_full[t], n >> 1)

                def product(n=n, t=t, seg=seg):
                    c.look(("v", t), n, "v tile")
                    c.look(("s", t), ("p", n), "p")
                    c.put("o", (seg, n))
                pipe.todo += [product, c.v_empty[t].arrive]
                yield ("step",)
                n += 1

    def softmax(w, one):
        n = 0
        for seg, m in enumerate(parts):
            if seg == 0:
                yield from queries(0)
            for i in range(m):
                t = n & 1
                yield ("wait", c.s_full[t], n >> 1)
                if i == 0:
                    c.look(("f", seg % factors), seg, "factors")
                if c.held.get(("s", t)) != ("p", n):  # the other warps' columns may be P by now
                    c.look(("s", t), n, "s")
                c.look(("ok", n & 3), n, "unit_ok")
                yield ("step",)
                if i > 0 and one == 0:  # O rescaled
                    yield ("wait", c.v_empty[(n - 1) & 1], (n - 1) >> 1)
                    c.look("o", (seg, n - 1), "o")
                c.put(("s", t), ("p", n))
                c.p_full[t].arrive()
                n += 1
            yield ("wait", c.v_empty[(n - 1) & 1], (n - 1) >> 1)
            c.look("o", (seg, n - 1), "o")
            c.merge.arrive()
            yield ("wait", c.merge, 2 * seg)
            for _ in range(4):  # results written
                yield ("step",)
            c.look("o", (seg, n - 1), "o")
            c.merge.arrive()
            yield ("wait", c.merge, 2 * seg + 1)

    c.roles = [decoder(kv, i) for kv in (0, 1) for i in range(dec)] + [softmax(w, i) for w in (0, 1) for i in range(soft)]
    c.roles += [qk_issuer(c.pipe()), pv_issuer(c.pipe())]
    return c


def rows256(parts, factors=2):
    """attend_rows_kernel, 256 rows: one issuer, a softmax group a row tile, the next unit's S over this one's P."""
    c = Cta(parts)
    dec, soft = 2, 2
    c.bars(k_full=(2, dec), v_full=(2, dec), v_empty=(2, 1), s_full=(3, 1), p_full=(2, soft), pv_done=(2, 1), q_full=2 * dec, q_empty=1)

    def queries(seg):
        if seg > 0:
            yield ("wait", c.q_empty, seg - 1)
        yield ("step",)
        c.put("q", seg)
        c.put(("f", seg % factors), seg)
        c.q_full.arrive()

    def decoder(kv, one):
        full, n = c.v_full if kv else c.k_full, 0
        empty = c.v_empty if kv else c.s_full[1:]
        for seg, m in enumerate(parts):
            if seg > 0:
                yield from queries(seg)
            for _ in range(m):
                if n > 1:
                    yield ("wait", empty[n & 1], (n >> 1) - 1)
                yield ("step",)
                c.put(("v" if kv else "k", n & 1), n)
                if not kv and one == 0:
                    c.put(("ok", n & 3), n)
                full[n & 1].arrive()
                n += 1

    def issuer(pipe):
        nk = nv = 0
        for seg, m in enumerate(parts):
            yield ("wait", c.q_full, seg)
            for i in range(m + 1):
                if i > 0:
                    yield ("wait", c.v_full[nv & 1], nv >> 1)
                for w in (0, 1):
                    if i > 0:
                        yield ("wait", c.p_full[w], nv)
                    if w == 0 and i < m:
                        yield ("wait", c.k_full[nk & 1], nk >> 1)

                    def second(n=nv, w=w, seg=seg):
                        c.look(("v", n & 1), n, "v tile")
                        c.look(("s", w), ("p", n), "p")
                        c.put(("o", w), (seg, n))

                    def first(n=nk, w=w, seg=seg):
                        c.look(("k", n & 1), n, "k tile")
                        c.look("q", seg, "queries")
                        c.put(("s", w), n)
                    if i > 0:
                        pipe.todo += [second] + ([c.v_empty[nv & 1].arrive] if w else []) + ([c.pv_done[w].arrive] if i == m else [])
                    if i < m:
                        pipe.todo += [first, c.s_full[1 + (nk & 1) if w else 0].arrive]
                        pipe.todo += [c.q_empty.arrive] if w and i == m - 1 else []
                    yield ("step",)
                nv += i > 0
                nk += i < m

    def softmax(w, one):
        n = 0
        for seg, m in enumerate(parts):
            if seg == 0:
                yield from queries(0)
            for i in range(m):
                yield ("wait", c.s_full[1 + (n & 1)], n >> 1) if w else ("wait", c.s_full[0], n)
                if i == 0:
                    c.look(("f", seg % factors), seg, "factors")
                if c.held.get(("s", w)) != ("p", n):
                    c.look(("s", w), n, "s")
                c.look(("ok", n & 3), n, "unit_ok")
                if i > 0:
                    c.look(("o", w), (seg, n - 1), "o")
                yield ("step",)
                c.put(("s", w), ("p", n))
                c.p_full[w].arrive()
                n += 1
            yield ("wait", c.pv_done[w], seg)
            for _ in range(4):
                c.look(("o", w), (seg, n - 1), "o")
                yield ("step",)

    c.roles = [decoder(kv, i) for kv in (0, 1) for i in range(dec)] + [softmax(w, i) for w in (0, 1) for i in range(soft)]
    c.roles += [issuer(c.pipe())]
    return c


def causal(parts, end_by_product=False):
    """attend_tc_kernel: a ring of raw rows, one issuer, the queries staged by the softmax groups, a part at a time.
    end_by_product: a part's end waits for its last product by that product's phase, as it once did."""
    c = Cta(parts)
    dec, soft, ring = 2, 2, 3
    c.bars(raw_full=(ring, 1), raw_empty=(ring, 2 * dec), k_full=(2, dec), k_empty=(2, 1), v_full=(2, dec), v_empty=(2, 1), s_full=(2, 1),
           p_full=(4, soft), pv_done=(2, 1), part_done=(2, 1), q_full=2 * soft, merge=2 * soft)

    def producer():
        for n in range(sum(parts)):
            if n >= ring:
                yield ("wait", c.raw_empty[n % ring], n // ring - 1)
            c.put(("raw", n % ring), n)
            yield ("step",)
            c.raw_full[n % ring].arrive()

    def decoder(kv, one):
        full, empty = (c.v_full, c.v_empty) if kv else (c.k_full, c.k_empty)
        for n in range(sum(parts)):
            yield ("wait", c.raw_full[n % ring], n // ring)
            if n > 1:
                yield ("wait", empty[n & 1], (n >> 1) - 1)
            c.look(("raw", n % ring), n, "raw")
            yield ("step",)
            c.put(("v" if kv else "k", n & 1), n)
            if not kv and one == 0:
                c.put(("ok", n & 3), n)
            full[n & 1].arrive()
            c.raw_empty[n % ring].arrive()

    def issuer(pipe):
        nk = nv = 0
        for seg, m in enumerate(parts):
            yield ("wait", c.q_full, seg)
            for i in range(m + 1):
                if i < m:
                    yield ("wait", c.k_full[nk & 1], nk >> 1)

                    def first(n=nk, seg=seg):
                        c.look(("k", n & 1), n, "k tile")
                        c.look("q", seg, "queries")
                        c.put(("s", n & 1, 0), n)
                        c.put(("s", n & 1, 1), n)
                    pipe.todo += [first, c.k_empty[nk & 1].arrive, c.s_full[nk & 1].arrive]
                    yield ("step",)
                    nk += 1
                if i > 0:
                    t = nv & 1
                    yield ("wait", c.v_full[t], nv >> 1)
                    for w in (0, 1):
                        yield ("wait", c.p_full[2 * t + w], nv >> 1)

                        def second(n=nv, w=w, seg=seg):
                            c.look(("v", n & 1), n, "v tile")
                            c.look(("s", n & 1, w), ("p", n), "p")
                            c.put(("o", w), (seg, n))
                        pipe.todo += [second, c.pv_done[w].arrive] + ([c.part_done[w].arrive] if i == m else [])
                        yield ("step",)
                    pipe.todo += [c.v_empty[t].arrive]
                    nv += 1

    def softmax(w, one):
        n = 0
        for seg, m in enumerate(parts):
            c.put("q", seg)
            c.put("f", seg)
            yield ("step",)
            c.q_full.arrive()
            for i in range(m):
                t = n & 1
                yield ("wait", c.s_full[t], n >> 1)
                c.look("f", seg, "factors")
                c.look(("ok", n & 3), n, "unit_ok")
                if c.held.get(("s", t, w)) != ("p", n):
                    c.look(("s", t, w), n, "s")
                yield ("step",)
                if i > 0 and one == 0:
                    yield ("wait", c.pv_done[w], n - 1)
                    c.look(("o", w), (seg, n - 1), "o")
                c.put(("s", t, w), ("p", n))
                c.p_full[2 * t + w].arrive()
                n += 1
            yield ("wait", c.pv_done[w], n - 1) if end_by_product else ("wait", c.part_done[w], seg)
            c.look(("o", w), (seg, n - 1), "o")
            c.merge.arrive()
            yield ("wait", c.merge, 2 * seg)
            for _ in range(4):
                for g in (0, 1):
                    c.look(("o", g), (seg, n - 1), "o")
                yield ("step",)
            c.merge.arrive()
            yield ("wait", c.merge, 2 * seg + 1)

    c.roles = [producer(), issuer(c.pipe())] + [decoder(kv, i) for kv in (0, 1) for i in range(dec)]
    c.roles += [softmax(w, i) for w in (0, 1) for i in range(soft)]
    return c
