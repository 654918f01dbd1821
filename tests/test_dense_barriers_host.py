"""The barriers of the tensor-core dense kernels, as a model run on the host.

A wait tests the parity of a barrier's current phase, so it takes two completed phases for
none: whoever waits for phase n has to look before phase n + 1 completes, and must not look
before phase n - 1 has.  The roles below wait, arrive, load and issue in the order of the
kernels' code (k_dense_fwd_tc.cu, k_dense_bwd_tc.cu); products and loads complete later, products in
the order of their issue.  Schedules are random, with one role at a time held back for a
while; every wait is held to the phase that it means.
"""
from __future__ import annotations

import random

import pytest


class Wrong(Exception):
    pass


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.phase = name, count, count, 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def passed(self, n):
        """What the parity test answers for phase n (counted from 0)."""
        says = (self.phase & 1) != (n & 1)
        if says != (self.phase > n):
            raise Wrong(f"{self.name}: phase {n} meant, {self.phase} completed")
        return says


class Kernel:
    """Roles are generators that yield (barrier, phase) to wait; loads and products are queued."""

    def __init__(self, seed):
        self.rng, self.bars, self.products, self.loads, self.roles = random.Random(seed), {}, [], [], {}

    def bar(self, name, count=1):
        return self.bars.setdefault(name, Bar(name, count))

    def bars_of(self, name, n, count=1):
        return [self.bar(f"{name}{i}", count) for i in range(n)]

    def commit(self, bar):
        self.products.append(bar)

    def load(self, bar):
        self.loads.append(bar)

    def run(self, limit=100000):
        wants, r = {}, self.rng

        def go(name):
            try:
                wants[name] = next(self.roles[name])
            except StopIteration:
                del self.roles[name]
                wants.pop(name, None)

        for name in list(self.roles):
            go(name)
        everyone = list(self.roles) + ["products", "loads", None]
        held, left = None, 0
        for _ in range(limit):
            if not self.roles:
                return
            if left == 0:
                held, left = r.choice(everyone), r.randint(1, 60)
            left -= 1
            able = [n for n in self.roles if wants[n][0].passed(wants[n][1])]
            able += ["products"] * bool(self.products) + ["loads"] * bool(self.loads)
            if not able:
                raise Wrong("nobody can go on: " + ", ".join(f"{n} at {b.name}[{p}]" for n, (b, p) in wants.items()))
            free = [n for n in able if n != held]
            if not free:
                left = 0
                continue
            name = r.choice(free)
            if name == "products":
                self.products.pop(0).arrive()
            elif name == "loads":
                self.loads.pop(r.randrange(len(self.loads))).arrive()
            else:
                go(name)
        raise Wrong("no end")


class Ring:
    """The loader's side of a ring of tiles."""

    def __init__(self, k, stages):
        self.k, self.n, self.pos = k, stages, 0
        self.full, self.empty = k.bars_of("full", stages), k.bars_of("empty", stages)

    def load(self):
        st = self.pos % self.n
        if self.pos >= self.n:
            yield self.empty[st], self.pos // self.n - 1
        self.k.load(self.full[st])
        self.pos += 1


def items_role(k, items, ring, readers):
    """The item ring: (loader's side, reader's side)."""
    full, empty = k.bars_of("item_full", ring), k.bars_of("item_empty", ring, readers)

    def put(n):
        if n >= ring:
            yield empty[n % ring], n // ring - 1
        full[n % ring].arrive()

    def take(n):
        yield full[n % ring], n // ring
        if n < len(items):
            empty[n % ring].arrive()

    return put, take


def row_pass(seed, items, stages, warps=3, ds_bars=2):
    """items: key tiles of each item."""
    k = Kernel(seed)
    ring, sweep = Ring(k, stages), lambda nk: nk if nk <= 2 else 0
    put, take = items_role(k, items, 2, warps + 1)
    fix_full, fix_empty, dp, acc = k.bar("fix_full"), k.bar("fix_empty"), k.bar("dp"), k.bar("acc")
    s, ds = k.bars_of("s", 2), k.bars_of("ds", ds_bars, warps)
    dp_read, join, out_read = k.bar("dp_read", warps), k.bar("join", warps), k.bar("out_read", warps)

    def loader():
        for n, nk in enumerate(items):
            yield from put(n)
            if not sweep(nk):
                yield from ring.load()
            yield from ring.load()
            yield from ring.load()
            if n:
                yield fix_empty, n - 1
            k.load(fix_full)
            for _ in range(1, nk + sweep(nk)):
                yield from ring.load()
                yield from ring.load()
        yield from put(len(items))

    def mma():
        at = nt = nd = n_out = 0
        for n, nk in enumerate(items):
            yield from take(n)
            yield fix_full, n
            sw = sweep(nk)
            nn, tile = nk + sw, {}

            def scores(j):
                nonlocal at
                st = tile[j] = at % stages
                yield ring.full[st], at // stages
                at += 1
                k.commit(s[(nt + j) & 1])
                if j < sw:
                    k.commit(ring.empty[st])

            def dprob(j):
                nonlocal at
                st = at % stages
                yield ring.full[st], at // stages
                at += 1
                if j > 0:
                    yield dp_read, nt + j - 1
                k.commit(dp)
                k.commit(ring.empty[st])
                if j == nn - 1:
                    k.commit(fix_empty)

            out = at % stages
            if not sw:
                at += 1
            yield from scores(0)
            yield from dprob(0)
            if not sw:
                yield out_read, n_out
                n_out += 1
                ring.empty[out].arrive()
            for j in range(nn):
                if j + 1 < nn:
                    yield from scores(j + 1)
                    yield from dprob(j + 1)
                else:
                    yield dp_read, nt + j
                if j >= sw:
                    yield ds[nd % ds_bars], nd // ds_bars
                    nd += 1
                    k.commit(ring.empty[tile[j]])
                    if j == nn - 1:
                        k.commit(acc)
            nt += nn
        yield from take(len(items))

    def warp():
        nt = nd = n_join = at = 0
        for n, nk in enumerate(items):
            yield from take(n)
            sw = sweep(nk)
            if not sw:
                yield fix_full, n
                yield ring.full[at % stages], at // stages
                at += 1
                out_read.arrive()
                join.arrive()
                yield join, n_join
                n_join += 1
            at += 2 * (sw + nk)
            for step in range(sw + nk):
                yield s[nt & 1], nt >> 1
                yield dp, nt
                dp_read.arrive()
                nt += 1
                if step < sw:
                    if step == sw - 1:
                        join.arrive()
                        yield join, n_join
                        n_join += 1
                    continue
                ds[nd % ds_bars].arrive()
                nd += 1
            yield acc, n
        yield from take(len(items))

    k.roles = {"loader": loader(), "mma": mma(), **{f"warp{i}": warp() for i in range(warps)}}
    k.run()


def key_pass(seed, items, stages, two_s, warps=3, p_bars=None):
    """items: row tiles of each item; two_s: S of the next step ahead of this one's P."""
    k = Kernel(seed)
    p_bars = p_bars or (2 if two_s else 1)
    s_bars = 2 if two_s else 1
    ring = Ring(k, stages)
    put, take = items_role(k, items, 2, warps + 2)
    fix_full, fix_empty, dp, acc = k.bar("fix_full"), k.bar("fix_empty"), k.bar("dp"), k.bar("acc")
    s, p = k.bars_of("s", s_bars), k.bars_of("p", p_bars, warps)
    p_half, ds = k.bar("p_half", warps), k.bar("ds", warps)
    stat_full, stat_empty = k.bars_of("stat_full", 2), k.bars_of("stat_empty", 2, warps)

    def loader():
        for n, nj in enumerate(items):
            yield from put(n)
            if n:
                yield fix_empty, n - 1
            k.load(fix_full)
            for _ in range(2 * nj):
                yield from ring.load()
        yield from put(len(items))

    def statistics():
        nt = 0
        for n, nj in enumerate(items):
            yield from take(n)
            for _ in range(nj):
                if nt >= 2:
                    yield stat_empty[nt & 1], (nt >> 1) - 1
                stat_full[nt & 1].arrive()
                nt += 1
        yield from take(len(items))

    def mma():
        at = step = 0

        def tile(into):
            nonlocal at
            into[0] = at % stages
            yield ring.full[at % stages], at // stages
            at += 1

        for n, nj in enumerate(items):
            yield from take(n)
            yield fix_full, n
            q, d, qn = [0], [0], [0]
            yield from tile(q)
            k.commit(s[step % s_bars])
            yield from tile(d)
            k.commit(dp)
            for j in range(nj):
                more = j + 1 < nj

                def next_scores():
                    yield from tile(qn)
                    k.commit(s[(step + 1) % s_bars])

                if two_s:
                    if more:
                        yield from next_scores()
                else:
                    yield p_half, step
                yield p[step % p_bars], step // p_bars
                k.commit(ring.empty[d[0]])
                if not two_s and more:
                    yield from next_scores()
                yield ds, step
                step += 1
                k.commit(ring.empty[q[0]])
                if more:
                    yield from tile(d)
                    k.commit(dp)
                else:
                    k.commit(acc)
                    k.commit(fix_empty)
                q[0] = qn[0]
        yield from take(len(items))

    def warp():
        nt = 0
        for n, nj in enumerate(items):
            yield from take(n)
            for _ in range(nj):
                yield stat_full[nt & 1], nt >> 1
                yield s[nt % s_bars], nt // s_bars
                if not two_s:
                    p_half.arrive()
                p[nt % p_bars].arrive()
                yield dp, nt
                ds.arrive()
                stat_empty[nt & 1].arrive()
                nt += 1
            yield acc, n
        yield from take(len(items))

    k.roles = {"loader": loader(), "mma": mma(), "statistics": statistics(), **{f"warp{i}": warp() for i in range(warps)}}
    k.run()


def forward(seed, items, stages, warps=2):
    """items: (shared, key tiles of stream 0, of stream 1)."""
    k = Kernel(seed)
    ring = Ring(k, stages)
    put, take = items_role(k, items, 3, 2 * warps + 2)
    q_full, q_empty, s, o = (k.bars_of(n, 2) for n in ("q_full", "q_empty", "s", "o"))
    p_half, p_full = (k.bars_of(n, 2, warps) for n in ("p_half", "p_full"))
    join_full, join_empty = k.bar("join_full", warps), k.bar("join_empty", warps)
    clear_req, clean = k.bar("clear_req"), k.bar("clean")
    requests = []

    def loader():
        for n, (shared, n0, n1) in enumerate(items):
            yield from put(n)
            yield from ring.load()
            if not shared and n1:
                yield from ring.load()
            streams, nn = ((max(n0, n1),) if shared else (n0, n1)), max(n0, n1)
            for j in range(nn):
                for ns in streams:
                    if j < ns:
                        yield from ring.load()
                    if j + 1 < ns:
                        yield from ring.load()
        yield from put(len(items))

    def queries():
        nq = [0, 0]
        for n, (_, n0, n1) in enumerate(items):
            yield from take(n)
            for i, ns in enumerate((n0, n1)):
                if ns:
                    if nq[i]:
                        yield q_empty[i], nq[i] - 1
                    k.load(q_full[i])
                    nq[i] += 1
        yield from take(len(items))

    def mma():
        at, nq, np, nc = 0, [0, 0], [0, 0], 0
        for n, (shared, n0, n1) in enumerate(items):
            yield from take(n)
            num, nn, v, kt = (n0, n1), max(n0, n1), 0, 0
            last_reader = lambda i, j: not shared or i == 1 or j >= n1
            for i in (0, 1):
                if not num[i]:
                    continue
                if i == 0 or not shared:
                    kt, at = at, at + 1
                    yield ring.full[kt % stages], kt // stages
                yield q_full[i], nq[i]
                nq[i] += 1
                k.commit(s[i])
                if last_reader(i, 0):
                    k.commit(ring.empty[kt % stages])
                if num[i] == 1:
                    k.commit(q_empty[i])
            for j in range(nn):
                for i in (0, 1):
                    if j >= num[i]:
                        continue
                    more = j + 1 < num[i]
                    if not shared or i == 0 or j >= n0:
                        v, at = at, at + 1
                        yield ring.full[v % stages], v // stages
                        if j + 1 < nn if shared else more:
                            kt, at = at, at + 1
                    if j == nn - 1 and k.rng.random() < 0.5:  # values behind the sequence
                        requests.append(v)
                        clear_req.arrive()
                        yield clean, nc
                        nc += 1
                    yield p_half[i], np[i]
                    yield p_full[i], np[i]
                    np[i] += 1
                    if last_reader(i, j):
                        k.commit(ring.empty[v % stages])
                    if more:
                        yield ring.full[kt % stages], kt // stages
                        k.commit(s[i])
                        if last_reader(i, j + 1):
                            k.commit(ring.empty[kt % stages])
                        if j + 2 == num[i]:
                            k.commit(q_empty[i])
                    else:
                        k.commit(o[i])
        yield from take(len(items))
        requests.append(None)
        clear_req.arrive()

    def clearing():
        n = 0
        while True:
            yield clear_req, n
            if requests[n] is None:
                return
            clean.arrive()
            n += 1

    def warp(i):
        ns = no = n_join = 0
        for n, (shared, *num) in enumerate(items):
            yield from take(n)
            if not num[i]:
                continue
            for _ in range(num[i]):
                yield s[i], ns
                ns += 1
                p_half[i].arrive()
                p_full[i].arrive()
            yield o[i], no
            no += 1
            if shared or not num[1]:
                continue
            if i == 1:
                join_full.arrive()
                yield join_empty, n_join
            else:
                yield join_full, n_join
                join_empty.arrive()
            n_join += 1
        yield from take(len(items))

    k.roles = {"loader": loader(), "queries": queries(), "mma": mma(), "clearing": clearing(),
               **{f"warp{i}{w}": warp(i) for i in (0, 1) for w in range(warps)}}
    k.run()


def walks(seed):
    r = random.Random(seed)
    return [r.randint(1, 7) for _ in range(r.randint(1, 4))]


def pairs(seed):
    """Items as the forward kernel makes them: row tiles side by side, or halves of the keys."""
    r = random.Random(seed)
    out = []
    for _ in range(r.randint(1, 5)):
        shared, n0 = r.random() < 0.6, r.randint(1, 6)
        out.append((shared, n0, r.choice([0, n0, n0 + 1] if shared else [n0, n0 - 1])))
    return out


SEEDS = range(400)


@pytest.mark.parametrize("stages", [5, 10])
def test_forward(stages):
    for seed in SEEDS:
        forward(seed, pairs(seed), stages)


@pytest.mark.parametrize("stages", [5, 10])
def test_row_pass(stages):
    for seed in SEEDS:
        row_pass(seed, walks(seed), stages)


@pytest.mark.parametrize("stages,two_s", [(5, False), (10, True)])
def test_key_pass(stages, two_s):
    for seed in SEEDS:
        key_pass(seed, walks(seed), stages, two_s)


@pytest.mark.parametrize("broken", [lambda s: row_pass(s, walks(s), 5, ds_bars=1),
                                    lambda s: key_pass(s, walks(s), 10, True, p_bars=1)])
def test_the_model_sees_a_phase_that_completes_unseen(broken):
    """A single dS barrier in the row pass, a single P barrier where S is computed ahead: the MMA
    thread issues the next step before it waits for this one's."""
    seen = 0
    for seed in range(100):
        try:
            broken(seed)
        except Wrong:
            seen += 1
    assert seen >= 20
