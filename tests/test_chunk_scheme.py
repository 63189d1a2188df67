"""A model of the paged chunk attention's work split and of its barriers, written out in Python, and the
invariants the kernels rely on.

The split: every (row, key tile it sees) of every KV group lies in exactly one unit, whatever the cut; a
unit's rounds are exactly its groups' tiles; partial rows are distinct and within their number, and the merge
reads exactly the parts that hold keys its row sees.

The barriers: the TMA warp, the MMA warp and the two softmax groups step through random units in a random
order with random delays, the tensor core finishing in order behind them.  Every wait is by parity, as in
hardware, so a waiter that another role could lap would read the wrong tile or stop: the model checks
what every slot, S, P and O holds when it is used, and that all roles come to their end.  This checks
the scheme; the GPU parity tests check the kernels."""
import heapq
import random

import pytest


def cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------------------------------- split
def cut(nt, C):
    nc = 1 if nt <= C else cdiv(nt, C)
    ct = max(1, cdiv(nt, nc))
    return max(1, cdiv(nt, ct)), ct


def plan(cached, new, r, n_kv, C, rounds_whole, tiles):
    """The sequences' records as the plan kernel leaves them."""
    tpt, out = 128 // r, []
    unit0 = part0 = split0 = before = lo = 0
    for c, n in zip(cached, new):
        if n == 0:
            c = 0
        np_, nt = cdiv(n, tiles * tpt), cdiv(c + n, 128)
        nc, ct = cut(nt, C)
        wp = 0
        if np_ > 1:
            wp = min(max(rounds_whole - before, 0), np_)
            before += np_
        cut_n = min(n, (np_ - wp) * tiles * tpt) if nc > 1 else 0
        out.append(dict(unit0=unit0, lo=lo, n=n, c=c, np=np_, wp=wp, nc=nc, ct=ct, cut_n=cut_n, part0=part0, split0=split0,
                        span=tiles * tpt))
        unit0 += (wp + nc * (np_ - wp)) * n_kv
        part0 += nc * cut_n
        split0 += cut_n
        lo += n
    return out, unit0, part0, split0


def make_unit(s, u, r, n_kv):
    """(group, first key tile, rounds of groups 0 and 1, lone, first rows, part offset), None without keys."""
    tpt = 128 // r
    x = u - s["unit0"]
    item = x // n_kv
    uncut = item < s["wp"]
    y, nq = (item if uncut else item - s["wp"]), s["np"] - s["wp"]
    chunk = 0 if uncut or s["nc"] == 1 else y // nq
    pair = s["np"] - 1 - y if uncut else nq - 1 - (y - chunk * nq)
    first = pair * s["span"]
    nt1 = cdiv(s["c"] + min(s["n"], first + tpt), 128)
    nt0 = cdiv(s["c"] + min(s["n"], first + s["span"]), 128)
    t0 = chunk * s["ct"]
    t1 = nt0 if uncut else min(t0 + s["ct"], nt0)
    if t0 >= t1:
        return None
    lone = min(s["n"] - first, s["span"]) <= tpt
    n0 = (t1 - t0 + 1) // 2 if lone else t1 - t0
    n1 = (t1 - t0) // 2 if lone else max(0, min(t1, nt1) - t0)
    row1 = s["lo"] + first
    part = s["part0"] + chunk * s["cut_n"] - s["lo"] if not uncut and s["cut_n"] > 0 else None
    return x - item * n_kv, t0, n0, n1, lone, (row1 if lone else row1 + tpt, row1), part


def check_split(cached, new, r, n_kv, C, rounds_whole, tiles):
    tpt = 128 // r
    seqs, n_units, n_parts, n_split = plan(cached, new, r, n_kv, C, rounds_whole, tiles)
    seen, parts = {}, {}
    for b, s in enumerate(seqs):
        end = seqs[b + 1]["unit0"] if b + 1 < len(seqs) else n_units
        for u in range(s["unit0"], end):
            d = make_unit(s, u, r, n_kv)
            if d is None:
                continue
            g, t0, n0, n1, lone, rows, part = d
            for x, n in ((0, n0), (1, n1)):
                for row in range(rows[x], min(rows[x] + tpt, s["lo"] + s["n"])):
                    last = (s["c"] + row - s["lo"]) // 128           # the last tile the row sees
                    for i in range(n):
                        tile = t0 + (2 * i + x if lone else i)
                        if tile <= last:
                            assert seen.setdefault((row, g, tile), u) == u, "a tile twice"
                            seen[row, g, tile] = u
                    if part is not None and (n > 0 or lone):
                        at = row + part
                        assert 0 <= at < n_parts
                        assert parts.setdefault((at, g), (row, t0)) == (row, t0), "a partial row twice"
    for b, s in enumerate(seqs):
        for i in range(s["n"]):
            row, tiles = s["lo"] + i, (s["c"] + i) // 128 + 1
            for g in range(n_kv):
                assert all((row, g, t) in seen for t in range(tiles)), "a tile nobody takes"
                if i < s["cut_n"]:                                    # the merge's reads
                    for k in range(min(s["nc"], cdiv(tiles, s["ct"]))):
                        assert parts[s["part0"] + k * s["cut_n"] + i, g] == (row, k * s["ct"])
    # the merge finds a split row's sequence: the last one whose split0 is at or before it
    for x in range(n_split):
        b = max(b for b, s in enumerate(seqs) if s["split0"] <= x)
        assert 0 <= x - seqs[b]["split0"] < seqs[b]["cut_n"]


@pytest.mark.parametrize("seed", range(60))
def test_every_tile_in_one_unit(seed):
    r = random.Random(seed)
    ratio, n_kv = r.choice([(1, 2), (4, 2), (8, 1), (3, 1), (100, 1), (128, 1)])
    B = r.randrange(1, 7)
    new = [r.choice([0, 1, r.randrange(1, 9), r.randrange(1, 400 // min(ratio, 8))]) for _ in range(B)]
    cached = [r.choice([0, r.randrange(0, 300), r.randrange(0, 3000)]) for _ in range(B)]
    items = sum(cdiv(n, 2 * (128 // ratio)) for n in new)
    for C in (1, 2, 3, 6, 11, 1 << 20):
        check_split(cached, new, ratio, n_kv, C, r.choice([0, r.randrange(0, items + 2)]), 2)
        check_split(cached, new, ratio, n_kv, C, 0, 1)


# ---------------------------------------------------------------------------------------- barriers
class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase, self.tx = count, count, 0, 0

    def arrive(self):
        assert self.pending > 0, "more arrivals than the phase takes"
        self.pending -= 1
        self._check()

    def expect(self):
        self.tx += 1
        self.arrive()

    def landed(self):
        self.tx -= 1
        self._check()

    def _check(self):
        if self.pending == 0 and self.tx == 0:
            self.phase, self.pending = self.phase + 1, self.count

    def passed(self, parity):
        return (self.phase & 1) != parity


class Model:
    def __init__(self, units, slots, seed):
        self.rng, self.units, self.NS = random.Random(seed), units, slots
        self.now, self.serial, self.events, self.pipe = 0.0, 0, [], 0.0
        two = lambda n: [Bar(n), Bar(n)]
        self.q_full, self.q_empty, self.u_full, self.u_empty = two(1), two(1), two(1), two(3)
        self.s_full, self.o_done, self.o_free, self.ml = two(1), two(1), two(1), Bar(1)
        self.p_full = [two(1), two(1)]
        self.kv_full, self.kv_empty = [Bar(1) for _ in range(slots)], [Bar(1) for _ in range(slots)]
        self.record, self.q, self.kv = [None] * 2, [None] * 2, [None] * slots
        self.S, self.P, self.O, self.o_read = [None] * 2, [[None] * 2, [None] * 2], [None] * 2, [True] * 2

    def later(self, dt, f):
        self.serial += 1
        heapq.heappush(self.events, (self.now + dt, self.serial, f))

    def tensor(self, f):                       # the tensor core finishes its work in order
        self.pipe = max(self.pipe, self.now) + self.rng.uniform(0.1, 2)
        self.serial += 1
        heapq.heappush(self.events, (self.pipe, self.serial, f))

    def producer(self):
        e = qi = 0
        for n in range(len(self.units) + 1):
            us, unit = n & 1, self.units[n] if n < len(self.units) else None
            yield self.u_empty[us], ((n >> 1) & 1) ^ 1
            self.record[us] = unit
            self.u_full[us].arrive()
            if unit is None:
                return
            lone, n0, n1 = unit
            for x in range(1 if lone or n1 == 0 else 2):
                qs = qi & 1
                yield self.q_empty[qs], ((qi >> 1) & 1) ^ 1
                self.q_full[qs].expect()

                def q_in(qs=qs, what=(n, x)):
                    self.q[qs] = what
                    self.q_full[qs].landed()
                self.later(self.rng.uniform(0.1, 3), q_in)
                qi += 1
            for t in range(n0 + n1 if lone else n0):
                for kv in range(2):
                    slot = e % self.NS
                    yield self.kv_empty[slot], ((e // self.NS) & 1) ^ 1
                    self.kv_full[slot].expect()

                    def kv_in(slot=slot, what=(n, t, kv)):
                        self.kv[slot] = what
                        self.kv_full[slot].landed()
                    self.later(self.rng.uniform(0.1, 3), kv_in)
                    e += 1

    def mma(self):
        NS, qi, n = self.NS, 0, -1
        k, v = [0, 0], [1, 0]                   # ring slot and phase of the next K and V tile
        rounds, used = [0, 0], [0, 0]

        def step(at):
            at[0] += 2
            if at[0] >= NS:
                at[0], at[1] = at[0] - NS, at[1] ^ 1

        def release(bars):
            for b in bars:
                b.arrive()

        def issue_s(n, lone, n0, n1, x, i, last):
            if x == 0 or lone:
                yield self.kv_full[k[0]], k[1]
            qs, slot = (qi + (0 if lone else x)) & 1, k[0]
            assert self.q[qs] == (n, 0 if lone else x) and self.kv[slot] == (n, 2 * i + x if lone else i, 0)
            done = [self.s_full[x]] + ([self.kv_empty[slot]] if last else [])
            if (2 * i + x == n0 + n1 - 1) if lone else (i == (n1 if x else n0) - 1):
                done.append(self.q_empty[qs])

            def fin():
                self.S[x] = (n, i)
                release(done)
            self.tensor(fin)
            if last:
                step(k)

        def issue_pv(n, lone, n0, n1, x, i, last):
            if x == 0 or lone:
                yield self.kv_full[v[0]], v[1]
            for half in range(2):
                yield self.p_full[x][half], rounds[x] & 1
                assert self.P[x][half] == (n, i)
            slot = v[0]
            assert self.kv[slot] == (n, 2 * i + x if lone else i, 1)
            assert i > 0 or self.o_read[x], "O overwritten before it was read"
            if i == 0:
                self.o_read[x] = False
            done = ([self.o_done[x]] if i == (n1 if x else n0) - 1 else []) + ([self.kv_empty[slot]] if last else [])

            def fin():
                self.O[x] = (n, i)
                release(done)
            self.tensor(fin)
            rounds[x] += 1
            if last:
                step(v)

        while True:
            n += 1
            yield self.u_full[n & 1], (n >> 1) & 1
            if self.record[n & 1] is None:
                return
            lone, n0, n1 = a = self.record[n & 1]
            self.u_empty[n & 1].arrive()
            nq = 1 if lone or n1 == 0 else 2
            for j in range(nq):
                yield self.q_full[(qi + j) & 1], ((qi + j) >> 1) & 1
            yield from issue_s(n, *a, 0, 0, lone or n1 == 0)
            if n1:
                yield from issue_s(n, *a, 1, 0, True)
            for x in range(2 if n1 else 1):
                yield self.o_free[x], (used[x] & 1) ^ 1
                used[x] += 1
            for i in range(n0):
                yield from issue_pv(n, *a, 0, i, lone or i >= n1)
                if i + 1 < n0:
                    yield from issue_s(n, *a, 0, i + 1, lone or i + 1 >= n1)
                if i < n1:
                    yield from issue_pv(n, *a, 1, i, True)
                    if i + 1 < n1:
                        yield from issue_s(n, *a, 1, i + 1, True)
            qi += nq

    def softmax(self, x):
        rc = units = lones = e = 0
        n = -1
        while True:
            n += 1
            yield self.u_full[n & 1], (n >> 1) & 1
            if self.record[n & 1] is None:
                return
            lone, n0, n1 = unit = self.record[n & 1]
            mine = n1 if x else n0
            for i in range(mine):
                yield self.s_full[x], rc & 1
                assert self.S[x] == (n, i) and (i == 0 or self.O[x] == (n, i - 1))
                tile = 2 * i + x if lone else i
                if self.rng.random() < 0.5:            # a tile at the sequence's end: V is looked at
                    slot, lap = (e + 2 * tile + 1) % self.NS, (e + 2 * tile + 1) // self.NS
                    yield self.kv_full[slot], lap & 1
                    assert self.kv[slot] == (n, tile, 1)
                for half in range(2):
                    yield self.rng.uniform(0.05, 1.5)
                    self.P[x][half] = (n, i)
                    self.p_full[x][half].arrive()
                rc += 1
            if mine:
                yield self.o_done[x], units & 1
                units += 1
                assert self.O[x] == (n, mine - 1)
            e += 2 * (n0 + n1 if lone else n0)
            if lone and x:
                if mine:
                    self.ml.arrive()
                self.u_empty[n & 1].arrive()
                continue
            merge = lone and n1 > 0
            if merge:
                yield self.ml, lones & 1
                lones += 1
            yield self.rng.uniform(0.05, 3)
            assert mine == 0 or self.O[x] == (n, mine - 1)
            assert not merge or self.O[1] == (n, n1 - 1)
            assert self.record[n & 1] == unit
            for y in ([x] if mine else []) + ([1] if merge else []):
                self.o_read[y] = True
                self.o_free[y].arrive()
            self.u_empty[n & 1].arrive()

    def run(self):
        roles = {"tma": self.producer(), "mma": self.mma(), "s0": self.softmax(0), "s1": self.softmax(1)}
        wait, until = dict.fromkeys(roles), dict.fromkeys(roles, 0.0)
        slow = {k: self.rng.choice([0, 0, 0.05, 0.3]) for k in roles}
        while roles:
            moved = False
            for k in self.rng.sample(list(roles), len(roles)):
                if self.now < until[k] or wait[k] is not None and not wait[k][0].passed(wait[k][1]):
                    continue
                moved = True
                try:
                    w = next(roles[k])
                except StopIteration:
                    del roles[k]
                    continue
                delay = w if isinstance(w, float) else 0.0
                if self.rng.random() < slow[k]:          # now and then a role stands still for long
                    delay += self.rng.uniform(0, 25)
                wait[k], until[k] = (None if isinstance(w, float) else w), self.now + delay
                if delay:
                    self.later(delay, lambda: None)
            if not moved:
                assert self.events, "every role waits"
                self.now, _, f = heapq.heappop(self.events)
                f()


@pytest.mark.parametrize("slots", [5, 10])
@pytest.mark.parametrize("seed", range(40))
def test_barriers(slots, seed):
    r = random.Random(seed)
    for case in range(6):
        units = []
        for _ in range(r.randrange(1, 9)):
            if r.random() < 0.5:
                tiles = r.randrange(1, 12)
                units.append((True, (tiles + 1) // 2, tiles // 2))
            else:
                n0 = r.randrange(1, 8)
                units.append((False, n0, r.randrange(0, n0 + 1)))
        Model(units, slots, 1000 * seed + case).run()
