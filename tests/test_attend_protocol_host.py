"""The attention kernel's barriers, run on the CPU: each warp role as a generator that
waits and arrives as the kernel does, in random interleavings of unequal speeds, with
copies that land in any order. An mbarrier tells phases apart by parity alone, so a
wait that is two phases off passes early or never ends. Checked here: every wait
ends, none passes in another phase than its own, and every product finds the keys,
values, queries, scores and probabilities that belong to it."""
import random

import pytest


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.left, self.phase = name, count, count, 0

    def arrive(self):
        self.left -= 1
        assert self.left >= 0, self.name
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def wait(self, i):
        """Until phase i is complete, as try_wait.parity tells it."""
        while (self.phase & 1) == (i & 1):
            yield
        assert self.phase == i + 1, (self.name, self.phase, i)


class Pipe:
    """One CTA. segments: (tiles of keys, row tiles: 1 or 2, tiles that hold nodes' values)."""

    def __init__(self, segments, SK, SV, rng):
        self.segments, self.SK, self.SV, self.rng = segments, SK, SV, rng
        self.twin = all(act == 1 for _, act, _ in segments)

        def bars(name, n, count):
            return [Bar(f"{name}{i}", count) for i in range(n)]

        self.k_full, self.k_empty = bars("k_full", SK, 1), bars("k_empty", SK, 2)
        self.v_full, self.v_empty = bars("v_full", SV, 1), bars("v_empty", SV, 2)
        self.s_full, self.p_ready, self.pv_done = bars("s_full", 2, 1), bars("p_ready", 2, 5), bars("pv_done", 2, 1)
        self.turn, self.start = bars("turn", 2, 1), bars("start", 2, 1)
        self.q_full, self.q_empty = bars("q_full", 2, 1), bars("q_empty", 2, 2)
        self.o_free, self.merge = Bar("o_free", 10), Bar("merge", 8)
        self.keys, self.values, self.queries = [None] * SK, [None] * SV, [None, None]
        self.scores, self.output = [None, None], [None, None]
        self.flying, self.products = [], [[], []]     # copies on their way; products issued, per stream

    def slot(self, i):
        return (i & 1, i >> 1) if self.twin else (0, i)

    def copies(self, keys):
        n = 0
        full, empty, ring, S = (self.k_full, self.k_empty, self.keys, self.SK) if keys else \
            (self.v_full, self.v_empty, self.values, self.SV)
        for i, (nt, act, _) in enumerate(self.segments):
            ahead = 1 if act == 2 else 2

            def ask():
                slot, use = self.slot(i)
                if use > 0:
                    yield from self.q_empty[slot].wait(use - 1)
                self.flying.append((self.queries, slot, i, self.q_full[slot]))
                yield

            first = self.twin or i == 0
            if keys and first:
                yield from ask()
            for t in range(nt):
                if n >= S:
                    yield from empty[n % S].wait(n // S - 1)
                self.flying.append((ring, n % S, (i, t), full[n % S]))
                n += 1
                yield
                if keys and not first and t == min(nt, ahead) - 1:
                    yield from ask()

    def memory(self):
        while True:
            if self.flying:
                where, at, what, bar = self.flying.pop(self.rng.randrange(len(self.flying)))
                where[at] = what
                bar.arrive()
            yield

    def go(self):
        kn, vn, sent = 0, 0, [0, 0]

        def keys_there():
            nonlocal kn
            at, kn = kn, kn + 1
            yield from self.k_full[at % self.SK].wait(at // self.SK)

        def hand_on(g):
            if sent[g]:
                yield from self.p_ready[g].wait(sent[g] - 1)
            self.p_ready[g].arrive()
            sent[g] += 1
            yield

        for i, (nt, act, tails) in enumerate(self.segments):
            ahead = 1 if act == 2 else 2
            slot, use = self.slot(i)
            yield from self.q_full[slot].wait(use)
            for _ in range(min(nt, ahead)):
                yield from keys_there()
            self.start[slot].arrive()
            for t in range(nt):
                st = vn % self.SV
                yield from self.v_full[st].wait(vn // self.SV)
                vn += 1
                for _ in range(3 if t in tails else 0):      # the values are looked at, and written
                    assert self.values[st] == (i, t)
                    yield
                if t + ahead < nt:
                    yield from keys_there()
                for g in ((0, 1) if act == 2 else (t & 1,)):
                    yield from hand_on(g)

    def mma(self, g):
        n0, done, turns = 0, 0, 0
        issue = self.products[g].append
        for i, (nt, act, _) in enumerate(self.segments):
            two = act == 2
            step, first = (1, 0) if two else (2, g)
            slot, use = self.slot(i)

            def scores(t):
                def run(st=(n0 + t) % self.SK, what=(i, t), two=two, slot=slot):
                    assert self.keys[st] == what and self.queries[slot] == what[0]
                    self.scores[g] = ("S",) + what
                    self.s_full[g].arrive()
                    for _ in range(1 if two else 2):
                        self.k_empty[st].arrive()
                issue(run)
                if t + step >= nt:
                    issue(self.q_empty[slot].arrive)

            yield from self.start[slot].wait(use)
            if first < nt:
                scores(first)
            else:
                issue(self.q_empty[slot].arrive)
            if i > 0:
                yield from self.o_free.wait(i - 1)
            for t in range(first, nt, step):
                yield from self.p_ready[g].wait(done)
                if two:
                    if g:
                        yield from self.turn[1].wait(turns)
                    elif turns:
                        yield from self.turn[0].wait(turns - 1)
                    turns += 1

                def run(st=(n0 + t) % self.SV, what=(i, t), two=two):
                    assert self.values[st] == what and self.scores[g] == ("P",) + what
                    self.output[g] = what
                    self.pv_done[g].arrive()
                    for _ in range(1 if two else 2):
                        self.v_empty[st].arrive()
                issue(run)
                done += 1
                yield
                if t + step < nt:
                    scores(t + step)
                if two:
                    self.turn[g ^ 1].arrive()
            n0 += nt
            self.o_free.arrive()

    def tensor_cores(self):
        while True:
            some = [q for q in self.products if q]
            if some:
                self.rng.choice(some).pop(0)()
            yield

    def softmax(self, g):
        own, merges = 0, 0
        for i, (nt, act, _) in enumerate(self.segments):
            two = act == 2
            jobs = nt if two else (nt + 1 - g) // 2
            for j in range(jobs):
                yield from self.s_full[g].wait(own)
                assert self.scores[g][0] == "S"
                yield
                if j and self.rng.random() < 0.5:            # the output so far is rescaled
                    yield from self.pv_done[g].wait(own - 1)
                    yield
                self.p_ready[g].arrive()
                self.p_of[g] += 1
                if self.p_of[g] % 4 == 0:                    # the last of the stream's four warps
                    self.scores[g] = ("P",) + self.scores[g][1:]
                own += 1
            both = not two and nt > 1
            if both or two or g == 0:
                yield from self.pv_done[g].wait(own - 1)
            if not two:
                self.merge.arrive()
                yield from self.merge.wait(merges)
                merges += 1
            yield
            assert self.output[g if two else 0][0] == i and (not both or self.output[1][0] == i)
            self.o_free.arrive()

    p_of = None

    def run(self):
        self.p_of = [0, 0]
        roles = [self.copies(True), self.copies(False), self.go(), self.mma(0), self.mma(1)]
        roles += [self.softmax(g) for g in (0, 1) for _ in range(4)]
        ends = len(roles)
        roles += [self.memory(), self.tensor_cores()]
        alive = list(range(len(roles)))
        weight = [self.rng.choice([1, 1, 1, 8, 0.1]) for _ in roles]
        for _ in range(2_000_000):
            if alive[0] >= ends:
                break
            k = self.rng.choices(alive, [weight[x] for x in alive])[0]
            try:
                next(roles[k])
            except StopIteration:
                alive.remove(k)
        assert alive[0] >= ends, ("a wait does not end", self.segments, self.SK, self.SV)
        assert not self.flying                               # nothing is copied behind the last wait


@pytest.mark.parametrize("rings", [(3, 2), (3, 3), (5, 5), (6, 6)], ids=lambda r: "%d+%d stages" % r)
@pytest.mark.parametrize("mixed", [False, True])
def test_every_wait_ends_in_its_own_phase(rings, mixed):
    rng = random.Random(31 * rings[1] + mixed)
    for _ in range(40):
        segments = []
        for _ in range(rng.randint(1, 6)):
            nt = rng.choice([1, 1, 2, 3, 4, 7, 12])
            tails = set(range(nt - rng.choice([0, 1, 2]), nt))
            segments.append((nt, rng.choice([1, 1, 2]) if mixed else 1, tails))
        Pipe(segments, *rings, rng).run()
