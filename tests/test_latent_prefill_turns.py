"""The waits between the roles of pa_prefill_latent's CTA, as a model on the host.

Roles wait for counts that only grow, so whether all of them reach their end does
not depend on how they are interleaved: one run of the model per list of work
decides it.  A piece of work is (tiles of keys of query tile A, of tile B).  The
model's waits are those of pa_prefill_latent.cu: the queue of three turns, queries,
slabs of the ring, scores, weights and outputs.
"""
import collections
import itertools

import pytest

QUEUE, SLOTS = 3, 8
END = None


class Model:
    def __init__(self, works, look_past):
        self.works, self.look_past = [*works, END], look_past
        self.count = collections.Counter()
        self.loaded, self.issued = [], [[], []]

    def signal(self, *what):
        self.count[what] += 1

    def reached(self, n, *what):
        return lambda: self.count[what] >= n

    def fetcher(self):
        for turn in range(len(self.works)):
            if turn >= QUEUE:
                yield self.reached(10, "free", turn - QUEUE)
            self.signal("work", turn)

    def take(self, turn):
        yield self.reached(1, "work", turn)
        return self.works[turn]

    def producer(self):
        u, queries = 0, [0, 0]
        for turn in itertools.count():
            work = yield from self.take(turn)
            if work is END:
                return

            def load_q(x):
                yield self.reached(queries[x], "q free", x)
                queries[x] += 1
                self.signal("q", x)

            if work[0]:
                yield from load_q(0)
            for t in range(max(work)):
                for i in range(5):
                    if i == 3 and t == 0 and work[1]:
                        yield from load_q(1)
                    yield self.reached(u // SLOTS, "slot", u % SLOTS)
                    u += 1
                    self.signal("slab")
            self.loaded.append(turn)
            self.signal("free", turn)

    def products(self):
        works, steps = [0, 0], [0, 0]

        def release(slabs):
            for u in slabs:
                self.signal("slot", u % SLOTS)

        def scores(x, work, tile, t):
            if t == 0:
                yield self.reached(works[x] + 1, "q", x)
            u = 5 * (tile + t)
            yield self.reached(u + 3, "slab")
            if x == 1 or t >= work[1]:
                release(range(u, u + 3))
            self.signal("s", x)
            if t + 1 == work[x]:
                self.signal("q free", x)

        def values(x, work, tile, t):
            if t == 0:
                yield self.reached(4 * works[x], "o free", x)
            u = 5 * (tile + t)
            yield self.reached(u + 5, "slab")
            steps[x] += 1
            yield self.reached(4 * steps[x], "p", x)
            if x == 1 or t >= work[1]:
                release(range(u + 3, u + 5))
            if t + 1 == work[x]:
                self.signal("o", x)
                works[x] += 1
                self.issued[x].append(tile)

        def keyed(turn):  # the next work with keys
            while True:
                work = yield from self.take(turn)
                if work is END or max(work):
                    return turn, work
                self.signal("free", turn)
                turn += 1

        turn = tile = 0
        while True:
            turn, work = yield from keyed(turn)
            if work is END:
                return
            for x in range(2):
                if work[x]:
                    yield from scores(x, work, tile, 0)
            while work is not END and max(work):
                last = max(work) - 1
                for t in range(last):
                    for x in range(2):
                        if t < work[x]:
                            yield from values(x, work, tile, t)
                        if t + 1 < work[x]:
                            yield from scores(x, work, tile, t + 1)
                if last < work[0]:
                    yield from values(0, work, tile, last)
                # the work behind is looked at while this one's turn is held
                if self.look_past:
                    after, following = yield from keyed(turn + 1)
                else:
                    after = turn + 1
                    following = yield from self.take(after)
                here, ahead = tile, tile + max(work)
                if following is not END and following[0]:
                    yield from scores(0, following, ahead, 0)
                if last < work[1]:
                    yield from values(1, work, here, last)
                if following is not END and following[1]:
                    yield from scores(1, following, ahead, 0)
                self.signal("free", turn)
                turn, work, tile = after, following, ahead
            if work is END:
                return
            self.signal("free", turn)  # without keys, and nothing held
            turn += 1

    def softmax(self, x, warp):
        steps = works = 0
        for turn in itertools.count():
            work = yield from self.take(turn)
            if work is END:
                return
            for _ in range(work[x]):
                steps += 1
                yield self.reached(steps, "s", x)
                self.signal("p", x)
            if work[x]:
                works += 1
                yield self.reached(works, "o", x)
                self.signal("o free", x)
            self.signal("free", turn)

    def ends(self):
        roles = [self.fetcher(), self.producer(), self.products()]
        roles += [self.softmax(x, warp) for x in range(2) for warp in range(4)]
        waits = {role: next(role, None) for role in roles}
        moved = True
        while moved:
            moved = False
            for role, wait in waits.items():
                while wait is not None and wait():
                    moved = True
                    wait = next(role, None)
                waits[role] = wait
        return all(wait is None for wait in waits.values())


KINDS = [(0, 0), (1, 1), (0, 2), (3, 4), (2, 0), (3, 3)]


@pytest.mark.parametrize("length", range(6))
def test_every_list_of_work_ends(length):
    for works in itertools.product(KINDS, repeat=length):
        model = Model(works, False)
        assert model.ends(), works
        for x in range(2):
            assert len(model.issued[x]) == sum(w[x] > 0 for w in works)


def test_long_runs_without_keys_end():
    for run in range(12):
        works = [(2, 3)] + [(0, 0)] * run + [(0, 1), (2, 2)] + [(0, 0)] * run
        assert Model(works, False).ends(), run


def test_the_model_finds_a_turn_held_over_works_without_keys():
    """Looking past more than one work without keys while a turn is held waits for itself."""
    assert Model([(2, 2), (0, 0), (2, 2)], True).ends()
    assert not Model([(2, 2), (0, 0), (0, 0), (2, 2)], True).ends()
    assert not Model([(2, 2), (0, 0), (0, 0)], True).ends()
