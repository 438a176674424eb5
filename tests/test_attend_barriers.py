"""Models of the barriers between the warps of the attention kernel for up to 128 rows
(csrc/sv_attend_tiles.cu, SPLIT), run over random lists of units and random speeds of the warps.

A unit's key tiles go to two halves in turn, so that of a unit with one tile the second half has
none.  The first model checks that every product of scores reads its own unit's queries and that the
warps come to their end."""
import random

import pytest


class Bar:
    """An mbarrier: `count` arrivals make a phase, and a wait names the parity of a phase."""

    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending = self.count
            self.phase += 1

    def over(self, parity):  # the phase of this parity that came last is over
        return self.phase & 1 != parity & 1


class Cta:
    def __init__(self, units, stages, rng, idle_half_waits, output_a_unit=True):
        # idle_half_waits: a half waits for the queries of a unit of which it has no tile; output_a_unit: the products
        # report an output once a unit, not every tile, of which the softmax warps look at the last
        self.units, self.stages, self.rng, self.idle_half_waits = units, stages, rng, idle_half_waits
        self.output_a_unit = output_a_unit
        self.full = [Bar(1) for _ in range(stages)]
        self.empty = [Bar(2) for _ in range(stages)]
        self.q, self.q_free = [Bar(1), Bar(1)], [Bar(2), Bar(2)]
        self.scores, self.weights, self.out = ([Bar(1), Bar(1)] for _ in range(3))
        self.second, self.joined = Bar(1), Bar(1)
        self.place = [None, None]  # the unit whose queries a place holds (None: being written)
        self.issued = [[], []]     # the tensor cores' work of each half, in order
        self.arrivals = []         # what it reports as done, in any order
        self.outputs = [0, 0]      # output products done
        self.copies = []           # stages whose copy is in flight
        self.wrong = 0
        self.finished = False

    # each warp is a generator that yields what it waits for (None: goes on in a while)
    def loader(self):
        at = 0
        for tiles in self.units:
            for _ in range(2 * tiles):  # keys and values of a tile
                stage, turn = at % self.stages, at // self.stages
                yield lambda: self.empty[stage].over(turn + 1)
                self.copies.append(stage)
                at += 1

    def queries(self):
        for j in range(len(self.units)):
            place = j & 1
            if j >= 2:
                yield lambda: self.q_free[place].over((j >> 1) - 1)
            self.place[place] = None
            yield None
            self.place[place] = j
            self.q[place].arrive()

    def products(self, x):
        at = n_w = 0
        lap = lambda: (at // self.stages)
        for j, tiles in enumerate(self.units):
            place, last, begin = j & 1, at + 2 * tiles, at
            own = range(x, tiles, 2)

            def reach(i):
                nonlocal at
                while True:
                    stage, turn = at % self.stages, lap()
                    yield lambda: self.full[stage].over(turn)
                    if at == i:
                        return
                    self.empty[stage].arrive()
                    at += 1

            def scores(last_own):
                nonlocal at
                self.issued[x] += [("read", j, place), ("read", j, place), ("arrive", self.scores[x]),
                                   ("arrive", self.empty[at % self.stages])]
                if last_own:
                    self.issued[x].append(("arrive", self.q_free[place]))
                at += 1

            if own or self.idle_half_waits:
                yield lambda: self.q[place].over(j >> 1)
            if own:
                yield from reach(begin + 2 * x)
                scores(x + 2 >= tiles)
            else:
                self.q_free[place].arrive()
            for tile in own:
                yield from reach(begin + 2 * tile + 1)
                values = at % self.stages
                at += 1
                yield lambda: self.weights[x].over(n_w)
                n_w += 1
                self.issued[x].append(("output",))
                if tile + 2 >= tiles or not self.output_a_unit:
                    self.issued[x].append(("arrive", self.out[x]))
                self.issued[x].append(("arrive", self.empty[values]))
                if tile + 2 < tiles:
                    yield from reach(begin + 2 * tile + 4)
                    scores(tile + 4 >= tiles)
            while at != last:
                stage, turn = at % self.stages, lap()
                yield lambda: self.full[stage].over(turn)
                self.empty[stage].arrive()
                at += 1

    def softmax(self, x):
        n_scores = n_out = 0  # phases
        for j, tiles in enumerate(self.units):
            own = range(x, tiles, 2)
            if x == 1 and j > 0:
                yield lambda: self.joined.over(j - 1)
            for tile in own:
                yield lambda: self.scores[x].over(n_scores)
                self.wrong += self.outputs[x] != n_scores  # the product before is through: the output may be rescaled
                n_scores += 1
                n_out += tile != x and not self.output_a_unit
                yield None
                self.weights[x].arrive()
            if own:
                yield lambda: self.out[x].over(n_out)
                n_out += 1
                self.wrong += self.outputs[x] != n_scores
            if x == 1:
                self.second.arrive()
            else:
                yield lambda: self.second.over(j)
                yield None
                self.joined.arrive()

    def tensor_cores(self, x):
        while not self.finished:
            yield lambda: self.issued[x]
            op = self.issued[x].pop(0)
            if op[0] == "arrive":
                self.arrivals.append(op[1])
            elif op[0] == "output":
                self.outputs[x] += 1
            elif self.place[op[2]] != op[1]:
                self.wrong += 1

    def copier(self):
        while not self.finished:
            yield lambda: self.copies
            self.full[self.copies.pop(self.rng.randrange(len(self.copies)))].arrive()

    def reporter(self):  # of what the tensor cores have done
        while not self.finished:
            yield lambda: self.arrivals
            self.arrivals.pop(self.rng.randrange(len(self.arrivals))).arrive()

    def run(self):
        """The products that read wrong queries, and the outputs read too early; None: the warps wait for ever."""
        warps = [self.loader(), self.queries(), self.products(0), self.products(1), self.softmax(0), self.softmax(1)]
        live = {w: None for w in warps + [self.tensor_cores(0), self.tensor_cores(1), self.copier(), self.reporter()]}
        speed = {w: self.rng.choice([1.0, 0.2, 0.03]) for w in live}
        while any(w in live for w in warps):
            ready = [w for w, wait in live.items() if wait is None or wait()]
            if not ready:
                return None
            w = self.rng.choices(ready, [speed[w] for w in ready])[0]
            step = next(w, False)
            if step is False:
                del live[w]
            else:
                live[w] = step
        return self.wrong


def outcomes(idle_half_waits, stages, longest, lists=150, **kw):
    rng = random.Random(100 * stages + longest)
    res = []
    for _ in range(lists):
        short = rng.random()
        units = [1 if rng.random() < short else rng.randint(1, longest) for _ in range(rng.randint(1, 14))]
        res.append(Cta(units, stages, rng, idle_half_waits, **kw).run())
    return res


@pytest.mark.parametrize("stages", [5, 8])  # heads of 128, of 64
@pytest.mark.parametrize("longest", [1, 2, 5])
def test_every_product_reads_its_own_queries(stages, longest):
    assert outcomes(True, stages, longest) == [0] * 150


@pytest.mark.parametrize("stages", [5, 8])
def test_the_model_finds_a_half_that_does_not_wait(stages):
    """A half without a tile that frees the queries' place unseen: queries are mixed up, or a wait is never over."""
    res = outcomes(False, stages, 5)
    assert None in res and any(r for r in res if r)
    # units of two tiles and more are not concerned
    rng = random.Random(1)
    assert all(Cta([rng.randint(2, 5) for _ in range(10)], stages, rng, False).run() == 0 for _ in range(50))


def test_the_model_finds_an_output_whose_arrival_was_not_seen():
    """The product before some scores is through when they are there, but its arrival may be later than theirs: then
    the phase at a unit's end is not the one that a parity tells."""
    res = outcomes(True, 5, 5, output_a_unit=False)
    assert None in res or any(res)


class Ends:
    """The ends of units, where the first half's four softmax warps join what the second half's left, with one warp
    that gives up a wait somewhere.  A warp that gave up goes on through its units without waiting, and arrives."""

    def __init__(self, units, rng, looks, careful):
        # looks: after the waits for the other half, whether a warp has given up; careful: what a warp that has gives
        # to the other half is not written
        self.units, self.rng, self.looks, self.careful = units, rng, looks, careful
        self.done = [Bar(4), Bar(4)]  # the weights of a half, and with them its product
        self.second, self.joined = Bar(4), Bar(4)
        self.left = [None] * 4        # per warp: the unit whose maximum and sum the second half left
        self.dead = False
        self.wrong = 0

    def warp(self, x, w, gives_up):
        alive = True

        def wait(bar, parity):
            nonlocal alive
            if alive and not bar.over(parity):
                yield lambda: bar.over(parity) or self.dead
                alive = bar.over(parity)
                self.dead |= not alive

        for j in range(self.units):
            if x == 1 and j > 0:
                yield from wait(self.joined, j - 1)
                alive = alive and not (self.looks and self.dead)
            yield None
            if j == gives_up and alive:
                alive, self.dead = False, True
            if alive:
                self.done[x].arrive()
            yield from wait(self.done[x], j)
            if x == 1:
                if alive or not self.careful:
                    self.left[w] = j
                self.second.arrive()
                continue
            yield from wait(self.second, j)
            alive = alive and not (self.looks and self.dead)
            for _ in range(3 if alive else 0):  # reads it, for a while
                self.wrong += alive and self.left[w] != j
                yield None
            self.joined.arrive()

    def run(self):
        one = (self.rng.randrange(2), self.rng.randrange(4))
        at = self.rng.randrange(self.units)
        live = {self.warp(x, w, at if (x, w) == one else None): None for x in range(2) for w in range(4)}
        speed = {w: self.rng.choice([1.0, 0.1, 0.01]) for w in live}
        while live:
            ready = [w for w, wait in live.items() if wait is None or wait()]
            w = self.rng.choices(ready, [speed[w] for w in ready])[0]
            step = next(w, False)
            if step is False:
                del live[w]
            else:
                live[w] = step
        return self.wrong


def test_a_wait_given_up_leaves_no_wrong_row():
    rng = random.Random(5)
    wrong = lambda looks, careful: sum(Ends(rng.randint(1, 10), rng, looks, careful).run() for _ in range(600))
    assert wrong(True, True) == 0
    assert wrong(False, True) > 0 and wrong(True, False) > 0  # both are needed
