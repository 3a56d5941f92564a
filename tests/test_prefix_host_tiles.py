"""The prefix kernel's query tiles and accumulators in the protocol model.

The shared memory of a query tile holds the queries of a segment, then, in its
epilogue, rows of O on their way out, then the next segment's queries, while
the S products read it on their own time; O in TMEM is copied out row by row
while the next segment's first product waits to overwrite it.  The roles of
``test_prefix_host.py`` are run here with both owned: a product fails when the
queries under it, or the O that it overwrites, are not the ones of its segment.
"""

import random

import pytest

from tests.test_prefix_host import Cta, Early


class Tiles(Cta):
    """``mistake``: None, "queries early" (the next segment's queries are
    written before the last S of this one has landed), "queries before O" (after
    it, but before O went through the tile) or "weights before O" (the next
    segment starts before O is copied out)."""

    def __init__(self, segments, ns, rng, mistake=None):
        super().__init__(segments, ns, rng)
        self.mistake = mistake
        self.reads_o = [False, False]

    def qk(self):
        job, jobs, seg = 0, [0, 0], [0, 0]
        for g, (nt, first) in enumerate(self.steps):
            n = 2 * g
            if first:
                for x in range(nt):
                    yield self.q_full[x], seg[x]
                    seg[x] += 1
            yield self.full[n % self.ns], n // self.ns
            for x in range(nt):
                b = job & 1
                if job >= 2:
                    yield self.p_free[b], (job >> 1) - 1
                assert self.Q[x] == ("Q", seg[x])

                def done(n=n, x=x, b=b, job=job, c=jobs[x], own=seg[x], last=x == nt - 1):
                    assert self.tile[n % self.ns] == n and self.Q[x] == ("Q", own)
                    self.S[b] = (job, "S")
                    self.s_full[x][c & 1].arrive()
                    if last:
                        self.empty[n % self.ns].arrive()
                self.issue("qk", done)
                jobs[x] += 1
                job += 1

    def pv(self):
        job = 0
        for g, (nt, first) in enumerate(self.steps):
            n = 2 * g + 1
            yield self.full[n % self.ns], n // self.ns
            for x in range(nt):
                b = job & 1
                for h in range(2):
                    yield self.p_full[b][h], job >> 1
                    assert not self.reads_o[x]

                def done(n=n, x=x, b=b, job=job, last=x == nt - 1):
                    assert self.tile[n % self.ns] == n and self.S[b] == (job, "P")
                    assert not self.reads_o[x]
                    self.S[b] = (job, "used")
                    self.O[x] += 1
                    self.o_done[x].arrive()
                    self.p_free[b].arrive()
                    if last:
                        self.empty[n % self.ns].arrive()
                self.issue("pv", done)
                job += 1

    def softmax(self, x):
        mine = [i for i, (nt, _) in enumerate(self.seg) if x < nt]
        job0 = done = own = 0
        early = None                              # weights released before the epilogue
        for i, (nt, n) in enumerate(self.seg):
            if x < nt:
                more = i != mine[-1]
                if early is None and self.Q[x] != ("Q", own + 1):
                    self.Q[x] = ("Q", own + 1)
                    self.q_full[x].arrive()
                own += 1
                for st in range(n):
                    job = job0 + st * nt + x
                    if self.mistake == "queries early" and more and st == n - 1:
                        self.Q[x] = ("Q", own + 1)
                        self.q_full[x].arrive()
                    if early != job:
                        yield self.s_full[x][done & 1], done >> 1
                        assert self.S[job & 1] == (job, "S")
                        for h in range(2):
                            self.S[job & 1] = (job, "P")
                            self.p_full[job & 1][h].arrive()
                            if h == 0:
                                yield None
                    done += 1
                if self.mistake == "queries before O" and more:
                    self.Q[x] = ("Q", own + 1)
                    self.q_full[x].arrive()
                if nt == 1:
                    yield self.p_free[job & 1], job >> 1
                else:
                    yield self.o_done[x], done - 1
                self.reads_o[x] = True
                held = self.O[x]
                early = None
                if self.mistake == "weights before O" and more:
                    self.Q[x] = ("Q", own + 1)
                    self.q_full[x].arrive()
                    early = job0 + n * nt + x
                    yield self.s_full[x][done & 1], done >> 1
                    for h in range(2):
                        self.S[early & 1] = (early, "P")
                        self.p_full[early & 1][h].arrive()
                for _ in range(4):                # O goes through the tile in parts
                    if early is None:
                        self.Q[x] = ("O", own)
                    yield None
                    assert self.O[x] == held == done
                self.reads_o[x] = False
            job0 += n * nt


def segments(rng):
    return [(rng.randint(1, 2), rng.choice([1, 2, 3, 7, 12])) for _ in range(rng.randint(1, 6))]


@pytest.mark.parametrize("ns", [5, 8])
def test_queries_and_accumulators_belong_to_their_segment(ns):
    rng = random.Random(ns)
    for _ in range(400):
        Tiles(segments(rng), ns, rng).run()


@pytest.mark.parametrize("mistake", ["queries early", "queries before O", "weights before O"])
def test_the_model_sees_a_tile_that_changes_hands_too_early(mistake):
    rng = random.Random(2)
    with pytest.raises((Early, AssertionError)):
        for _ in range(50):
            Tiles([(2, 3), (2, 2), (1, 4), (2, 3)], 5, rng, mistake).run()
