"""The prefix kernel's work split and its barrier protocol, checked on the host.

``tests/px_host_check.cu`` includes the kernel header and checks by brute force
how steps are dealt to CTAs, which CTAs the merge reads and where their partial
states lie.

The protocol is checked on a model: the roles of one CTA (two producers, the
two issuing warps, two softmax warpgroups) run against one another with random
delays of loads and products.  An mbarrier wait names its phase by parity, so
it may pass on a phase two before the one it means; the model knows the count
and fails when a wait passes early, when a role overwrites what another still
reads, and when nobody can go on.
"""

import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "paged_kv_cache_115_gb300", "csrc")


def test_work_split(tmp_path):
    nvcc = next((c for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc")
                 if c and os.path.exists(c)), None)
    if nvcc is None:
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "px_host_check")
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-O1",
                        "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-DPKV_BUILD", "-o", exe,
                        os.path.join(ROOT, "tests", "px_host_check.cu")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "prefix work ok" in r.stdout, r.stdout + r.stderr


class Early(Exception):
    pass


class Bar:
    def __init__(self, need=1):
        self.need, self.arrived, self.count = need, 0, 0       # count: phases completed

    def arrive(self):
        self.arrived += 1
        if self.arrived == self.need:
            self.arrived, self.count = 0, self.count + 1

    def passes(self, phase):
        """Whether a wait for `phase` by its parity passes now."""
        if (self.count - 1) & 1 != phase & 1:
            return False
        if self.count < phase + 1:
            raise Early(phase)
        return True


class Cta:
    """One CTA: segments of (query tiles, steps), a ring of `ns` tiles.  A role
    yields the (barrier, phase) it waits for."""

    def __init__(self, segments, ns, rng, epilogue="mended"):
        self.seg, self.ns, self.rng, self.epilogue = segments, ns, rng, epilogue
        self.steps = [(nt, s == 0) for nt, n in segments for s in range(n)]
        self.full, self.empty = [Bar() for _ in range(ns)], [Bar() for _ in range(ns)]
        self.s_full = [[Bar(), Bar()], [Bar(), Bar()]]
        self.p_free, self.p_full = [Bar(), Bar()], [[Bar(), Bar()], [Bar(), Bar()]]
        self.o_done, self.q_full = [Bar(), Bar()], [Bar(), Bar()]
        self.tile = [None] * ns            # what a ring slot holds
        self.S = [None, None]              # (job, "S" / "P" / "used") of a buffer
        self.O = [0, 0]                    # products that have landed, by tile
        self.Q = [0, 0]                    # segment whose queries a tile holds
        self.pipes = {"qk": [], "pv": [], "load": []}

    def issue(self, pipe, effects):
        self.pipes[pipe].append([self.rng.choice([0, 1, 3, 6, 30]), effects])

    def producer(self, kv):
        for g in range(len(self.steps)):
            n = 2 * g + kv
            yield self.empty[n % self.ns], n // self.ns - 1

            def land(n=n):
                self.tile[n % self.ns] = n
                self.full[n % self.ns].arrive()
            self.issue("load", land)

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

                def done(n=n, x=x, b=b, job=job, c=jobs[x], last=x == nt - 1):
                    assert self.tile[n % self.ns] == n and self.S[b] in (None, (job - 2, "used"))
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

                def done(n=n, x=x, b=b, job=job, last=x == nt - 1):
                    assert self.tile[n % self.ns] == n and self.S[b] == (job, "P")
                    self.S[b] = (job, "used")
                    self.O[x] += 1
                    self.o_done[x].arrive()
                    self.p_free[b].arrive()
                    if last:
                        self.empty[n % self.ns].arrive()
                self.issue("pv", done)
                job += 1

    def softmax(self, x):
        job0 = done = 0
        for nt, n in self.seg:
            if x < nt:
                self.q_full[x].arrive()
                for st in range(n):
                    job = job0 + st * nt + x
                    yield self.s_full[x][done & 1], done >> 1
                    assert self.S[job & 1] == (job, "S")
                    if st and self.rng.random() < 0.3:           # O is rescaled
                        yield self.o_done[x], done - 1
                        assert self.O[x] == done
                    for h in range(2):
                        self.S[job & 1] = (job, "P")
                        self.p_full[job & 1][h].arrive()
                        if h == 0:
                            yield None
                    done += 1
                if self.epilogue == "mended" and nt == 1:
                    yield self.p_free[job & 1], job >> 1
                else:
                    yield self.o_done[x], done - 1
                assert self.O[x] == done
            job0 += n * nt

    def run(self):
        roles = [self.producer(0), self.producer(1), self.qk(), self.pv(), self.softmax(0),
                 self.softmax(1)]
        at = [next(r, "end") for r in roles]
        idle = 0
        while any(a != "end" for a in at) or any(self.pipes.values()):
            moved = False
            for name, ops in self.pipes.items():   # products in order, loads in any
                i = self.rng.randrange(len(ops)) if ops and name == "load" else 0
                if ops:
                    moved = True
                    if ops[i][0] <= 0:
                        ops.pop(i)[1]()
                    else:
                        ops[i][0] -= 1
            for i in self.rng.sample(range(6), self.rng.randint(1, 6)):
                if at[i] != "end" and (at[i] is None or at[i][0].passes(at[i][1])):
                    at[i] = next(roles[i], "end")
                    moved = True
            idle = 0 if moved else idle + 1
            assert idle < 500, "nobody can go on"


@pytest.mark.parametrize("ns", [5, 8])
def test_barrier_protocol(ns):
    rng = random.Random(ns)
    for _ in range(400):
        segments = [(rng.randint(1, 2), rng.choice([1, 2, 3, 7, 12])) for _ in range(rng.randint(1, 6))]
        Cta(segments, ns, rng).run()


def test_the_model_sees_an_ambiguous_wait():
    """A one-tile item that waits for its last product by o_done alone reads O
    too early now and then."""
    rng = random.Random(1)
    with pytest.raises((Early, AssertionError)):
        for _ in range(400):
            Cta([(1, rng.choice([2, 3, 7, 12]))], 5, rng, epilogue="o_done").run()
