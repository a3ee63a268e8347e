"""A step-by-step model of the INT8 product's tile kernel: the roles of every CTA
of a cluster (copies, the pair's products, widening, draining) and its barriers,
run on the CPU under random interleavings, with and without waits that run out.

As the kernel does it:

- copies fill byte stages (bempty -> bfull), one per 128 codes of K;
- four widening groups take one half of every other byte stage each (a turn has
  barriers bfull of its own: load i completes barrier i modulo 2 nbyte), hand it
  back (bempty) and arrive on the pair's first CTA (ffull) once the fp16 stage is
  written, having waited for the stage's last products (fempty);
- one thread of the pair's first CTA issues the products and commits them to
  fempty and, at a chunk's end, to tfull of BOTH CTAs: such an arrival travels on
  its own and may reach the second CTA late;
- draining warps wait for tfull, read, and arrive on the first CTA's tempty; where
  K is split, two cluster barriers stand around the exchange of sums, which every
  other role joins at its end;
- a wait that runs out sets the CTA's abort flag, and the role goes to its end.

Checks: a widening warp, the products and the draining warps only ever read what the
load, the stage or the chunk that they are at has put there; when a CTA goes, nothing may still arrive in it (a copy, a commit), the
pair's products are done, every wait of the closing part ends, and all barriers
balance (every CTA does go); without timeouts every chunk is read by every warp."""
import os
import random
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "combine_moe_dispatch_layout_gb300", "csrc", "linear_i8.cu")

DRAIN = 10 ** 6
HALVES, GROUPS, NF = 2, 4, 4
TURNS = GROUPS // HALVES


class Bar:
    """mbarrier: try_wait(parity) is true once the phase of that parity is done."""

    def __init__(self, count):
        self.count = self.pending = count
        self.done = 0

    def arrive(self):
        self.pending -= 1
        assert self.pending >= 0, "more arrivals than the barrier's count"
        if self.pending == 0:
            self.done += 1
            self.pending = self.count

    def try_wait(self, parity):
        return (self.done & 1) != parity


class Cta:
    def __init__(self, pair, rank, nbyte, warps):
        self.pair, self.rank = pair, rank
        self.bfull = [Bar(1) for _ in range(TURNS * nbyte)]
        self.holds = [None] * nbyte     # the load whose bytes are in a byte stage
        self.wide = [None] * NF         # the 64-code step whose numbers are in an fp16 stage
        self.bempty = [Bar(HALVES) for _ in range(nbyte)]
        self.ffull = [Bar(2) for _ in range(NF)]
        self.fempty = [Bar(1) for _ in range(NF)]
        self.tfull = [Bar(1) for _ in range(2)]
        self.tempty = [Bar(2 * warps) for _ in range(2)]
        self.abort = False
        self.coming = 0                 # copies in flight
        self.issued = None              # what the first CTA tells of its commits
        self.at_block = 0
        self.read = set()
        self.left = 0                   # roles that are through


class Cluster:
    """`pairs` pairs share one tile's K (split), or one pair walks `tiles` tiles."""

    def __init__(self, seed, pairs, tiles, nk, chunk, nbyte, warps, limit, early_wait=False,
                 own_drain=False, idle=False, stage_barriers=False):
        self.rng = random.Random(seed)
        self.split = pairs > 1
        self.tiles = 0 if idle else (1 if self.split else tiles)
        self.nk, self.chunk, self.nbyte, self.warps = nk, chunk, nbyte, warps
        self.limit, self.early_wait, self.own_drain = limit, early_wait, own_drain
        self.ctas = [[Cta(p, r, nbyte, warps) for r in range(2)] for p in range(pairs)]
        self.flat = [c for pair in self.ctas for c in pair]
        self.mma_issued = [0] * pairs
        self.mma_done = [0] * pairs
        self.queue = [[] for _ in range(pairs)]              # (accumulator, chunk) of products
        self.acc = [[(None, 0), (None, 0)] for _ in range(pairs)]   # chunk, products in it
        self.fills = []                 # (cta, stage)
        self.commits = []               # [pair, products it follows, cta, barrier]
        # barriers that the byte stages take turns with: 2 nbyte, or nbyte
        self.nfull = nbyte if stage_barriers else TURNS * nbyte
        self.timeouts = 0
        self.roles_per_cta = 2 + GROUPS + warps
        self.cluster_count = len(self.flat) * self.roles_per_cta
        self.cluster_at = 0
        self.faults = []

    # ---- waits ---------------------------------------------------------------
    def wait(self, bar, parity, limit=None):
        for _ in range(self.limit if limit is None else limit):
            if bar.try_wait(parity):
                return True
            yield
        return False

    def give_up(self, cta):
        self.timeouts += 1
        cta.abort = True

    def cluster_sync(self):
        phase = self.cluster_at // self.cluster_count
        self.cluster_at += 1
        while self.cluster_at // self.cluster_count == phase:
            yield

    def nchunks(self):
        return -(-self.nk // self.chunk)

    # ---- roles -----------------------------------------------------------------
    def copies(self, c):
        s = phase = n = 0
        ok = True
        for _ in range(self.tiles):
            for _ in range(self.nk):
                ok = yield from self.wait(c.bempty[s], phase ^ 1)
                if not ok:
                    self.give_up(c)
                    break
                self.fills.append((c, s, n))
                c.coming += 1
                n += 1
                s += 1
                if s == self.nbyte:
                    s, phase = 0, phase ^ 1
                yield
            ok = ok and not c.abort
            if not ok:
                c.abort = True
                break
        for i in range(max(0, n - self.nbyte), 0 if self.own_drain and ok else n):
            got = yield from self.wait(c.bfull[i % self.nfull], (i // self.nfull) & 1, DRAIN)
            assert got, "a closing wait ran out"
        yield from self.finish(c)

    def await_commits(self, c, ncommit, nchunk):
        for i in range(max(0, ncommit - NF), ncommit):
            got = yield from self.wait(c.fempty[i % NF], (i // NF) & 1, DRAIN)
            assert got, "a closing wait ran out"
        for i in range(max(0, nchunk - 2), nchunk):
            got = yield from self.wait(c.tfull[i & 1], (i >> 1) & 1, DRAIN)
            assert got, "a closing wait ran out"

    def commit(self, c, name, index):
        for to in self.ctas[c.pair]:
            self.commits.append((c.pair, self.mma_issued[c.pair], to, getattr(to, name)[index]))

    def products(self, c):
        f = phase = chunk = ncommit = step = 0
        ok = True
        for t in range(self.tiles):
            for k in range(self.nchunks()):
                b, use = chunk & 1, (chunk >> 1) & 1
                ok = yield from self.wait(c.tempty[b], use ^ 1)
                if not ok or c.abort:
                    ok = False
                    break
                for _ in range(min(self.chunk, self.nk - k * self.chunk) * HALVES):
                    ok = yield from self.wait(c.ffull[f], phase)
                    if not ok:
                        break
                    for x in self.ctas[c.pair]:
                        if x.wide[f] != step:
                            self.faults.append("a product of the wrong codes")
                    step += 1
                    self.mma_issued[c.pair] += 1
                    self.queue[c.pair].append((b, (t, k)))
                    self.commit(c, "fempty", f)
                    ncommit += 1
                    f += 1
                    if f == NF:
                        f, phase = 0, phase ^ 1
                    yield
                if not ok:
                    break
                self.commit(c, "tfull", b)
                chunk += 1
            if not ok:
                self.give_up(c)
                break
        yield from self.await_commits(c, ncommit, chunk)
        self.ctas[c.pair][1].issued = (ncommit, chunk)
        yield from self.finish(c)

    def second(self, c):
        """The role of the second CTA's warp that issues nothing."""
        if self.early_wait:             # a wait that starts before the commits are issued
            n = self.tiles * self.nk * HALVES
            for i in range(max(0, n - NF), n):
                for _ in range(DRAIN):
                    if c.abort or c.fempty[i % NF].try_wait((i // NF) & 1):
                        break
                    yield
        yield from self.finish(c)

    def widen(self, c, g):
        load, f, bphase, fphase = g // HALVES, g, 0, 0
        ok = True
        for i in range(g // HALVES, self.tiles * self.nk, TURNS):
            ok = yield from self.wait(c.bfull[load], bphase)
            if not ok:
                break
            s = load % self.nbyte
            if c.holds[s] != i:
                self.faults.append("a stage's old bytes are read")
            ok = yield from self.wait(c.fempty[f], fphase ^ 1)
            if not ok:
                break
            if c.holds[s] != i:
                self.faults.append("a stage is overwritten while it is read")
            c.bempty[s].arrive()
            yield
            c.wide[f] = HALVES * i + g % HALVES
            self.ctas[c.pair][0].ffull[f].arrive()
            load += TURNS
            while load >= self.nfull:
                load, bphase = load - self.nfull, bphase ^ 1
            f += GROUPS
            while f >= NF:
                f, fphase = f - NF, fphase ^ 1
            yield
        if not ok:
            self.give_up(c)
        yield from self.finish(c)

    def drain(self, c, w):
        chunk = 0
        ok = True
        for t in range(self.tiles):
            for k in range(self.nchunks()):
                ok = yield from self.wait(c.tfull[chunk & 1], (chunk >> 1) & 1)
                if not ok or c.abort:
                    ok = False
                    break
                if self.split and k == self.nchunks() - 1:
                    yield from self.cluster_sync()
                want = min(self.chunk, self.nk - k * self.chunk) * HALVES
                yield
                if self.acc[c.pair][chunk & 1] != ((t, k), want):
                    self.faults.append("sums of the wrong chunk")
                c.read.add((w, t, k))
                self.ctas[c.pair][0].tempty[chunk & 1].arrive()
                chunk += 1
                yield
            if not ok:
                self.give_up(c)
                break
            if self.split:
                yield from self.cluster_sync()
        yield from self.finish(c, synced=self.split and self.tiles > 0 and ok)

    # ---- the closing part, the same for every role ----------------------------------
    def finish(self, c, synced=False):
        if self.split and not synced:
            yield from self.cluster_sync()
            yield from self.cluster_sync()
        c.at_block += 1
        while c.at_block < self.roles_per_cta:
            yield
        yield from self.cluster_sync()
        c.left += 1
        while c.left < self.roles_per_cta:
            yield
        if c.left == self.roles_per_cta:            # one agent closes for the CTA
            c.left += 1
            if c.rank == 1 and not self.early_wait:
                yield from self.await_commits(c, *c.issued)
            if c.coming:
                self.faults.append("a copy is still in flight")
            if any(to is c for _, _, to, _ in self.commits):
                self.faults.append("a commit may arrive in a CTA that has gone")
            if self.mma_done[c.pair] != self.mma_issued[c.pair]:
                self.faults.append("a product is still running")

    # ---- what runs by itself -----------------------------------------------------
    def engine(self):
        some = []
        if self.fills:
            some.append("copy")
        some += ["mma"] * any(d < i for d, i in zip(self.mma_done, self.mma_issued))
        ready = [x for x in self.commits if x[1] <= self.mma_done[x[0]]]
        if ready:
            some.append("commit")
        if not some:
            return
        kind = self.rng.choice(some)
        if kind == "copy":
            c, s, n = self.fills.pop(self.rng.randrange(len(self.fills)))
            c.coming -= 1
            c.holds[s] = n
            c.bfull[n % self.nfull].arrive()
        elif kind == "mma":
            p = self.rng.choice([p for p in range(len(self.ctas))
                                 if self.mma_done[p] < self.mma_issued[p]])
            b, chunk = self.queue[p][self.mma_done[p]]
            at, n = self.acc[p][b]
            self.acc[p][b] = (chunk, n + 1 if at == chunk else 1)
            self.mma_done[p] += 1
        else:
            x = self.rng.choice(ready)
            self.commits.remove(x)
            x[3].arrive()

    def run(self, p_engine):
        roles = []
        for c in self.flat:
            roles += [self.copies(c), self.products(c) if c.rank == 0 else self.second(c)]
            roles += [self.widen(c, g) for g in range(GROUPS)]
            roles += [self.drain(c, w) for w in range(self.warps)]
        steps = 0
        while roles:
            steps += 1
            assert steps < 3_000_000, "the cluster never ends"
            if self.rng.random() < p_engine:
                self.engine()
                continue
            r = self.rng.choice(roles)
            try:
                next(r)
            except StopIteration:
                roles.remove(r)
        return self


def _shape(rng):
    pairs = rng.choice([1, 1, 2, 3, 4])
    return dict(pairs=pairs, tiles=rng.randint(1, 3), nk=rng.randint(1, 9),
                chunk=rng.choice([1, 2, 3]), nbyte=rng.choice([2, 3, 5]),
                warps=rng.choice([1, 2]))


@pytest.mark.parametrize("seed", range(40))
def test_without_timeouts_everything_is_read_and_nothing_is_left(seed):
    rng = random.Random(seed)
    shape = _shape(rng)
    c = Cluster(seed, limit=DRAIN, **shape).run(rng.choice([0.1, 0.3, 0.6]))
    assert c.timeouts == 0 and not c.faults, c.faults
    for cta in c.flat:
        assert cta.read == {(w, t, k) for w in range(c.warps) for t in range(c.tiles)
                            for k in range(c.nchunks())}


@pytest.mark.parametrize("seed", range(60))
def test_timeouts_anywhere_leave_nothing_in_flight(seed):
    rng = random.Random(1000 + seed)
    shape = _shape(rng)
    c = Cluster(seed, limit=rng.choice([1, 2, 8, 40, 300]), **shape).run(
        rng.choice([0.05, 0.2, 0.5]))
    assert not c.faults, c.faults


def test_a_cluster_without_a_tile_goes():
    for pairs in (1, 2, 4):
        c = Cluster(1, pairs, 1, 4, 2, 3, 2, DRAIN, idle=True).run(0.2)
        assert not c.faults and c.timeouts == 0


def test_a_wait_that_starts_before_the_commits_guards_nothing():
    """Why the second CTA waits at the end and not from the start: a phase's
    parity is also that of the phase two uses back, and of a fresh barrier."""
    left = 0
    for seed in range(60):
        c = Cluster(seed, 1, 1, 6, 2, 3, 1, DRAIN, early_wait=True).run(0.02)
        left += "a commit may arrive in a CTA that has gone" in c.faults
    assert left > 0


def test_copies_are_waited_for_also_when_another_role_gave_up():
    """A copying warp that waits only after a timeout of its own leaves copies
    behind that a widening warp no longer waits for."""
    left = 0
    for seed in range(60):
        c = Cluster(seed, 1, 1, 3, 2, 5, 1, 3, own_drain=True).run(0.02)
        left += "a copy is still in flight" in c.faults
    assert left > 0
    kernel = _code().split("linear_i8_tile_kernel", 1)[1]
    role = kernel[kernel.index("tensor_load_2d"):kernel.index("cluster_wait_all();")]
    own = role[role.index("if (!ok) {"):]
    assert own.index("}") < own.index("bar_wait(bfull(i %")


def test_a_turn_that_skips_the_other_turns_phases_reads_old_bytes():
    """Why a byte stage has a barrier per turn: with one per stage and three stages, a
    group does not see the other turn's phases, and the parity it waits for is
    already true.  (With five, the fp16 stages keep the turns close enough.)"""
    def faults(nbyte, stage_barriers):
        found = 0
        for seed in range(80):
            c = Cluster(seed, 1, 2, 8, 2, nbyte, 1, DRAIN, stage_barriers=stage_barriers)
            try:
                c.run(0.05)
            except AssertionError:       # the barriers run out of step after it
                pass
            found += "a stage's old bytes are read" in c.faults
        return found

    assert faults(3, True) > 0
    for nbyte in (2, 3, 4, 5, 7):
        assert faults(nbyte, False) == 0
    kernel = _code().split("linear_i8_tile_kernel", 1)[1]
    assert "role_wait(bfull(load), bphase)" in kernel
    assert re.search(r"\(load \+= kTurns\) >= kTurns \* nbyte", kernel)
    assert "bar_init(bfull(lane), 1)" in kernel and "lane < kTurns * nbyte" in kernel


def _code():
    text = open(SOURCE).read()
    return re.sub(r"//[^\n]*", "", text)


def test_the_kernel_waits_for_the_commits_after_the_closing_barrier():
    kernel = _code().split("linear_i8_tile_kernel", 1)[1]
    kernel = re.sub(r"\n\s*\n", "\n", kernel)
    close = kernel[kernel.index("__syncthreads();\n  cluster_sync();"):]
    at = close.index("await_commits(smem_load(issued), smem_load(issued + 4))")
    assert close.index("cluster_sync()") < at < close.index("pair_tmem_free")
    # no role of the second CTA looks at the commits' parity on its own before that
    assert "bar_poll" not in kernel
    # both counts are handed over; the first CTA, whose role waits by itself, has none left
    assert kernel.count("cluster_store(to") == 2
    assert "smem_store(issued, 0)" in kernel and "smem_store(issued + 4, 0)" in kernel
    assert "await_commits(ncommit, chunk)" in kernel
