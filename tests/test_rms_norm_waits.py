"""The norm's gradient where a wait for a row runs out.

On the CPU: a step-by-step model of a team's ring of rows (bulk copies that land when they
like, threads that reach their waits in any order, waits that give up anywhere).  No row is
asked for in a place whose last phase is still open, no copy lands once the team has gone, no
place is written while a thread may read it, no barrier waits for a thread that has left.
The model also shows that asking for rows after a wait that ran out breaks the first two.

On the GPU: calls whose waits give up at once or here and there must end, report
MOE_ERR_TIMEOUT, write rows of d_x whole and as the normal call does or not at all, nothing
outside, and leave the GPU as a normal call right behind them needs it."""
import ctypes
import os
import random
import re

import pytest
import torch

import plain_f8 as P

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "combine_moe_dispatch_layout_gb300", "csrc", "rms_norm.cu")


class Fault(Exception):
    pass


class Place:
    """A row of the ring with its barrier (one arrival, and the bytes it announces)."""

    def __init__(self):
        self.done = 0              # phases completed
        self.coming = False        # a copy announced and not landed
        self.row = None
        self.readers = set()

    def ask(self, row):
        if self.coming:
            raise Fault("a row asked for while the place's phase is open")
        if self.readers:
            raise Fault("a row asked for while another is read")
        self.coming, self.next = True, row

    def land(self):
        self.row, self.coming = self.next, False
        self.done += 1

    def passed(self, parity):
        return self.done % 2 != parity


class Team:
    """Threads 0 .. n-1 (0 asks for rows), rows 0 .. rows-1; odds: one wait in so many gives
    up.  asks_on: thread 0 goes on asking after a wait that ran out, and each thread skips
    only its own waits."""

    def __init__(self, rng, n, rows, depth, odds, asks_on=False):
        self.rng, self.n, self.rows, self.depth, self.odds = rng, n, rows, depth, odds
        self.asks_on = asks_on
        self.ring = [Place() for _ in range(depth)]
        self.gave_up = [False, False]
        self.at_barrier, self.left, self.written = set(), set(), []
        self.round = 0

    def fetch(self, row, at):
        if row < self.rows:
            self.ring[at].ask(row)

    def thread(self, i):
        if i == 0:
            for r in range(self.depth):
                self.fetch(r, r)
        at, phase, turn, ok, row = 0, 0, 0, True, 0
        while row < self.rows:
            place = self.ring[at]
            landed = ok
            if ok:
                if self.rng.random() * self.odds < 1:
                    landed = False
                else:
                    while not place.passed(phase):
                        yield "wait"
            if not landed:
                if self.asks_on:
                    ok = False
                else:
                    self.gave_up[turn] = True
            else:
                place.readers.add(i)
                if place.row != row:
                    raise Fault("read row %s for row %d" % (place.row, row))
            yield "reduce"
            yield "barrier"
            if not self.asks_on and self.gave_up[turn]:
                place.readers.discard(i)
                ok = False
                break
            if i == 0 and row:
                self.fetch(row + self.depth - 1, (at - 1) % self.depth)
            yield "second pass"
            place.readers.discard(i)
            if i == 0 and ok:
                self.written.append(row)
            at += 1
            if at == self.depth:
                at, phase = 0, phase ^ 1
            row, turn = row + 1, turn ^ 1
        if not ok and self.asks_on:
            for place in self.ring:             # a phase of either parity
                for parity in (0, 1):
                    while not place.passed(parity):
                        yield "closing"
                        if not any(q.coming for q in self.ring):
                            break
        elif not ok:
            left = self.depth if row == 0 else self.depth - 1
            while left > 0 and row < self.rows:
                while not self.ring[at].passed(phase):
                    yield "closing"
                at += 1
                if at == self.depth:
                    at, phase = 0, phase ^ 1
                left, row = left - 1, row + 1

    def run(self):
        threads = {i: self.thread(i) for i in range(self.n)}
        state = {}
        for _ in range(100000):
            if not threads:
                break
            copies = [p for p in self.ring if p.coming]
            ready = [i for i in threads if i not in self.at_barrier]
            if copies and (not ready or self.rng.random() < 0.2):
                self.rng.choice(copies).land()
                continue
            if not ready:
                if len(self.at_barrier) < self.n:
                    raise Fault("a barrier waits for a thread that has left")
                self.at_barrier.clear()
                continue
            i = self.rng.choice(ready)
            try:
                state[i] = next(threads[i])
                if state[i] == "barrier":
                    self.at_barrier.add(i)
            except StopIteration:
                del threads[i]
            if len(self.at_barrier) == self.n:
                self.at_barrier.clear()
        else:
            raise Fault("the team does not end")
        if any(p.coming for p in self.ring):
            raise Fault("a copy lands once the team has gone")


def test_model_of_the_ring():
    rng = random.Random(1)
    cut = 0
    for trial in range(3000):
        rows, depth = rng.randint(1, 14), rng.randint(2, 4)
        odds = rng.choice([1, 3, 10, 40, 1e9])
        t = Team(rng, rng.choice([1, 2, 4]), rows, depth, odds)
        t.run()
        assert t.written == list(range(len(t.written)))
        assert odds < 1e9 or len(t.written) == rows
        assert odds > 1 or not t.written
        cut += len(t.written) < rows
    assert cut > 1000


def test_model_catches_rows_asked_for_after_a_timeout():
    rng = random.Random(2)
    faults = set()
    for trial in range(2000):
        try:
            Team(rng, 1, rng.randint(6, 14), rng.randint(2, 4), 5, asks_on=True).run()
        except Fault as e:
            faults.add(str(e))
    assert {"a row asked for while the place's phase is open",
            "a copy lands once the team has gone"} & faults


def test_the_kernel_leaves_before_it_asks():
    """In the row loop: a way out, by what the team's threads found, stands between the
    wait and the next fetch and the row's stores."""
    src = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    body = src[src.index("rms_norm_backward_kernel("):]
    loop = body[body.index("for (; row < p.T;"):body.index("set_status(p.dev_status")]
    order = ["ok = row_wait(", "ok = __all_sync(kAll, ok)", "s_part[turn][kGaveUp] = 1.0f",
             "row_reduce<TPR>(dot", "ok = s_part[turn][kGaveUp] == 0.0f", "if (!ok) break;",
             "fetch(row +", "*reinterpret_cast<uint4*>(dx"]
    assert [loop.count(w) for w in order] == [1] * len(order)
    assert sorted(order, key=loop.index) == order


# ---- on the GPU ------------------------------------------------------------------------

@pytest.fixture(scope="module")
def ep():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a CUDA device")
    import combine_moe_dispatch_layout_gb300 as ep
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    fn = ep.lib().moe_test_rms_norm_backward_odds
    fn.argtypes = [vp, i64, i32, i64, vp, i64, vp, vp, vp, i64, vp, i64, vp, ctypes.c_uint32,
                   vp, vp]
    fn.restype = ctypes.c_int
    return ep


# every width that a kernel is compiled for; rows of all CTAs, of some, and one
@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(20000, 504), (9000, 1000), (1, 1000), (3000, 2048), (304, 4096),
                                 (2500, 7168), (1200, 16384), (3, 16384)])
@pytest.mark.parametrize("with_sum", [True, False])
@pytest.mark.parametrize("odds", [1, 20, 1000, 50000, 1 << 30])
def test_waits_that_run_out(ep, T, H, with_sum, odds):
    g = torch.Generator(device="cuda")
    g.manual_seed(T + H)

    def rows():
        return torch.randn((T, H), generator=g, device="cuda").bfloat16()

    x, dy, ds = rows(), rows(), rows() if with_sum else None
    gamma = 1 + 0.3 * torch.randn(H, generator=g, device="cuda")
    rstd = P.norm(x, None, gamma, 1e-6)[1][:, 0].float()
    raw = torch.empty((T + 2, H), dtype=torch.bfloat16, device="cuda")
    dx = raw[1:T + 1]
    dg = torch.empty(H, device="cuda")
    ws = torch.empty(ep.rms_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def normal():
        ep.moe_rms_norm_backward(dy, x, gamma, rstd, ds, dx, dg, ws, st)

    normal()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    want, want_g = dx.clone(), dg.clone()
    for _ in range(3):
        raw.fill_(-7.0)
        rc = ep.lib().moe_test_rms_norm_backward_odds(
            dy.data_ptr(), T, H, H, x.data_ptr(), H, gamma.data_ptr(), rstd.data_ptr(),
            ds.data_ptr() if with_sum else None, H, dx.data_ptr(), H, ws.data_ptr(), odds,
            st.data_ptr(), torch.cuda.current_stream().cuda_stream)
        got = raw.clone()
        code = st.clone()
        st.zero_()
        normal()                                    # right behind it
        torch.cuda.synchronize()
        assert rc == 0 and int(st.item()) == 0
        assert torch.equal(dx, want) and torch.equal(dg, want_g)
        assert bool((got[0] == -7).all()) and bool((got[-1] == -7).all())
        status, got = int(code.item()), got[1:-1]
        assert status in (0, ep.MOE_ERR_TIMEOUT)
        left = (got == -7.0).all(1)
        assert torch.equal(got[~left], want[~left])
        if status == 0:
            assert torch.equal(got, want)
        if odds == 1:
            assert status == ep.MOE_ERR_TIMEOUT and bool(left.all())
        if odds == 1 << 30:
            assert int((~left).sum()) > 0
