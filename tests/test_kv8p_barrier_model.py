"""A host model of the barrier protocol of the attention over page scales (csrc/attn_kv8p.cu): two
TMA producers, four converter warps, two MMA issuers with a queue each, two slots of four softmax
warps; of two row tiles each slot takes every block, of one the slots take the blocks in turn.
Random delays; every wait is by parity and is checked against the phase it means, every stage
against the block that should stand in it. Mistakes are planted in the model to see that it finds
them."""

import heapq
import itertools
import random

import pytest

K, C, V = 8, 6, 2        # stages of K, of V's codes, of V
GROUPS, GROUP = 4, 8     # groups of page scales kept, blocks of a group


class Fault(Exception):
    pass


class Bar:
    def __init__(self, need):
        self.need, self.got, self.done, self.waiters = need, 0, 0, []

    def arrive(self, sim):
        self.got += 1
        if self.got > self.need:
            raise Fault("more arrivals than a phase has")
        if self.got == self.need:
            self.got, self.done = 0, self.done + 1
            for w in self.waiters:
                sim.at(0, w)
            self.waiters = []

    def passes(self, phase):
        """What a parity wait sees; a pass has to mean that phase, not one two away."""
        if (self.done & 1) != (phase & 1):
            if self.done != phase + 1:
                raise Fault(f"a wait for phase {phase} passed with {self.done} complete")
            return True
        if self.done > phase:
            raise Fault(f"a wait for phase {phase} misses it: {self.done} complete")
        return False


class Sim:
    def __init__(self, seed, heavy):
        self.rng, self.heavy = random.Random(seed), heavy
        self.now, self.q, self.tie = 0.0, [], itertools.count()

    def at(self, dt, fn):
        heapq.heappush(self.q, (self.now + dt, next(self.tie), fn))

    def delay(self, mean):
        r = self.rng
        return mean * (r.paretovariate(1.2) if self.heavy else r.uniform(0.1, 2.0))

    def spawn(self, gen):
        def step():
            try:
                what = next(gen)
            except StopIteration:
                self.live -= 1
                return
            if isinstance(what, tuple):
                bar, phase = what

                def retry():
                    if bar.passes(phase):
                        step()
                    else:
                        bar.waiters.append(retry)
                retry()
            else:
                self.at(self.delay(what), step)
        self.live = getattr(self, "live", 0) + 1
        self.at(self.delay(1), step)

    def run(self):
        while self.q:
            self.now, _, fn = heapq.heappop(self.q)
            fn()
        if self.live:
            raise Fault(f"{self.live} roles wait for ever")


def kernel(seed, nb, tiles, heavy=False, mistake=None, kst=K, vst=V):
    s = Sim(seed, heavy)
    step = 1 if tiles == 2 else 2
    k_full, k_empty = [Bar(1) for _ in range(kst)], [Bar(tiles) for _ in range(kst)]
    c_full, c_empty = [Bar(1) for _ in range(C)], [Bar(4) for _ in range(C)]
    v_full, v_empty = [Bar(4) for _ in range(vst)], [Bar(tiles) for _ in range(vst)]
    s_full, p_full, pv_done = ([[Bar(n) for _ in range(2)] for _ in range(2)] for n in (1, 4, 1))
    sc_full = [Bar(1) for _ in range(2)]
    k_in, c_in, v_in = [None] * kst, [None] * C, [[None] * 4 for _ in range(vst)]
    k_use, v_use = [0] * kst, [0] * vst                   # products reading the stage
    scales = [None] * GROUPS
    S = [[None, None], [None, None]]
    P = [[[None] * 4, [None] * 4] for _ in range(2)]
    pv_started, pv_ended = [-1, -1], [-1, -1]
    queue, busy = [[], []], [False, False]

    def expect(ok, what):
        if not ok:
            raise Fault(what)

    def produce(full, empty, held, use, depth, with_scales):
        for j in range(nb):
            st = j % depth
            if j >= depth and not (mistake == "no wait" and with_scales):
                yield empty[st], j // depth - 1
            expect(use is None or use[st] == 0, "a copy into a stage that is being read")
            held[st] = None

            def land(st=st, j=j):
                held[st] = j
                full[st].arrive(s)
            s.at(s.delay(8), land)
            if with_scales and j % GROUP == 0:
                scales[j // GROUP % (2 if mistake == "two groups" else GROUPS)] = j // GROUP
                sc_full[j // GROUP & 1].arrive(s)
            yield 1

    def convert(w):
        for j in range(nb):
            yield c_full[j % C], j // C
            expect(c_in[j % C] == j, "another block's codes")
            if j >= vst:
                yield v_empty[j % vst], j // vst - 1
            expect(v_use[j % vst] == 0, "V written while products read it")
            yield 6
            v_in[j % vst][w] = j
            v_full[j % vst].arrive(s)
            c_empty[j % C].arrive(s)

    def pump(t):
        """The tensor cores' queue of an issuer: one product batch after the other, in order."""
        if busy[t] or not queue[t]:
            return
        start, end, cost = queue[t].pop(0)
        busy[t] = True
        start()

        def finish():
            end()
            busy[t] = False
            pump(t)
        s.at(s.delay(cost), finish)

    def issue(t):
        j0 = 0 if tiles == 2 else t

        def qk(j, n):
            def start():
                expect(k_in[j % kst] == j, "QK over another block's K")
                k_use[j % kst] += 1
                S[t][n & 1] = None

            def end():
                expect(k_in[j % kst] == j, "K overwritten under QK")
                k_use[j % kst] -= 1
                S[t][n & 1] = n
                s_full[t][n & 1].arrive(s)
                k_empty[j % kst].arrive(s)
            queue[t].append((start, end, 4))
            pump(t)

        if j0 >= nb:
            return
        yield k_full[j0 % kst], j0 // kst
        qk(j0, 0)
        for n, j in enumerate(range(j0, nb, step)):
            if j + step < nb:
                yield k_full[(j + step) % kst], (j + step) // kst
                qk(j + step, n + 1)
            yield v_full[j % vst], j // vst
            yield p_full[t][n & 1], n >> 1

            def start(j=j, n=n):
                expect(v_in[j % vst] == [j] * 4, "PV over another block's V")
                expect(P[t][n & 1] == [n] * 4, "PV over another block's P")
                v_use[j % vst] += 1
                pv_started[t] = n

            def end(j=j, n=n):
                expect(P[t][n & 1] == [n] * 4 and v_in[j % vst] == [j] * 4, "P or V overwritten under PV")
                v_use[j % vst] -= 1
                pv_ended[t] = n
                pv_done[t][n & 1].arrive(s)
                v_empty[j % vst].arrive(s)
            queue[t].append((start, end, 4))
            pump(t)

    def softmax(t, w):
        n = -1
        for n, j in enumerate(range(0 if tiles == 2 else t, nb, step)):
            if j % GROUP < step:
                yield sc_full[j // GROUP & 1], j // GROUP >> 1
            yield s_full[t][n & 1], n >> 1
            expect(S[t][n & 1] == n, "another block's S")
            yield 5 if w else 0.2                           # (a warp without rows is quick)
            at = j // GROUP % (2 if mistake == "two groups" else GROUPS)
            expect(scales[at] == j // GROUP, "another group's scales")
            if n and s.rng.random() < 0.2:                   # M moves: O is rescaled
                if mistake != "no pv wait":
                    yield pv_done[t][n - 1 & 1], n - 1 >> 1
                expect(pv_ended[t] == n - 1 and pv_started[t] == n - 1, "O rescaled under PV")
                yield 3
                expect(pv_started[t] == n - 1, "PV began under the rescaling")
            P[t][n & 1][w] = n
            p_full[t][n & 1].arrive(s)
        if n >= 0:
            yield pv_done[t][n & 1], n >> 1
            expect(pv_ended[t] == n, "O read before its last products")

    s.spawn(produce(k_full, k_empty, k_in, k_use, kst, True))
    s.spawn(produce(c_full, c_empty, c_in, None, C, False))
    for w in range(4):
        s.spawn(convert(w))
    for t in range(2):
        s.spawn(issue(t))
        for w in range(4):
            s.spawn(softmax(t, w))
    s.run()


@pytest.mark.parametrize("heavy", [False, True])
@pytest.mark.parametrize("tiles", [1, 2])
def test_protocol(tiles, heavy):
    for seed in range(60):
        for nb in (1, 2, 3, 7, 8, 9, 31, 70):
            kernel(1000 * seed + nb, nb, tiles, heavy)


@pytest.mark.parametrize("tiles,kw", [
    (2, dict(mistake="no wait")), (1, dict(mistake="no pv wait")), (2, dict(mistake="no pv wait")),
    (1, dict(mistake="two groups")), (2, dict(mistake="two groups")),
    (1, dict(kst=3))])      # an odd number of stages: a slot does not see each phase
def test_planted_mistakes_are_found(tiles, kw):
    found = 0
    for seed in range(200):
        try:
            kernel(seed, 70, tiles, heavy=seed % 2 == 0, **kw)
        except Fault:
            found += 1
    assert found > 0
