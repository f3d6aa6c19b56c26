"""A host model of the barrier protocol of the attention over a 4-bit cache (csrc/attn_kv4.cu): two producers, the first of
which says what the CTA's runs of blocks are, converters of K and of V in one or two groups, two MMA issuers with a queue
each, two slots of one or two groups of softmax warps; of 128 rows each slot takes every block, below that the slots take
the blocks in turn, so that a run of one block leaves a slot without any. Random delays; every wait is by parity and is checked
against the phase it means, every buffer against what should stand in it. Mistakes are planted in the model to
see that it finds them."""

import random
import re
from pathlib import Path

import pytest

from test_kv8p_barrier_model import Bar, Fault, Sim

SEGS = 4
# rows: (each slot has its own half of the rows, groups of converters an operand, softmax groups a slot, stages)
SHAPES = {16: (False, 2, 1, 6), 32: (False, 2, 1, 6), 64: (False, 1, 2, 5), 128: (True, 1, 2, 4)}


def kernel(seed, runs, rows, heavy=False, mistake=None, stages=None):
    """runs: (blocks, prefix blocks among them) of each run, in order."""
    dual, conv, groups, depth = SHAPES[rows]
    depth = stages or depth
    s = Sim(seed, heavy)
    step = 1 if dual else 2
    runs = list(runs) + [(0, 0)]
    full, empty = [Bar(1) for _ in range(depth)], [Bar(8) for _ in range(depth)]
    t_full = {x: [Bar(4) for _ in range(2)] for x in "kv"}
    t_free = {x: [Bar(2 if dual else 1) for _ in range(2)] for x in "kv"}
    s_full, s_free = [Bar(1) for _ in range(2)], [Bar(4 * groups) for _ in range(2)]
    p_full, pv_done = ([[Bar(n) for _ in range(2)] for _ in range(2)] for n in (4 * groups, 1))
    q_full = [Bar((4 if dual else 8) * groups) for _ in range(2)]
    seg_full, seg_empty = [Bar(1) for _ in range(SEGS)], [Bar(3 + 8 * groups + 8 * conv) for _ in range(SEGS)]
    meet_all, meet_slot = Bar(8 * groups), [Bar(4 * groups) for _ in range(2)]
    meet_group = [[Bar(4) for _ in range(groups)] for _ in range(2)]
    seg = [None] * SEGS
    held = [None] * depth
    wide = {x: [[None] * 4 for _ in range(2)] for x in "kv"}
    using = {x: [0, 0] for x in "kv"}                                # products that read the buffer
    q_in, q_use = [[None] * (4 * groups) for _ in range(2)], [0, 0]  # (of shared q: each slot's view of the same rows)
    S = [None, None]
    P = [[[None] * (4 * groups), [None] * (4 * groups)] for _ in range(2)]
    pv_started, pv_ended, done = [-1, -1], [-1, -1], [-1, -1]
    votes = [[set() for _ in range(groups)] for _ in range(2)]
    queue, busy = [[], []], [False, False]

    def expect(ok, what):
        if not ok:
            raise Fault(what)

    def at_seg(n):
        expect(seg[n % SEGS] is not None and seg[n % SEGS][0] == n, "another run's sizes")
        return seg[n % SEGS][1:]

    def copies(me, state, nb):
        for _ in range(nb):
            i = state["i"]
            st, turn = i % depth, i // depth
            state["i"] += 1
            if i % 2 != me:
                continue
            if turn > 0:
                yield empty[st], turn - 1
            held[st] = None

            def land(st=st, i=i):
                held[st] = i
                full[st].arrive(s)
            s.at(s.delay(8), land)
            yield 1

    def producer():
        state = {"i": 0}
        for n, (nb, np) in enumerate(runs):
            if n >= SEGS:
                yield seg_empty[n % SEGS], n // SEGS - 1
            seg[n % SEGS] = (n, nb, np)
            seg_full[n % SEGS].arrive(s)
            yield from copies(0, state, nb)

    def producer2():
        state = {"i": 0}
        for n in range(len(runs)):
            yield seg_full[n % SEGS], n // SEGS
            nb, _ = at_seg(n)
            seg_empty[n % SEGS].arrive(s)
            yield from copies(1, state, nb)

    def converter(x, group, w):
        i = 0
        for n in range(len(runs)):
            yield seg_full[n % SEGS], n // SEGS
            nb, _ = at_seg(n)
            seg_empty[n % SEGS].arrive(s)
            yield 0.2
            for _ in range(nb):
                st, turn, b = i % depth, i // depth, i & 1
                i += 1
                if conv == 2 and (i - 1) % 2 != group:
                    continue
                yield full[st], turn
                expect(held[st] == i - 1, "another block's records")
                if i - 1 >= 2:
                    yield t_free[x][b], (i - 1 >> 1) - 1
                expect(using[x][b] == 0, "an operand written while products read it")
                yield 5
                expect(held[st] == i - 1, "records overwritten while they are widened")
                wide[x][b][w] = i - 1
                empty[st].arrive(s)
                yield 0.2
                t_full[x][b].arrive(s)

    def pump(t):
        if busy[t] or not queue[t]:
            return
        start, end = queue[t].pop(0)
        busy[t] = True
        start()

        def finish():
            end()
            busy[t] = False
            pump(t)
        s.at(s.delay(4), finish)

    def issuer(t):
        i = n_qk = n_pv = n_q = 0

        def qk(at, run):
            nonlocal n_qk
            yield t_full["k"][at & 1], at >> 1
            if n_qk > 0:
                yield s_free[t], n_qk - 1
            n = n_qk

            def start():
                expect(wide["k"][at & 1] == [at] * 4, "QK over another block's K")
                expect(q_in[t] == [run] * len(q_in[t]), "QK over another tile's q")
                using["k"][at & 1] += 1
                q_use[t] += 1
                S[t] = None

            def end():
                expect(q_in[t] == [run] * len(q_in[t]), "q overwritten under QK")
                using["k"][at & 1] -= 1
                q_use[t] -= 1
                S[t] = n
                s_full[t].arrive(s)
                t_free["k"][at & 1].arrive(s)
            queue[t].append((start, end))
            pump(t)
            n_qk += 1

        for run in range(len(runs)):
            yield seg_full[run % SEGS], run // SEGS
            nb, _ = at_seg(run)
            seg_empty[run % SEGS].arrive(s)
            if nb == 0:
                break
            yield 300 if s.rng.random() < 0.05 else 0.2     # (nothing says how soon a warp goes on)
            k0 = 0 if dual else (i ^ t) & 1
            if mistake == "an idle slot waits for q":
                yield q_full[t], run
            elif mistake == "an idle slot's tiles count" and k0 < nb:
                yield q_full[t], run
            elif k0 < nb:
                yield q_full[t], n_q
                n_q += 1
            if k0 < nb:
                yield from qk(i + k0, run)
            for k in range(k0, nb, step):
                if k + step < nb:
                    yield from qk(i + k + step, run)
                at, buf, n = i + k, n_pv & 1, n_pv
                yield t_full["v"][at & 1], at >> 1
                yield p_full[t][buf], n_pv >> 1

                def start(at=at, buf=buf, n=n):
                    expect(wide["v"][at & 1] == [at] * 4, "PV over another block's V")
                    expect(P[t][buf] == [n] * len(P[t][buf]), "PV over another block's P")
                    using["v"][at & 1] += 1
                    pv_started[t] = n

                def end(at=at, buf=buf, n=n):
                    expect(P[t][buf] == [n] * len(P[t][buf]), "P overwritten under PV")
                    using["v"][at & 1] -= 1
                    pv_ended[t] = n
                    pv_done[t][buf].arrive(s)
                    t_free["v"][at & 1].arrive(s)
                queue[t].append((start, end))
                pump(t)
                n_pv += 1
            i += nb

    moves = random.Random(seed + 1)
    moved = {}

    def moves_at(*key):     # the same answer for all of a group's warps
        if key not in moved:
            moved[key] = moves.random() < 0.2
        return moved[key]

    def softmax(slot, g, w):
        me = 4 * g + w
        gen = {}
        i = n = 0

        def meet(bar):
            phase = gen.get(id(bar), 0)
            gen[id(bar)] = phase + 1
            bar.arrive(s)
            yield bar, phase

        def move(first):
            yield from meet(meet_group[slot][g])
            yield 0.2
            yield from meet(meet_group[slot][g])
            if first or not moves_at(slot, g, n):
                return
            if mistake != "no wait before O is rescaled":
                yield pv_done[slot][n - 1 & 1], n - 1 >> 1
            expect(pv_ended[slot] == n - 1 and pv_started[slot] == n - 1, "O rescaled under PV")
            yield 3
            expect(pv_started[slot] == n - 1, "PV began under the rescaling")

        for run in range(len(runs)):
            if run == 0:
                yield seg_full[0], 0
                yield from meet(meet_all)
            nb, np = at_seg(run)
            if nb == 0:
                break
            yield 2
            for t in (slot,) if dual else (0, 1):
                expect(q_use[t] == 0, "q written while products read it")
            q_in[slot][me] = run
            yield 0.2
            mine = [(i ^ t) & 1 < nb for t in range(2)]
            if dual:
                q_full[slot].arrive(s)
                yield from meet(meet_slot[slot])
            else:
                for t in range(2):
                    if mine[t] or mistake in ("an idle slot waits for q", "an idle slot's tiles count"):
                        q_full[t].arrive(s)
                yield from meet(meet_all)
            k0 = 0 if dual else (i ^ slot) & 1
            for k in range(k0, nb, step):
                first = k == k0
                yield s_full[slot], n
                expect(S[slot] == n, "another block's S")
                yield 1
                expect(S[slot] == n, "S overwritten while it is read")
                if k < np:
                    if not first and moves_at(slot, g, n) and w == 1:
                        votes[slot][g].add(n)
                    s_free[slot].arrive(s)
                    if first:
                        yield from move(True)
                    yield 5
                    if not first:
                        yield s_free[slot], n
                        if n in votes[slot][g]:
                            yield from move(False)
                            yield 5
                else:
                    s_free[slot].arrive(s)
                    yield from move(first)
                    if not first and mistake != "V's wait alone":
                        yield pv_done[slot][n - 1 & 1], n - 1 >> 1
                    if mistake != "no wait for V":
                        yield t_full["v"][i + k & 1], i + k >> 1
                    expect(wide["v"][i + k & 1] == [i + k] * 4, "another block's nodes of V")
                    yield 2
                expect(pv_ended[slot] >= n - 2, "P written while a product reads it")
                P[slot][n & 1][me] = n
                p_full[slot][n & 1].arrive(s)
                n += 1
            done[slot] = n - 1
            yield seg_full[(run + 1) % SEGS], (run + 1) // SEGS
            at_seg(run + 1)
            if nb > k0:
                yield pv_done[slot][n - 1 & 1], n - 1 >> 1
            yield from meet(meet_all)
            yield from meet(meet_group[slot][g])
            if not dual:
                yield from meet(meet_all)
            yield from meet(meet_group[slot][g]) if dual else meet(meet_all)
            at_seg(run)
            seg_empty[run % SEGS].arrive(s)
            for t in (slot,) if dual else (0, 1):
                expect(pv_ended[t] == done[t] == pv_started[t], "O read before its last products")
            yield 4
            for t in (slot,) if dual else (0, 1):
                expect(pv_started[t] == done[t], "O overwritten while it is read")
            i += nb
            yield from meet(meet_all)

    s.spawn(producer())
    s.spawn(producer2())
    for g in range(conv):
        for w in range(4):
            for x in "kv":
                s.spawn(converter(x, g, w))
    for t in range(2):
        s.spawn(issuer(t))
        for g in range(groups):
            for w in range(4):
                s.spawn(softmax(t, g, w))
    s.run()


def work(seed):
    """Runs of a CTA: mostly short ones, with and without prefix or tree blocks."""
    rng = random.Random(seed)
    out = []
    for _ in range(rng.choice((1, 2, 5, 9, 14))):
        nb = rng.choice((1, 1, 1, 2, 3, 4, 9))
        out.append((nb, rng.randint(0, nb)))
    return out


@pytest.mark.parametrize("heavy", [False, True])
@pytest.mark.parametrize("rows", SHAPES)
def test_protocol(rows, heavy):
    for seed in range(120):
        kernel(seed, work(seed), rows, heavy)


@pytest.mark.parametrize("rows,kw", [
    (16, dict(mistake="an idle slot waits for q")), (64, dict(mistake="an idle slot waits for q")),
    (16, dict(mistake="an idle slot's tiles count")), (64, dict(mistake="an idle slot's tiles count")),
    (64, dict(mistake="no wait before O is rescaled")), (128, dict(mistake="no wait before O is rescaled")),
    (16, dict(mistake="no wait for V")), (128, dict(mistake="no wait for V")),
    (16, dict(mistake="V's wait alone")), (64, dict(mistake="V's wait alone")),     # (its phase before may not be over)
    (16, dict(stages=5))])      # an odd number of stages with two groups of converters: a stage belongs to neither
def test_planted_mistakes_are_found(rows, kw):
    found = 0
    for seed in range(300):
        try:
            kernel(seed, work(seed), rows, heavy=seed % 2 == 0, **kw)
        except Fault:
            found += 1
    assert found > 0


def test_the_source_does_as_the_model():
    """q of a tile is said to be there only to the slots that have a block of it, and an issuer counts those tiles."""
    src = (Path(__file__).parent.parent / "speculative_decoding_tree_parent_gb300" / "csrc" / "attn_kv4.cu").read_text()
    arrivals = re.findall(r"mbar_arrive_if\(([^;]*), bar\(bars\.q_full\[([01])\]\)\)", src)
    assert len(arrivals) == 2
    assert {slot: when for when, slot in arrivals} == {"0": "lane == 0 && nb > (i & 1)", "1": "lane == 0 && nb > ((i & 1) ^ 1)"}
    waits = re.findall(r"(.*)wait_one\(bar\(bars\.q_full\[t\]\), ([^)]*)\)", src)
    assert len(waits) == 1 and waits[0][1] == "n_q & 1"
    assert re.search(r"if \(k0 < nb\) \{[^}]*bars\.q_full\[t\]\), n_q & 1\);[^}]*\+\+n_q;", src)
