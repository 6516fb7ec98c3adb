"""The order of the latent attention kernels' roles, as a graph of what comes before what (CPU
only; the numbers of the wide kernel's barriers are read from its source).

A wait on an mbarrier names a phase by its parity alone. So for a wait on phase k, phase
k - 1 has to be complete before the wait begins, and phase k + 1 must not complete before
the wait is over: otherwise it passes too early, or blocks until its limit. Both have to
follow from the order of events, not from how long they take."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_attention_indexer_pmqa_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def number(name, default=None):
    m = re.search(r"\b%s = (\d+)" % name, source("pmqa_latent_wide.cu"))
    return int(m.group(1)) if m else default


STAGES, AHEAD = number("kStages"), number("kAhead")
TILES = STAGES + AHEAD + number("kSpare", 0)
TURNS = number("kTurns", 2)     # barriers of "scores issued"
OUTS = number("kOuts", 2)       # of "output done"
PIECES_KEPT = number("kPieces")


class Order:
    """Events with the events before them; a thread's events follow one another."""

    def __init__(self):
        self.before, self.thread, self.names = [], {}, {}
        self.arrivals, self.waits = {}, []

    def event(self, who, name=None, after=()):
        e = len(self.before)
        self.before.append(set(after))
        if who is not None:
            if who in self.thread:
                self.before[e].add(self.thread[who])
            self.thread[who] = e
        if name is not None:
            self.names.setdefault(name, []).append(e)
        return e

    def arrive(self, who, bar, phase, after=()):
        self.arrivals.setdefault((bar, phase), []).append(self.event(who, after=after))

    def wait(self, who, bar, phase):
        if phase >= 0:
            start = self.event(who)
            self.waits.append((who, bar, phase, start, self.event(who)))

    def close(self, counts):
        """Adds what waits depend on; returns each event's set of all events before it, as the
        bits of a number."""
        done = {}
        for (bar, phase), events in self.arrivals.items():
            assert len(events) == counts[bar[0]], (bar, phase, len(events))
            done[bar, phase] = self.event(None, after=events)
        for (bar, phase), e in done.items():
            if (bar, phase - 1) in done:
                self.before[e].add(done[bar, phase - 1])
        for _, bar, phase, _, end in self.waits:
            self.before[end].add(done[bar, phase])
        n = len(self.before)
        left = [len(b) for b in self.before]
        after = [[] for _ in range(n)]
        for e, b in enumerate(self.before):
            for x in b:
                after[x].append(e)
        ready, all_before, count = [e for e in range(n) if not left[e]], [0] * n, 0
        while ready:
            e = ready.pop()
            count += 1
            for x in self.before[e]:
                all_before[e] |= all_before[x] | 1 << x
            for x in after[e]:
                left[x] -= 1
                if not left[x]:
                    ready.append(x)
        assert count == n, "events that wait for one another"
        return done, all_before

    def check(self, counts, only=None):
        done, past = self.close(counts)
        for who, bar, phase, start, end in self.waits:
            if only and bar[0] != only:
                continue
            if phase > 0:
                assert all(past[start] >> e & 1 for e in self.arrivals[bar, phase - 1]), \
                    (who, bar, phase, "may pass a phase early")
            if (bar, phase + 1) in done:
                assert past[done[bar, phase + 1]] >> end & 1, (who, bar, phase, "may be lapped")
        return past


COUNTS = dict(info=1, used=4, ready=4, vempty=1, sfull=1, sfree=4, pfull=4, pempty=1, m=4, qfull=8, turn=1, exit=8)


def of(name, ring, tile):
    return ((name, tile % ring), tile // ring)


def wide(pieces, moved=None):
    """The kernel's events over pieces of so many tiles. moved: (warp, tile) where a softmax warp
    found a maximum moved and waits for the output of the tile before."""
    o = Order()
    place = [(t, n) for n in pieces for t in range(n)]
    seg = -1
    for it, (t, n) in enumerate(place):
        first, last, steady = t == 0, t == n - 1, t + 2 < n
        seg += first
        # the planner
        if it >= AHEAD:
            o.wait("plan", *of("used", TILES, it - AHEAD))
        o.event("plan", ("write", it))
        if first:
            o.event("plan", ("piece", seg))
        o.arrive("plan", *of("info", TILES, it))
        # the producers
        for w in range(4):
            me = "copy", w
            o.wait(me, *of("info", TILES, it))
            o.event(me, ("read", it))
            o.event(me, ("rows", it))
            o.wait(me, *of("vempty", STAGES, it - STAGES))
            o.arrive(me, *of("used", TILES, it))
            o.arrive(None, *of("ready", STAGES, it), after=[o.event(me)])
        # the softmax: eight warps, a group takes every second tile
        for w in range(8):
            me, own = ("soft", w), it % 2 == w // 4
            o.wait(me, *of("info", TILES, it))
            o.event(me, ("read", it))
            if first:
                o.event(me, ("piece read", seg))
                o.arrive(me, ("qfull", 0), seg)
            if own:
                if not first:
                    o.wait(me, *of("m", 2, it - 1))
                o.event(me, ("read", it))
                o.wait(me, *of("sfull", 2, it))
                o.arrive(me, ("sfree", 0), it)
                o.arrive(me, *of("m", 2, it))
                o.wait(me, *of("pempty", OUTS, it - 2))
                if moved == (w, it) and not first:
                    o.wait(me, *of("pempty", OUTS, it - 1))
                o.arrive(me, *of("pfull", 2, it))
            if last:
                if it > 0:
                    o.wait(me, *of("pempty", OUTS, it - 1))
                o.wait(me, *of("pempty", OUTS, it))
                for k in range(2):
                    o.arrive(me, ("exit", 0), 2 * seg + k)
                    o.wait(me, ("exit", 0), 2 * seg + k)
                o.event(me, ("piece read", seg))
        # the scores
        o.wait("scores", *of("info", TILES, it))
        o.event("scores", ("read", it))
        o.wait("scores", *of("ready", STAGES, it))
        if first:
            o.wait("scores", ("qfull", 0), seg)
        o.wait("scores", ("sfree", 0), it - 1)
        o.arrive("scores", *of("turn", TURNS, it))  # before the last of the products
        issued = o.event("scores")
        o.arrive(None, *of("sfull", 2, it), after=[issued])
        # the output
        o.wait("out", *of("info", TILES, it))
        o.event("out", ("read", it))
        o.wait("out", *of("pfull", 2, it))
        if steady:
            o.wait("out", *of("turn", TURNS, it + 2))
        issued = o.event("out")
        for name, ring in (("vempty", STAGES), ("pempty", OUTS)):
            o.arrive(None, *of(name, ring, it), after=[issued])
    return o


def narrow(pieces, stages, ahead, groups, moved=None):
    """The same of the kernel for up to 64 packed rows, each softmax group on every tile. Scores and
    outputs are issued by one warp in either order: here by two, which is less."""
    o = Order()
    place = [(t, n) for n in pieces for t in range(n)]
    ring, seg = stages + ahead, -1
    for it, (t, n) in enumerate(place):
        first, last = t == 0, t == n - 1
        seg += first
        if it >= ahead:
            o.wait("plan", *of("used", ring, it - ahead))
        o.event("plan", ("write", it))
        if first:
            o.event("plan", ("piece", seg))
        o.arrive("plan", *of("info", ring, it))
        for w in range(4):
            me = "copy", w
            o.wait(me, *of("info", ring, it))
            o.event(me, ("read", it))
            o.event(me, ("rows", it))
            if first:
                o.wait(me, ("qempty", 0), seg - 1)
                o.event(me, ("piece read", seg))
            o.wait(me, *of("vempty", stages, it - stages))
            o.wait(me, *of("rempty", 2, it - 2))
            o.arrive(me, *of("used", ring, it))
            o.arrive(None, *of("ready", stages, it), after=[o.event(me)])
        for w in range(4 * groups):
            me = "soft", w
            o.wait(me, *of("info", ring, it))
            o.event(me, ("read", it))
            o.wait(me, *of("sfull", 2, it))
            o.wait(me, *of("pempty", 2, it - 2))
            o.arrive(me, ("group", w // 4), it)
            o.wait(me, ("group", w // 4), it)
            o.arrive(me, *of("sfree", 2, it))
            if moved == (w, it) and not first:
                o.wait(me, *of("pempty", 2, it - 1))
            o.event(me, ("read", it))
            o.arrive(me, *of("pfull", 2, it))
            if last:
                o.wait(me, *of("pempty", 2, it))
                o.event(me, ("piece read", seg))
        o.wait("scores", *of("ready", stages, it))
        o.wait("scores", *of("info", ring, it))
        o.wait("scores", *of("sfree", 2, it - 2))
        o.event("scores", ("read", it))
        issued = o.event("scores")
        for name in ("sfull", "rempty"):
            o.arrive(None, *of(name, 2, it), after=[issued])
        if last:
            o.arrive(None, ("qempty", 0), seg, after=[issued])
        o.wait("out", *of("pfull", 2, it))
        o.event("out", ("read", it))
        issued = o.event("out", after=[issued])
        o.arrive(None, *of("vempty", stages, it), after=[issued])
        o.arrive(None, *of("pempty", 2, it), after=[issued])
    return o


PIECES = [[20], [1] * 24, [2] * 8, [3] * 6, [1, 9, 2, 7, 1, 1, 3], [5, 6, 4, 5]]


@pytest.mark.parametrize("pieces", PIECES)
def test_the_wait_for_later_scores_is_not_lapped(pieces):
    wide(pieces).check(COUNTS, "turn")


@pytest.mark.parametrize("pieces", PIECES)
def test_no_wait_but_for_outputs_is_lapped(pieces):
    for bar in COUNTS.keys() - {"pempty"}:
        wide(pieces).check(COUNTS, bar)


@pytest.mark.parametrize("pieces", PIECES)
def test_no_wait_is_lapped_where_a_maximum_moves(pieces):
    wide(pieces).check(COUNTS)
    for it in range(sum(pieces)):
        wide(pieces, (4 * (it % 2) + it // 2 % 4, it)).check(COUNTS)


@pytest.mark.parametrize("pieces", PIECES)
def test_descriptions_are_read_before_their_place_is_used_again(pieces):
    o = wide(pieces)
    _, past = o.close(COUNTS)
    for it in range(sum(pieces)):
        for name, ring in (("read", TILES), ("rows", AHEAD)):
            for written in o.names.get(("write", it + ring), []):
                assert all(past[written] >> e & 1 for e in o.names[name, it]), (name, it)


@pytest.mark.parametrize("pieces", PIECES)
def test_pieces_are_read_before_their_place_is_used_again(pieces):
    o = wide(pieces)
    _, past = o.close(COUNTS)
    for seg in range(len(pieces)):
        for written in o.names.get(("piece", seg + PIECES_KEPT), []):
            assert all(past[written] >> e & 1 for e in o.names["piece read", seg]), seg


@pytest.mark.parametrize("stages,ahead,groups,kept", [(3, 1, 1, 8), (2, 2, 2, 8)])
@pytest.mark.parametrize("pieces", PIECES)
def test_the_kernel_of_few_rows(pieces, stages, ahead, groups, kept):
    counts = dict(COUNTS, sfree=4 * groups, pfull=4 * groups, group=4, qempty=1, rempty=1)
    for it in range(sum(pieces)):
        narrow(pieces, stages, ahead, groups, (it % (4 * groups), it)).check(counts)
    o = narrow(pieces, stages, ahead, groups)
    past = o.check(counts)
    for it in range(sum(pieces)):
        for name, ring in (("read", stages + ahead), ("rows", ahead)):
            for written in o.names.get(("write", it + ring), []):
                assert all(past[written] >> e & 1 for e in o.names[name, it]), (name, it)
    for seg in range(len(pieces)):
        for written in o.names.get(("piece", seg + kept), []):
            assert all(past[written] >> e & 1 for e in o.names["piece read", seg]), seg
