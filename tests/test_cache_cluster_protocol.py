"""A model of the cluster form of the few-row cache attention kernel
(csrc/s2_cache_dec.cu, CL), run on the CPU: a cluster of CTAs, each a producer
warp and four consumer warps over one segment of its share of an item's key tiles
(none, for some), the segment's end mark, the parts left over the query slots
that the segment does not use, the two meetings of the whole cluster with the
reads of the other CTAs' parts between them, and the copies in flight,
interleaved at random.  Any bounded wait may also be given up, by any warp: its
CTA's other waits then end without success too.  Checked: every warp reaches both
meetings (they are the kernel's only waits without a limit) and ends, nothing is
read of a CTA that has ended, no copy lands in one, and, where nothing was given
up, every part is whole when it is read, in place of no query row in use."""
import random

import pytest

from tests.test_cache_attn_protocol import Bar

WARPS, NQ = 4, 3


class _Cta:
    def __init__(self, tiles, NS):
        self.tiles, self.NS = tiles, NS
        self.bars = {("sync", 0): Bar(WARPS)}
        for s in range(NS):
            self.bars[("full", s)], self.bars[("empty", s)] = Bar(1), Bar(WARPS)
        for s in range(NQ):
            self.bars[("qfull", s)], self.bars[("qempty", s)] = Bar(1), Bar(WARPS)
        self.abort, self.ended, self.ring, self.part = False, 0, [None] * NS, set()
        self.query = [None] * NQ           # what the query slots hold
        self.sums, self.flight = {}, 0     # and copies in flight


def run(shares, seed, NS=3, give_up=0.0, second_meeting=True, meet_after_giving_up=True, drain_late=True, slow=False):
    rnd = random.Random(seed)
    ctas = [_Cta(n, NS) for n in shares]
    everyone = len(ctas) * (WARPS + 1)
    meeting = Bar(everyone)
    err, tma, gave_up = [], [], [False]

    def land_on(c, what):
        c.flight += 1

        def land():
            c.flight -= 1
            if c.ended == WARPS + 1:
                err.append("a copy lands in a CTA that has ended")
            what()
        tma.append(land)

    def producer(c):
        L = qu = 0
        ok = True
        while True:
            more = qu == 0
            qs = qu % NQ
            if more and c.tiles > 0:
                def landed(qs=qs):
                    if c.query[qs] is not None:
                        err.append("query rows over a part")
                    c.query[qs] = "q"
                    c.bars[("qfull", qs)].arrive()
                land_on(c, landed)
            else:
                c.bars[("qfull", qs)].arrive()
            yield ("pause",)
            qu += 1
            if not more:
                break
            for i in range(c.tiles):
                s, r = L % NS, L // NS
                if r > 0:
                    ok = yield ("wait", ("empty", s), r - 1)
                    if not ok:
                        break

                def landed(s=s, i=i):
                    c.ring[s] = i
                    c.bars[("full", s)].arrive()
                land_on(c, landed)
                yield ("pause",)
                L += 1
            if not ok:
                break
        if c.abort:
            for s in range(min(NQ, qu)):
                yield ("drain", ("qfull", s), (qu - 1 - s) // NQ)
            for s in range(min(NS, L)):
                yield ("drain", ("full", s), (L - 1 - s) // NS)
        yield from meet(c, ok, drains=True)

    def consumer(c, w):
        L = 0
        ok = yield ("wait", ("qfull", 0), 0)
        if ok:
            if c.tiles > 0 and c.query[0] != "q":
                err.append("query rows not there")
            for i in range(c.tiles):
                s = L % NS
                ok = yield ("wait", ("full", s), L // NS)
                if not ok:
                    break
                if c.ring[s] != i:
                    err.append(f"stage {s} holds {c.ring[s]} for {i}")
                L += 1
                if i + 1 < c.tiles:
                    yield ("arrive", ("empty", s))
        if ok:
            yield ("arrive", ("qempty", 0))
            if c.tiles > 0:
                c.sums[w] = True
                yield ("arrive", ("sync", 0))
                ok = yield ("wait", ("sync", 0), 0)
                if ok and len(c.sums) != WARPS:
                    err.append("joined before every warp left its sums")
        if ok:
            for qs in (1, 2):  # its share of the part's rows
                if c.query[qs] == "q":
                    err.append("a part over query rows")
                c.query[qs] = "part"
            c.part.add(w)
            yield ("pause",)
            if c.tiles > 0:
                yield ("arrive", ("empty", (L - 1) % NS))
            ok = yield ("wait", ("qfull", 1), 0)  # the end mark
        yield from meet(c, ok, reader=True)

    def meet(c, ok, reader=False, drains=False):
        if ok or meet_after_giving_up:
            meeting.arrive()
            yield ("meet", 0)
            if drains and drain_late and c.abort:   # nobody of the CTA gives up any more
                yield ("drain", ("qfull", 0), 0)
                for s in range(min(NS, c.tiles)):
                    yield ("drain", ("full", s), (c.tiles - 1 - s) // NS)
            if reader:
                for p in ctas:
                    yield ("pause",)
                    if p.ended:
                        err.append("read of a CTA that has ended")
                    if not gave_up[0] and len(p.part) != WARPS:
                        err.append(f"read of a part that {len(p.part)} warps have left")
            if second_meeting:
                meeting.arrive()
                yield ("meet", 1)
        c.ended += 1

    actors = {}
    for x, c in enumerate(ctas):
        actors[x, "producer"] = producer(c)
        for w in range(WARPS):
            actors[x, f"warp {w}"] = consumer(c, w)
    pending, finished = {n: None for n in actors}, set()

    def ready(n):
        op = pending[n]
        if op is None:
            return True
        if op[0] == "meet":
            return meeting.done >= op[1] + 1
        c = ctas[n[0]]
        if op[0] == "drain" and c.flight == 0:   # (its limit: a copy that was never issued)
            return True
        return c.bars[op[1]].done >= op[2] + 1 or (op[0] == "wait" and (c.abort or give_up > 0))

    while not err:
        choices = [n for n in actors if n not in finished and ready(n)]
        if tma and not (slow and choices and rnd.random() < 0.97):
            choices.append("tma")
        if not choices:
            if len(finished) == len(actors):
                return []
            return ["deadlock: " + ", ".join(f"{n} in {pending[n]}" for n in actors if n not in finished)]
        n = rnd.choice(choices)
        if n == "tma":
            tma.pop(rnd.randrange(len(tma)))()
            continue
        c, op, answer = ctas[n[0]], pending[n], None
        if op is not None and op[0] in ("wait", "drain"):
            done = c.bars[op[1]].done
            if done >= op[2] + 2:
                return [f"{n}: phase overrun on {op[1]}"]
            answer = done >= op[2] + 1
            if not answer and op[0] == "wait":
                if not c.abort:
                    if rnd.random() >= give_up:
                        continue
                    c.abort = gave_up[0] = True
        try:
            nxt = actors[n].send(answer) if op is not None else next(actors[n])
        except StopIteration:
            finished.add(n)
            continue
        if nxt[0] == "arrive":
            c.bars[nxt[1]].arrive()
            nxt = None
        elif nxt[0] == "pause":
            nxt = None
        elif nxt[0] == "wait" and c.bars[nxt[1]].done < nxt[2]:
            return [f"{n}: parity wait ahead on {nxt[1]}"]
        pending[n] = nxt
    return err[:3]


SHARES = [[0], [1], [2], [5], [1, 0], [3, 3, 2], [4, 4, 4, 0], [1] * 8, [2] * 7 + [0], [7, 7, 3, 0, 0], [1] * 5 + [0] * 11, [5] * 16]


@pytest.mark.parametrize("NS", [3, 6])
def test_cluster_protocol_runs_clean(NS):
    for shares in SHARES:
        for seed in range(12):
            problems = run(shares, seed, NS)
            assert not problems, (problems, shares, seed)


def test_every_warp_that_gives_up_reaches_both_meetings():
    for shares in SHARES:
        for seed in range(40):
            problems = run(shares, seed, give_up=0.02 if seed % 2 else 0.3, slow=seed % 3 == 0)
            assert not problems, (problems, shares, seed)


def test_model_finds_a_missing_second_meeting():
    assert any(run([2, 2, 1], seed, second_meeting=False) for seed in range(20))


def test_model_finds_a_warp_that_leaves_without_the_meetings():
    assert any(run([3, 3, 2], seed, give_up=0.3, meet_after_giving_up=False) for seed in range(20))


def test_model_finds_copies_left_in_flight():
    """A producer that asks only before the meeting whether a consumer has given up: one may do so later."""
    assert any(run([3, 2], seed, give_up=0.3, drain_late=False, slow=True) for seed in range(100))
