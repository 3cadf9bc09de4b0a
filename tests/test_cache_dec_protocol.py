"""A model of the few-row cache attention kernel's synchronisation
(csrc/s2_cache_dec.cu), run on the CPU: the TMA producer with its three-slot ring of
segment descriptions and query rows and its ring of K/V stages, the four consumer
warps, their join through the last stage's memory (each over its own keys' rows,
one meeting, then all read all) with the row statistics in buffers used by turns,
and the copies in flight, interleaved at random with the kernel's
arrival counts and phases.  It checks that every program finishes, that no parity
wait is ahead of or overrun by its barrier, that every warp reads the stage and
the segment it means, that the join reads what it means and no statistics are
overwritten in use, and that no stage is refilled in use.  A
segment is its number of stages; 0: nothing visible."""
import random

import pytest

from tests.test_cache_attn_protocol import Bar

WARPS, NQ = 4, 3


def run(segs, seed, NS=3, release_early=False, by_segment=False):
    rnd = random.Random(seed)
    bars = {("sync", 0): Bar(WARPS)}
    for s in range(NS):
        bars[("full", s)], bars[("empty", s)] = Bar(1), Bar(WARPS)
    for s in range(NQ):
        bars[("qfull", s)], bars[("qempty", s)] = Bar(1), Bar(WARPS)
    err, tma = [], []
    ring, users = [None] * NS, [0] * NS       # stage contents, warps that still need them
    slot, susers = [None] * NQ, [0] * NQ      # segment slots
    sums, stats = {}, {}                      # what the warps left in a stage, and in the statistics' buffers
    reading = [None] * WARPS                  # the statistics a warp reads

    def producer():
        L = qu = 0
        for k, n in enumerate([*segs, -1]):
            qs = qu % NQ
            if qu >= NQ:
                yield ("wait", ("qempty", qs), qu // NQ - 1)
            if susers[qs]:
                err.append("segment slot overwritten")
            slot[qs], susers[qs] = ("in flight" if n > 0 else k), WARPS

            def land(qs=qs, k=k):
                slot[qs] = k
                bars[("qfull", qs)].arrive()
            tma.append(land) if n > 0 else land()
            yield ("pause",)
            qu += 1
            for i in range(max(n, 0)):
                s, r = L % NS, L // NS
                if r > 0:
                    yield ("wait", ("empty", s), r - 1)
                if users[s]:
                    err.append(f"stage {s} refilled while {users[s]} warps need it")
                ring[s], users[s] = "in flight", WARPS

                def land(s=s, tile=(k, i)):
                    ring[s] = tile
                    bars[("full", s)].arrive()
                tma.append(land)
                L += 1

    def consumer(w):
        L = nsync = 0
        for qu, n in enumerate([*segs, -1]):
            qs = qu % NQ
            yield ("wait", ("qfull", qs), qu // NQ)
            if slot[qs] != qu:
                err.append(f"warp {w} reads segment {slot[qs]} for {qu}")
            if n < 0:
                return
            last = None
            for i in range(n):
                s = L % NS
                yield ("wait", ("full", s), L // NS)
                if ring[s] != (qu, i):
                    err.append(f"warp {w} reads {ring[s]} for {(qu, i)}")
                L += 1
                if i + 1 < n:
                    users[s] -= 1
                    yield ("arrive", ("empty", s))
                    continue
                last = s
                if release_early:
                    yield ("arrive", ("empty", s))
                yield ("pause",)
            susers[qs] -= 1
            yield ("arrive", ("qempty", qs))
            if last is None:
                continue
            buf = qu & 1 if by_segment else nsync & 1
            if any(x == buf for x in reading):
                err.append(f"statistics of segment {qu} written over those in use")
            sums[last, w], stats[buf, w] = qu, qu
            yield ("arrive", ("sync", 0))
            yield ("wait", ("sync", 0), nsync)
            nsync += 1
            reading[w] = buf
            yield ("pause",)
            if ring[last] != (qu, n - 1) or any((sums[last, x], stats[buf, x]) != (qu, qu) for x in range(WARPS)):
                err.append(f"warp {w} joins {sums} {stats} in {ring[last]}")
            reading[w] = None
            users[last] -= 1
            if not release_early:
                yield ("arrive", ("empty", last))

    actors = {"producer": producer(), **{f"warp {w}": consumer(w) for w in range(WARPS)}}
    pending, finished = {n: None for n in actors}, set()
    while not err:
        runnable = [n for n in actors if n not in finished and
                    (pending[n] is None or bars[pending[n][1]].done >= pending[n][2] + 1)]
        choices = runnable + (["tma"] if tma else [])
        if not choices:
            if len(finished) == len(actors):
                return []
            return ["deadlock: " + ", ".join(f"{n} waits {pending[n]}" for n in actors if n not in finished)]
        c = rnd.choice(choices)
        if c == "tma":
            tma.pop(rnd.randrange(len(tma)))()
            continue
        while True:
            try:
                op = next(actors[c])
            except StopIteration:
                finished.add(c)
                pending[c] = None
                break
            if op[0] == "pause":
                pending[c] = None
                break
            if op[0] == "arrive":
                bars[op[1]].arrive()
                pending[c] = None
                break
            done = bars[op[1]].done
            if done < op[2]:
                return [f"{c}: parity wait ahead on {op[1]} (waits phase {op[2]}, {done} complete)"]
            if done >= op[2] + 2:
                return [f"{c}: phase overrun on {op[1]}"]
            if done >= op[2] + 1:
                continue
            pending[c] = op
            break
    return err[:3]


def sequences():
    out = [[n] for n in range(8)] + [[1] * 7, [2, 1] * 4, [0, 3, 0, 0, 1], [5, 0, 4]]
    rnd = random.Random(11)
    return out + [[rnd.choice([0, 1, 1, 2, 3, 6, 9]) for _ in range(rnd.randint(2, 8))] for _ in range(60)]


@pytest.mark.parametrize("NS", [3, 6])
def test_few_row_protocol_runs_clean(NS):
    for segs in sequences():
        for seed in range(8):
            problems = run(segs, seed, NS)
            assert not problems, (problems, segs, seed)


def test_model_finds_a_stage_released_before_the_join():
    """Releasing the last stage before the join that uses its memory: the check is not vacuous."""
    assert any(run([4, 5, 3], seed, release_early=True) for seed in range(40))


def test_model_finds_statistics_buffers_that_do_not_alternate():
    """Buffers chosen by the segment's number: one without a stage between two others breaks the turns."""
    assert any(run([2, 0, 1, 0, 1], seed, 6, by_segment=True) for seed in range(200))
