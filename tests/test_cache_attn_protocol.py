"""A model of the cache attention kernel's synchronisation (csrc/s2_cache_tc.cu),
run on the CPU: the TMA producer, the UMMA issuer, the two softmax warpgroups
(four warps each, one of them possibly without a live row, all modelled apart)
with their epilogues, the tensor pipe and the copies in flight, as programs of
mbarrier waits and arrivals with the kernel's counts and phases, interleaved at
random.  It checks that every program finishes, that no parity wait is ahead of
or overrun by its barrier, that every UMMA reads the tile it means, that rows of
V are zeroed in the tile they belong to before the product reads them, and that
nothing is overwritten while a reader needs it.  A segment is (tiles, paired,
ragged): paired feeds both query tiles from every key tile, otherwise the
warpgroups alternate over the key tiles of one query tile; ragged: the last key
tile ends inside a 16-key step; 0 tiles: nothing visible."""
import random

import pytest


class Bar:
    def __init__(self, count):
        self.count, self.rem, self.done = count, count, 0

    def arrive(self, n=1):
        for _ in range(n):
            self.rem -= 1
            if self.rem == 0:
                self.done += 1
                self.rem = self.count


NG = 4  # segment descriptions


def run(segs, seed, NQ=2, NS=5, early_zero=False):
    rnd = random.Random(seed)
    bars = {}
    for s in range(NQ):
        bars[("qfull", s)], bars[("qempty", s)] = Bar(1), Bar(1)
    for s in range(NS):
        bars[("full", s)], bars[("empty", s)] = Bar(1), Bar(1)
    for w in (0, 1):
        for name, cnt in (("s", 1), ("plo", 4), ("p", 4), ("o", 1), ("ofree", 4)):
            bars[(name, w)] = Bar(cnt)
    bars[("mb", 0)] = Bar(4)
    for s in range(NG):
        bars[("gfull", s)], bars[("gempty", s)] = Bar(1), Bar(9)
    descr, users = [None] * NG, [0] * NG     # segment descriptions, and who still needs them
    err, tma, pipe = [], [], []
    qslot, qreads, ring, ringreads = [None] * NQ, [0] * NQ, [None] * NS, [0] * NS
    sbuf = [[None] * 4, [None] * 4]          # per warp quarter: what its lanes of S/P hold
    zeroed, pv_done, o_read, stats = set(), set(), set(), [None] * 4

    def shape(k):
        n, paired, ragged = segs[k]
        return (n, n, n) if paired else (n, (n + 1) // 2, n // 2)

    def key_tile(k, w, j):
        return j if segs[k][1] else 2 * j + w

    def take(k):
        yield ("wait", ("gfull", k % NG), k // NG)
        if descr[k % NG] != k:
            err.append(f"segment {descr[k % NG]} for {k}")

    def give(k):
        users[k % NG] -= 1
        return ("arrive", ("gempty", k % NG), 1)

    def producer():
        qu = L = 0
        for k, (n, paired, _) in enumerate(segs):
            if k >= NG:
                yield ("wait", ("gempty", k % NG), k // NG - 1)
            if users[k % NG]:
                err.append("segment description overwritten")
            descr[k % NG], users[k % NG] = k, 9
            yield ("arrive", ("gfull", k % NG), 1)
            if n == 0:
                continue
            _, nA, nB = shape(k)
            for w in range(2 if paired else 1):
                s, r = qu % NQ, qu // NQ
                if r > 0:
                    yield ("wait", ("qempty", s), r - 1)
                if qreads[s]:
                    err.append("Q slot reloaded with reads pending")
                qslot[s], qreads[s] = "in flight", ((nA, nB)[w] if paired else nA + nB)

                def land(s=s, tile=(k, w)):
                    qslot[s] = tile
                    bars[("qfull", s)].arrive()
                tma.append(land)
                qu += 1
            for t in range(n):
                for kind in "KV":
                    s, r = L % NS, L // NS
                    if r > 0:
                        yield ("wait", ("empty", s), r - 1)
                    if ringreads[s]:
                        err.append("K/V slot reloaded with reads pending")
                    ring[s], ringreads[s] = "in flight", (2 if paired else 1)

                    def land(s=s, tile=(k, kind, t)):
                        ring[s] = tile
                        bars[("full", s)].arrive()
                    tma.append(land)
                    L += 1

    def issuer():
        L = qu = 0
        np_, nseg = [0, 0], [0, 0]

        def full(Lx):
            return ("wait", ("full", Lx % NS), Lx // NS)

        for k, (n, paired, _) in enumerate(segs):
            yield from take(k)
            yield give(k)
            if n == 0:
                continue
            alt = not paired
            _, nA, nB = shape(k)
            qa, qb, L0 = qu % NQ, (qu if alt else qu + 1) % NQ, L

            def lk(w, j):
                return L0 + (4 * j + 2 * w if alt else 2 * j)

            def issue_s(w, j):
                pipe.append(("S", w, k, j, qb if w else qa, lk(w, j) % NS))
                pipe.append(("commit", ("s", w)))

            def release(Lx):
                pipe.append(("commit", ("empty", Lx % NS)))

            def pv(w, j):
                Lv = lk(w, j) + 1
                yield ("wait", ("plo", w), np_[w])
                if j == 0 and nseg[w] > 0:
                    yield ("wait", ("ofree", w), nseg[w] - 1)
                yield full(Lv)
                pipe.append(("PVlo", w, k, j, Lv % NS))
                yield ("wait", ("p", w), np_[w])
                pipe.append(("PVhi", w, k, j, Lv % NS))
                pipe.append(("commit", ("o", w)))
                np_[w] += 1

            yield ("wait", ("qfull", qa), qu // NQ)
            if paired:
                yield ("wait", ("qfull", qb), (qu + 1) // NQ)
            yield full(lk(0, 0))
            issue_s(0, 0)
            if alt:
                release(lk(0, 0))
            if nB > 0:
                if alt:
                    yield full(lk(1, 0))
                issue_s(1, 0)
                release(lk(1, 0))
            for j in range(nA):
                yield from pv(0, j)
                if alt:
                    release(lk(0, j) + 1)
                if j + 1 < nA:
                    yield full(lk(0, j + 1))
                    issue_s(0, j + 1)
                    if alt:
                        release(lk(0, j + 1))
                if j < nB:
                    yield from pv(1, j)
                    release(lk(1, j) + 1)
                    if j + 1 < nB:
                        if alt:
                            yield full(lk(1, j + 1))
                        issue_s(1, j + 1)
                        release(lk(1, j + 1))
            pipe.append(("commit", ("qempty", qa)))
            if paired:
                pipe.append(("commit", ("qempty", qb)))
            qu += 1 if alt else 2
            L = L0 + 2 * n
            nseg[0] += 1
            nseg[1] += nB > 0

    def softmax(w, quarter):
        ns = L = nmb = 0
        no = [0, 0]
        for k, (n, paired, ragged) in enumerate(segs):
            yield from take(k)
            alt = not paired
            _, nA, nB = shape(k)
            steps, L0 = (nA, nB)[w], L
            L += 2 * n
            busy = quarter == 0 or (k + quarter) % 3 > 0
            for j in range(steps):
                t = key_tile(k, w, j)
                zero = ragged and t == n - 1 and (alt or w == 0)
                Lv = L0 + (4 * j + 2 * w if alt else 2 * j) + 1

                def fill():
                    yield ("wait", ("full", Lv % NS), Lv // NS)
                    if ring[Lv % NS] != (k, "V", t):
                        err.append(f"zeroes rows of {ring[Lv % NS]} for V({k},{t})")
                    zeroed.add((k, t, quarter))
                if zero and early_zero:
                    yield from fill()
                yield ("wait", ("s", w), ns)
                ns += 1
                if zero and not early_zero:
                    yield from fill()
                if sbuf[w][quarter] != ("S", k, j):
                    err.append(f"softmax {w}.{quarter} reads {sbuf[w][quarter]} for S({k},{j})")
                if busy and j > 0 and rnd.random() < 0.3:
                    yield ("wait", ("o", w), no[w] - 1)
                sbuf[w][quarter] = ("Plo", k, j)
                yield ("arrive", ("plo", w), 1)
                sbuf[w][quarter] = ("P", k, j)
                yield ("arrive", ("p", w), 1)
                no[w] += 1
            if w == 0:
                no[1] += nB
            if steps > 0:
                yield ("wait", ("o", w), no[w] - 1)
                if any((w, k, j) not in pv_done for j in range(steps)):
                    err.append("epilogue before its P V")
            if alt and w == 1:
                if steps > 0:
                    if stats[quarter] is not None:
                        err.append("row statistics overwritten")
                    stats[quarter] = k
                    yield ("arrive", ("mb", 0), 1)
            elif alt and nB > 0:
                yield ("wait", ("mb", 0), nmb)
                yield ("wait", ("o", 1), no[1] - 1)
                nmb += 1
                if stats[quarter] != k or any((1, k, j) not in pv_done for j in range(nB)):
                    err.append("join before warpgroup B is done")
                stats[quarter] = None
                o_read.update({(0, k, quarter), (1, k, quarter)})
                yield ("arrive", ("ofree", 0), 1)
                yield ("arrive", ("ofree", 1), 1)
            elif steps > 0:
                o_read.add((w, k, quarter))
                yield ("arrive", ("ofree", w), 1)
            if descr[k % NG] != k:
                err.append("segment description replaced in use")
            yield give(k)

    def execute():
        op = pipe.pop(0)
        if op[0] == "commit":
            bars[op[1]].arrive()
            return
        kind, w, k, j = op[:4]
        t = key_tile(k, w, j)
        if kind == "S":
            qs, ks = op[4], op[5]
            if qslot[qs] != (k, w if segs[k][1] else 0) or ring[ks] != (k, "K", t):
                err.append(f"S{w}({k},{j}) reads Q {qslot[qs]} K {ring[ks]}")
            for x in sbuf[w]:
                if x is not None and (x[0] != "P" or (w, x[1], x[2]) not in pv_done):
                    err.append(f"S{w}({k},{j}) overwrites {x}")
            qreads[qs] -= 1
            ringreads[ks] -= 1
            sbuf[w][:] = [("S", k, j)] * 4
            return
        if ring[op[4]] != (k, "V", t):
            err.append(f"{kind}{w}({k},{j}) reads V {ring[op[4]]}")
        if segs[k][2] and t == segs[k][0] - 1 and any((k, t, x) not in zeroed for x in range(4)):
            err.append(f"{kind}{w}({k},{j}) reads rows behind the last key")
        want = ("Plo", "P") if kind == "PVlo" else ("P",)
        if any(x is None or x[0] not in want or x[1:] != (k, j) for x in sbuf[w]):
            err.append(f"{kind}{w}({k},{j}) reads {sbuf[w]}")
        if kind == "PVlo":
            prev = [kk for kk in range(k) if shape(kk)[1 + w] > 0]
            if j == 0 and prev and any((w, prev[-1], x) not in o_read for x in range(4)):
                err.append(f"PV{w}({k},0) overwrites O of segment {prev[-1]}")
        else:
            ringreads[op[4]] -= 1
            pv_done.add((w, k, j))

    actors = {"producer": producer(), "issuer": issuer()}
    actors.update({f"softmax {w}.{x}": softmax(w, x) for w in (0, 1) for x in range(4)})
    pending, finished = {n: None for n in actors}, set()
    while not err:
        runnable = [n for n in actors if n not in finished and
                    (pending[n] is None or bars[pending[n][1]].done >= pending[n][2] + 1)]
        choices = runnable + (["pipe"] if pipe else []) + (["tma"] if tma else [])
        if not choices:
            if len(finished) == len(actors):
                return []
            return ["deadlock: " + ", ".join(f"{n} waits {pending[n]}" for n in actors if n not in finished)]
        c = rnd.choice(choices)
        if c == "pipe":
            execute()
            continue
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
            if op[0] == "arrive":
                bars[op[1]].arrive(op[2])
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
    out = [[(n, p, r)] for n in range(1, 8) for p in (False, True) for r in (False, True)]
    out += [[(1, False, True)] * 6, [(1, True, True)] * 6, [(2, False, True), (1, True, False)] * 3, [(0, False, False), (3, False, True)],
            [(1, False, True), (0, True, False), (2, True, True), (0, False, False), (1, False, False)]]
    rnd = random.Random(5)
    for _ in range(60):
        out.append([(rnd.choice([0, 1, 1, 2, 3, 4, 5, 9]), rnd.random() < 0.5, rnd.random() < 0.6)
                    for _ in range(rnd.randint(2, 7))])
    return out


@pytest.mark.parametrize("NQ,NS", [(2, 5), (4, 10)])
def test_cache_attention_protocol_runs_clean(NQ, NS):
    for segs in sequences():
        for seed in range(8):
            problems = run(segs, seed, NQ, NS)
            assert not problems, (problems, segs, seed)


def test_model_finds_rows_zeroed_too_early():
    """Zeroing before the wait for S mistakes the slot's earlier tile in a four-slot ring: the check is not vacuous."""
    assert any(run([(5, False, True)], seed, 3, 4, early_zero=True) for seed in range(40))
