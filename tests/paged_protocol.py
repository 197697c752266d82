"""An event model of the barriers of csrc/paged_attention.cu: every warp of a CTA, mbarriers with the hardware's parity waits,
bulk copies and products that end later, in an order and after delays that a seed draws.  Every buffer carries the number of the
token tile (or row tile) that it holds, which whoever reads it checks.

A warp here does what the kernel's warp of the same part does, wait for wait and arrival for arrival; where the model knows
a rule by which the kernel may go or not (source_rules), it goes by the source."""
import heapq
import os
import random

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIMIT = 1e6  # a bounded wait gives up after that long; everything else takes about one


def source_rules():
    with open(os.path.join(ROOT, "gemm_rocmfp4_dequant_gb300", "csrc", "paged_attention.cu")) as f:
        s = " ".join(f.read().split())
    return {"queries_by_need": "if (more) wait.warp(&ctl.q_full" in s,
            "stand_in": "bar.sync" not in s and "while (!chains_meet(true)) { }" in s,
            "end_together": "if (__syncthreads_or(!wait.ok)) {" in s}


class Bar:
    def __init__(self, sim, count):
        self.sim, self.count, self.pending, self.phase, self.tx, self.waiters = sim, count, count, 0, 0, []

    def arrive(self, tx=0):
        self.tx += tx
        self.pending -= 1
        assert self.pending >= 0, "more arrivals than the barrier counts"
        self._check()

    def land(self, tx):
        self.tx -= tx
        self._check()

    def _check(self):
        if self.pending == 0 and self.tx == 0:
            self.phase += 1
            self.pending = self.count
            waiting, self.waiters = self.waiters, []
            for w in waiting:
                if self.done(w[1]):
                    self.sim.after(0.05 * self.sim.r.random(), lambda w=w: self.sim.woken(w, True))
                else:
                    self.waiters.append(w)

    def done(self, parity):  # of the phases of that parity the last one to begin has completed
        return (self.phase & 1) != parity


class Warp:
    ok = True  # no wait has given up

    def __init__(self, name, slow):
        self.name, self.slow = name, slow


class Sim:
    def __init__(self, seed):
        self.r, self.events, self.now, self.n, self.live, self.flying, self.end = random.Random(seed), [], 0.0, 0, 0, 0, None
        self.pause = None  # (name of a warp, after how many of its steps)

    def after(self, d, f):
        self.n += 1
        heapq.heappush(self.events, (self.now + d, self.n, f))

    def flight(self, d, f):
        """Something asynchronous that ends by f."""
        self.flying += 1

        def landed():
            self.flying -= 1
            f()
        self.after(d, landed)

    def spawn(self, w, body):
        self.live += 1
        w.steps, w.body = 0, body
        self.after(self.r.random(), lambda: self.step(w))

    def woken(self, entry, result):
        w, _, token = entry
        if w.token is token:
            w.token = None
            self.step(w, result)

    def wait(self, w, bar, parity, limited):
        if bar.done(parity):
            self.after(0.01, lambda: self.step(w, True))
        elif not w.ok and not limited:
            self.after(0.01, lambda: self.step(w, False))
        else:
            w.token = token = object()
            bar.waiters.append((w, parity, token))

            def late():
                if w.token is token:
                    if not limited:
                        w.ok = False
                    bar.waiters = [x for x in bar.waiters if x[2] is not token]
                    self.woken((w, parity, token), False)
            self.after(LIMIT, late)

    def step(self, w, result=None):
        w.steps += 1
        if self.pause and self.pause[0] == w.name and w.steps == self.pause[1]:
            self.pause = None
            self.after(1.5 * LIMIT, lambda: self.step(w, result))
            return
        if w.slow and self.r.random() < w.slow and not getattr(w, "rested", False):
            w.rested = True  # a warp that is not scheduled for a long while
            self.after(self.r.choice((3, 30, 300)) * self.r.random(), lambda: self.step(w, result))
            return
        w.rested = False
        try:
            op = w.body.send(result)
        except StopIteration:
            self.live -= 1
            if not self.live:
                self.end = self.flying
            return
        if op[0] == "wait":
            self.wait(w, op[1], op[2], False)
        elif op[0] == "drain":
            self.wait(w, op[1], op[2], True)
        elif op[0] == "sleep":
            self.after(op[1] * self.r.choice((.1, .5, 1, 1, 2, 20)) * self.r.random(), lambda: self.step(w))
        else:  # a barrier of the block's, without a limit: whether all said yes
            meeting = op[1]
            meeting.append((w, op[3]))
            if len(meeting) == op[2]:
                there, every = [x for x, _ in meeting], all(yes for _, yes in meeting)
                meeting.clear()
                for x in there:
                    self.after(0.01, lambda x=x: self.step(x, every))

    def run(self):
        while self.events:
            self.now, _, f = heapq.heappop(self.events)
            f()


def run(seed, stages, items, rules, slow=None, pause=None, late_copy=None):
    """One CTA over `items`, (wide, token tiles, whole) each, with a raw ring of `stages`.  slow: the name of a warp that often
    rests; pause: a warp that once stops for longer than a wait lasts; late_copy: the number of the copy that lands that late.
    Returns the warps and how much was in flight when the last of them ended (None: some never did)."""
    sim = Sim(seed)
    r = sim.r
    sim.pause = pause
    clean = pause is None and late_copy is None  # then every buffer is checked
    bars = lambda n, count: [Bar(sim, count) for _ in range(n)]  # noqa: E731
    full, empty = [bars(2, 4), bars(2, 4)], [bars(2, 2), bars(2, 2)]  # of K, of V
    s_full, o_full, turn, drained = (bars(2, 1) for _ in range(4))
    p_full, q_full = bars(2, 4), bars(2, 4)
    raw_full, raw_empty = bars(stages, 1), bars(stages, 4)
    item_full, item_empty = bars(4, 1), bars(4, 10)
    slot, tiles, raw = [(None, 0)] * 4, [(None, True)] * 16, [None] * stages
    kv = [[[None] * 4 for _ in range(2)] for _ in range(2)]
    S, P, Q, q_by = [None] * 2, [[None] * 4, [None] * 4], [None] * 2, [[None] * 4, [None] * 4]
    meeting, ending, pipe, copies = [], [], [0.0, 0.0], [0]
    warps = []

    def warp(name):
        w = Warp(name, 0.3 if slow == name else 0.0)
        warps.append(w)
        return w

    def check(ok, *what):
        assert ok or not clean or not all(w.ok for w in warps), what

    def product(t, dur, f):  # a chain's run in order
        pipe[t] = max(pipe[t], sim.now) + dur * r.choice((.2, 1, 1, 4)) * r.random()
        sim.flight(pipe[t] - sim.now, f)

    def leave(w, left=(), start=lambda: None):
        """The end of the block: what may be on its way is waited for where some warp gave up (by the former rule, only by those
        who had)."""
        late = not w.ok
        if rules["end_together"]:
            late = not (yield "meet", ending, len(NAMES), w.ok)
        if late:
            start()
            for bar, parity in left:
                yield "drain", bar, parity

    def loader(w):
        n = tile = issued = stopped = 0
        more = True
        while more and w.ok:
            it = items[n] if n < len(items) else None
            more = it is not None
            yield "wait", item_empty[n % 4], (n // 4 & 1) ^ 1
            if not w.ok:
                break
            slot[n % 4] = (it, tile)
            item_full[n % 4].arrive()
            if more:
                for _ in range(it[1]):
                    for which in range(2):
                        yield "sleep", .5
                        st = issued % stages
                        yield "wait", raw_empty[st], (issued // stages & 1) ^ 1
                        if not w.ok:
                            break
                        if which == 0:
                            tiles[tile % 16] = (tile, False)
                        if r.random() < .1:  # nothing to copy
                            raw[st] = (tile, which)
                            raw_full[st].arrive()
                        else:
                            parts = r.randint(1, 8)
                            raw_full[st].arrive(parts)
                            raw[st] = None
                            for c in range(parts):
                                def landed(c=c, st=st, x=(tile, which)):
                                    if c == 0:
                                        raw[st] = x
                                    raw_full[st].land(1)
                                copies[0] += 1
                                sim.flight(1.3 * LIMIT if copies[0] == late_copy else r.random() * 5 * r.choice((1, 1, 10)), landed)
                        issued += 1
                    if not w.ok:
                        break
                    tile += 1
            else:
                st = issued % stages
                yield "wait", raw_empty[st], (issued // stages & 1) ^ 1
                if w.ok:
                    tiles[tile % 16] = (tile, True)
                    raw_full[st].arrive()
                    stopped = 1
            n += 1
        left = [(raw_full[i % stages], i // stages & 1) for i in range(max(issued + stopped - stages, 0), issued)]
        yield from leave(w, left)

    def decode(w, part):
        yield from decode_all(w, part)
        yield from leave(w)

    def decode_all(w, part):
        n = used = 0
        while True:
            for which in range(2):
                st = used % stages
                yield "wait", raw_full[st], used // stages & 1
                if not w.ok:
                    return
                if which == 0:
                    check(tiles[n % 16][0] == n, "description", tiles[n % 16], n)
                    if tiles[n % 16][1]:
                        return
                check(raw[st] == (n, which), "raw rows", raw[st], n, which)
                yield "wait", empty[which][n % 2], (n // 2 & 1) ^ 1
                if not w.ok:
                    return
                yield "sleep", .7
                check(raw[st] == (n, which), "raw rows", raw[st], n, which)
                kv[which][n % 2][part] = n
                raw_empty[st].arrive()
                full[which][n % 2].arrive()
                used += 1
            n += 1

    def issue(w, t):
        n = n_q0 = n_q1 = n_p = n_turn = 0
        place = [0, 0]  # K's and V's ring
        while True:
            yield "wait", item_full[n % 4], n // 4 & 1
            if not w.ok or slot[n % 4][0] is None:
                break
            (wide, count, _), tile = slot[n % 4]
            item_empty[n % 4].arrive()
            n += 1
            j = [0, 0]

            def own(kind):
                while j[kind] < count:
                    st = place[kind] % 2
                    yield "wait", full[kind][st], place[kind] // 2 & 1
                    check(kv[kind][st] == [tile + j[kind]] * 4, "decoded rows", kind, kv[kind][st], tile + j[kind])
                    if wide or (j[kind] & 1) == t:
                        return True
                    empty[kind][st].arrive()
                    j[kind] += 1
                    place[kind] += 1
                return False

            def scores():
                st, number, item = place[0] % 2, tile + j[0], n

                def ended():
                    check(kv[0][st] == [number] * 4, "K", kv[0][st], number)
                    check(Q[t if wide else 0] == item, "queries", Q, item, t)
                    S[t] = number
                product(t, .6, ended)
                product(t, 0, s_full[t].arrive)
                product(t, 0, empty[0][st].arrive)
                j[0] += 1
                place[0] += 1
            have = False
            while True:
                if have:
                    yield from own(1)
                more = yield from own(0)
                if not have:
                    half = t if wide else 0
                    if more or not rules["queries_by_need"]:
                        yield "wait", q_full[half], (n_q1 if half else n_q0) & 1
                    n_q0 += 1
                    n_q1 += bool(wide)
                else:
                    yield "wait", turn[t], (n_turn & 1) ^ (t ^ 1)
                    n_turn += 1
                    yield "wait", p_full[t], n_p & 1
                    n_p += 1
                    st, number = place[1] % 2, tile + j[1]

                    def ended(st=st, number=number):
                        check(kv[1][st] == [number] * 4, "V", kv[1][st], number)
                        check(P[t] == [number] * 4, "P", P[t], number)
                    product(t, .6, ended)
                    product(t, 0, empty[1][st].arrive)
                    if not more:
                        product(t, 0, o_full[t].arrive)
                    j[1] += 1
                    place[1] += 1
                if more:
                    scores()
                if have:
                    turn[t ^ 1].arrive()
                if not more:
                    break
                have = True
            if t == 1 and not wide and count & 1:
                yield "wait", turn[1], n_turn & 1
                n_turn += 1
                turn[0].arrive()
            yield from own(1)
        yield from leave(w, [(drained[t], 0)], lambda: product(t, 0, drained[t].arrive))

    def softmax(w, t, part):
        n = n_s = n_o = 0

        def bring(it, number):
            if t == 1 and not it[0]:
                return
            Q[t] = None
            yield "sleep", 1
            q_by[t][part] = number
            if all(x == number for x in q_by[t]):
                Q[t] = number
            q_full[t].arrive()

        def get(i):
            yield "wait", item_full[i % 4], i // 4 & 1
            return slot[i % 4] if w.ok and slot[i % 4][0] is not None else None

        def meet():
            yield "meet", meeting, 8, False
        at = yield from get(0)
        if at:
            yield from bring(at[0], 1)
        while at:
            (wide, count, whole), tile = at
            first = True
            for k in range(0 if wide else t, count, 1 if wide else 2):
                yield "wait", s_full[t], n_s & 1
                n_s += 1
                check(S[t] == tile + k, "scores", S[t], tile + k)
                check(tiles[(tile + k) % 16][0] == tile + k, "description")
                yield "sleep", 1.5
                check(S[t] == tile + k, "scores", S[t], tile + k)
                P[t][part] = tile + k
                p_full[t].arrive()
                first = False
            nx = yield from get(n + 1)
            if nx and wide:
                yield from bring(nx[0], n + 2)
            if not first:
                yield "wait", o_full[t], n_o & 1
                n_o += 1
            yield "sleep", 1.0
            if not (wide and whole):
                yield from meet()
                if not whole:
                    yield from meet()
                yield "sleep", .5
                yield from meet()
                if nx and not wide:
                    yield from bring(nx[0], n + 2)
            item_empty[n % 4].arrive()
            n += 1
            at = nx
        while rules["stand_in"] and not (yield "meet", meeting, 8, True):
            pass
        yield from leave(w)
    w = warp("loader")
    sim.spawn(w, loader(w))
    for t in range(2):
        w = warp(f"issue {t}")
        sim.spawn(w, issue(w, t))
    for part in range(4):
        w = warp(f"decode {part}")
        sim.spawn(w, decode(w, part))
        for t in range(2):
            w = warp(f"softmax {t}.{part}")
            sim.spawn(w, softmax(w, t, part))
    sim.run()
    return warps, sim.end


NAMES = ["loader", "issue 0", "issue 1"] + [f"decode {i}" for i in range(4)] + [f"softmax {t}.{i}" for t in range(2) for i in range(4)]
