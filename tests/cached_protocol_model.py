"""Model of cached_attn_kernel's barriers: the K and V producers, the two issuers, the eight softmax warps and their
asynchronous copies and products, under random timings.

Every barrier counts its phases exactly.  A wait passes, as on the device, when the parity of the phases says so; the
model raises ProtocolError when it passed a phase too early or too late, when a barrier gets more arrivals than it
expects, when a tile, a score buffer, an accumulator or an exchanged state is overwritten or read at the wrong time,
and when nothing can go on."""
import random


class ProtocolError(Exception):
    pass


def expect(ok, *what):
    if not ok:
        raise ProtocolError(what)


class Bar:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.copies, self.done = name, count, count, 0, 0

    def arrive(self, n=1):
        expect(self.pending >= n, "too many arrivals", self.name)
        self.pending -= n
        self._complete()

    def expect_copy(self):
        self.copies += 1
        self.arrive()

    def land(self):
        self.copies -= 1
        self._complete()

    def _complete(self):
        if self.pending == 0 and self.copies == 0:
            self.done += 1
            self.pending = self.count


def wait(bar, phase):
    """Until phase `phase` (0, 1, ...) of the barrier is complete; -1: the phase before the first."""
    while (bar.done & 1) == (phase & 1):
        yield bar, bar.done
    expect(bar.done == phase + 1, "waited for phase", phase, "passed at", bar.done, bar.name)


STAGES, RING = 4, 8
FEW, SINGLE, PAIR, END = "few", "single", "pair", "end"


def simulate(tasks, seed, stages=STAGES, passed=True, fews_over=True):
    """tasks: (kind, key tiles) in order.  passed: warps start a task of few rows when both issuers are past it;
    fews_over: issuers go on when the warps are done with those before."""
    rng = random.Random(seed)
    bars = lambda name, n, count: [Bar(f"{name}{i}", count) for i in range(n)]  # noqa: E731
    q_full, q_empty = bars("q_full", 2, 1), bars("q_empty", 2, 8)
    full = {"k": bars("k_full", stages, 1), "v": bars("v_full", stages, 1)}
    empty = {"k": bars("k_empty", stages, 8), "v": bars("v_empty", stages, 8)}
    s_full = [bars(f"s_full{w}", 3, 1) for w in range(2)]
    p_ready = [bars(f"p_ready{w}", 3, 4) for w in range(2)]
    o_final, buf_free = bars("o_final", 2, 1), bars("buf_free", 3, 1)
    merge_ready, merge_free, few_q = Bar("merge_ready", 4), Bar("merge_free", 4), Bar("few_q", 8)
    few_full = bars("few_full", 2, 8)
    task_full, task_empty = bars("task_full", RING, 1), bars("task_empty", RING, 11)
    task_passed = bars("task_passed", 2 * RING, 2)

    ring = [None] * RING
    loads = []                       # copies in flight
    products = {"s": [], "pv": []}   # products and commits in flight, in order
    held = {"k": [None] * stages, "v": [None] * stages, "q": [None] * 2}  # the tile that a buffer holds
    scores = [None] * 3              # step whose scores (or P) a score buffer holds
    o_task = [None, None]            # task whose sums an accumulator holds
    o_read = [set(), set()]          # warps that still read it
    exchange = [None] * 8            # per 16 rows of the exchanged (m, l): what they hold
    exchange_read = [set() for _ in range(8)]  # warps that have to read it before it is written again

    def load(kind, slot, tile, bar):
        bar.expect_copy()

        def land():
            held[kind][slot] = tile
            bar.land()
        held[kind][slot] = None
        loads.append(land)

    def task(it):
        yield from wait(task_full[it % RING], it // RING)
        t = ring[it % RING]
        expect(t[0] == it, "task overwritten", it)
        return t[1:]

    def k_producer():
        tile = 0
        for it, (kind, n) in enumerate(tasks + [(END, 0)]):
            rot = rng.randrange(n) if kind in (SINGLE, PAIR) else 0
            yield from wait(task_empty[it % RING], it // RING - 1)
            ring[it % RING] = (it, kind, n, rot, rng.random() < 0.7)
            task_full[it % RING].arrive()
            yield
            if kind == END:
                return
            yield from wait(q_empty[it & 1], (it >> 1) - 1)
            load("q", it & 1, it, q_full[it & 1])
            for _ in range(n):
                yield from wait(empty["k"][tile % stages], tile // stages - 1)
                load("k", tile % stages, tile, full["k"][tile % stages])
                tile += 1
                yield

    def v_producer():
        tile = it = 0
        while True:
            kind, n, _, _ = yield from task(it)
            task_empty[it % RING].arrive()
            if kind == END:
                return
            for _ in range(n):
                yield from wait(empty["v"][tile % stages], tile // stages - 1)
                load("v", tile % stages, tile, full["v"][tile % stages])
                tile += 1
                yield
            it += 1

    def issuer(what):
        kv = "k" if what == "s" else "v"
        tile = step = it = few = over = 0
        turn = [0, 0]

        def commit(*acts):
            products[what].extend(acts)

        def tiles_done():
            nonlocal over
            if fews_over and over < few:
                yield from wait(few_full[over & 1], over >> 1)
                over += 1

        while True:
            kind, n, _, _ = yield from task(it)
            task_empty[it % RING].arrive()
            if kind == END:
                return
            if kind == FEW:
                task_passed[it % (2 * RING)].arrive()
                yield from tiles_done()
                few += 1
                tile += n
                it += 1
                continue
            yield from tiles_done()
            steps = 2 * n if kind == PAIR else n
            if what == "s":
                yield from wait(q_full[it & 1], it >> 1)
            for s in range(steps):
                wg = s & 1
                if kind == SINGLE or not wg:
                    yield from wait(full[kv][tile % stages], tile // stages)
                if what == "s":
                    yield from wait(buf_free[step % 3], step // 3 - 1)

                    def product(slot=tile % stages, want=tile, buf=step % 3, step=step, it=it):
                        expect(held["k"][slot] == want, "K overwritten", want)
                        expect(held["q"][it & 1] == it, "Q overwritten", it)
                        scores[buf] = ("s", step)
                    bar = s_full[wg][turn[wg] % 3]
                    commit(product, bar.arrive)
                else:
                    yield from wait(p_ready[wg][turn[wg] % 3], turn[wg] // 3)

                    def product(slot=tile % stages, want=tile, buf=step % 3, step=step, it=it, wg=wg, first=s < 2):
                        expect(held["v"][slot] == want, "V overwritten", want)
                        expect(scores[buf] == ("p", step, 4), "P not there", step, scores[buf])
                        expect(not first or not o_read[wg], "O overwritten", it, o_read[wg])
                        expect(first or o_task[wg] == it, "O of another task", it)
                        o_task[wg] = it
                    commit(product, buf_free[step % 3].arrive)
                    if s >= steps - 2:
                        commit(lambda wg=wg, warps=frozenset(range(4 * wg, 4 * wg + 4)): o_read[wg].update(warps),
                               o_final[wg].arrive)
                if kind == SINGLE or wg:
                    empty[kv][tile % stages].arrive(7)
                    commit(empty[kv][tile % stages].arrive)
                    tile += 1
                step += 1
                turn[wg] += 1
                yield
            if what == "s":
                q_empty[it & 1].arrive(7)
                commit(q_empty[it & 1].arrive)
            task_passed[it % (2 * RING)].arrive()
            it += 1

    def put(part, w, what, readers):
        expect(not exchange_read[part], "exchanged state overwritten by", w, exchange_read[part])
        exchange[part], exchange_read[part] = what, set(readers)

    def take(part, w, what):
        expect(exchange[part] == what, "exchanged state of another", exchange[part], what)
        exchange_read[part].discard(w)

    def warp(w):
        wg, quad = w >> 2, w & 3
        step0 = turn = tile0 = finals = merges = few = it = 0
        merge_open = False
        while True:
            kind, n, rot, ragged = yield from task(it)
            task_empty[it % RING].arrive()
            if kind == END:
                return
            if kind == FEW:
                if passed:
                    yield from wait(task_passed[it % (2 * RING)], it // (2 * RING))
                yield from wait(q_full[it & 1], it >> 1)
                expect(held["q"][it & 1] == it, "Q overwritten", it)
                few_q.arrive()
                yield
                for j in range(wg, n, 2):
                    u = tile0 + j
                    for kv in ("k", "v"):
                        yield from wait(full[kv][u % stages], u // stages)
                        yield
                        expect(held[kv][u % stages] == u, "tile overwritten", kv, u)
                        empty[kv][u % stages].arrive(2)
                yield from wait(few_q, few)
                held["q"][it & 1] = ("states", it)
                put(w, w, (it, w), range(8))
                yield
                few_full[few & 1].arrive()
                yield from wait(few_full[few & 1], few >> 1)
                for x in range(8):
                    yield
                    take(x, w, (it, x))
                expect(held["q"][it & 1] == ("states", it), "states overwritten", it)
                q_empty[it & 1].arrive()
                few += 1
                tile0 += n
                it += 1
                continue
            steps = n if kind == PAIR else (n + 1 - wg) >> 1
            for x in range(steps):
                j = x if kind == PAIR else 2 * x + wg
                step = step0 + 2 * x + wg
                yield from wait(s_full[wg][turn % 3], turn // 3)
                expect(scores[step % 3][1] == step, "scores of another step", step, scores[step % 3])
                if ragged and (j + rot) % n == n - 1 and (kind == SINGLE or wg == 0):
                    u = tile0 + j
                    yield from wait(full["v"][u % stages], u // stages)
                    expect(held["v"][u % stages] == u, "V overwritten", u)
                if x > 0 and rng.random() < 0.3:  # a rescale: the warpgroup's last product is complete
                    yield from wait(buf_free[(step - 2) % 3], (step - 2) // 3)
                yield
                if x == 0 and merge_open:
                    yield from wait(merge_free, merges - 1)
                    merge_open = False
                was = scores[step % 3]
                expect(was[1] == step, "scores of another step", step, was)
                scores[step % 3] = ("p", step, was[2] + 1 if was[0] == "p" else 1)
                p_ready[wg][turn % 3].arrive()
                turn += 1
                yield
            step0 += 2 * n if kind == PAIR else n
            tile0 += n
            it += 1
            if steps == 0:
                continue
            yield from wait(o_final[wg], finals)
            finals += 1
            merged = kind == SINGLE and n > 1
            if merged and wg == 1:
                if merge_open:
                    yield from wait(merge_free, merges - 1)
                for part in (2 * quad, 2 * quad + 1):
                    put(part, w, (it - 1, "merge"), [quad])
                yield
                o_read[1].discard(w)     # its lanes are the other warpgroup's to read
                o_read[1].add(quad)
                merge_ready.arrive()
                merges += 1
                merge_open = True
                continue
            if merged:
                yield from wait(merge_ready, merges)
                merges += 1
                for part in (2 * quad, 2 * quad + 1):
                    yield
                    take(part, w, (it - 1, "merge"))
                expect(o_task[1] == it - 1, "O of another task", it - 1)
            expect(o_task[wg] == it - 1, "O of another task", it - 1)
            yield
            o_read[wg].discard(w)
            if merged:
                o_read[1].discard(w)
                merge_free.arrive()

    agents = {"k": k_producer(), "v": v_producer(), "s": issuer("s"), "pv": issuer("pv")}
    agents.update({w: warp(w) for w in range(8)})
    pace = {a: rng.choice([0.02, 0.2, 1, 1, 3]) for a in agents}
    land, finish = rng.choice([0.05, 0.3, 0.9]), rng.choice([0.05, 0.3, 0.9])
    blocked = {}  # agents that wait: the barrier and its phase when they last looked
    while agents:
        ready = [a for a in agents if a not in blocked or blocked[a][0].done != blocked[a][1]]
        expect(ready or loads or any(products.values()), "nothing goes on", list(agents))
        if ready:
            a = rng.choices(ready, [pace[x] for x in ready])[0]
            blocked.pop(a, None)
            try:
                at = next(agents[a])
                if at is not None:
                    blocked[a] = at
            except StopIteration:
                del agents[a]
        if loads and rng.random() < land:
            loads.pop(rng.randrange(len(loads)))()
        for queue in products.values():
            while queue and rng.random() < finish:
                queue.pop(0)()


def random_tasks(rng):
    lengths = rng.choice([[1], [1, 2], [1, 2, 3, 7], [1, 5, 9]])
    kinds = rng.choice([[FEW], [SINGLE], [PAIR], [FEW, SINGLE], [FEW, SINGLE, PAIR], [SINGLE, SINGLE, SINGLE, FEW],
                        [FEW, FEW, FEW, PAIR]])
    return [(rng.choice(kinds), rng.choice(lengths)) for _ in range(rng.randint(1, 40))]
