"""Models of the serving kernels' synchronisation, run on the CPU.

As for the other kernels, the roles run as coroutines with random latencies over barriers with the hardware's parity
rule; every MMA, every TMEM read and write, every buffer's reuse and every parity wait is checked, and planted changes
show what the load-bearing pieces guard.

Packed forward (csrc/fa_fwd_packed.cu): the steps of the bf16 forward over items that follow one another in the same
CTA: ring slots, parities and Q buffers run on, the next item's first S may be issued before the last group's last P V,
K_0's barrier stands for group 0's Q tile, and the watcher returns Q tiles when an item's last S is done.

Cache attention (csrc/fa_cache8.cu): segments of a few tiles; S^T and P double-buffered (without barriers of their own that say
they have been read: the order of the products does), one O per CTA, which the next
segment's first P V overwrites; info slots without a barrier of their own for emptiness; Q and its scales in two buffers.
"""
import heapq
import random

import pytest

from test_wide_schedule import Barrier

WARPS = 4
ITEMS = 4


class Run:
    """The clock, the roles and what went wrong."""

    def __init__(self, seed):
        self.rng = random.Random(seed)
        self.errors, self.events, self.now = [], [], 0.0

    def wait(self, bar, parity, who, phase=None):
        yield ("wait", lambda: bar.passes(parity))
        if phase is not None and bar.done < phase + 1:
            self.errors.append(f"{who}: parity wait for phase {phase} passed on an older phase")

    def delay(self, lo, hi):
        return "delay", self.rng.uniform(lo, hi)

    def later(self, lo, hi, fn):
        heapq.heappush(self.events, (self.now + self.rng.uniform(lo, hi), self.rng.random(), ("call", fn)))

    def go(self, roles, endless, horizon, idle):
        """Runs the roles; those in `endless` need not finish. idle(): nothing is left for them to do."""
        waiting, finished = {}, set()
        needed = set(range(len(roles))) - endless
        for i in range(len(roles)):
            heapq.heappush(self.events, (0.0, self.rng.random(), ("run", i)))
        try:
            while self.events and self.now < horizon:
                self.now, _, (what, r) = heapq.heappop(self.events)
                if what == "call":
                    r()
                    continue
                if r in finished:
                    continue
                try:
                    y = waiting.pop(r) if r in waiting else next(roles[r])
                    while True:
                        if y[0] == "delay":
                            heapq.heappush(self.events, (self.now + y[1], self.rng.random(), ("run", r)))
                            break
                        if y[1]():
                            y = next(roles[r])
                            continue
                        waiting[r] = y
                        heapq.heappush(self.events, (self.now + self.rng.uniform(20, 200), self.rng.random(), ("run", r)))
                        break
                except StopIteration:
                    finished.add(r)
                if needed <= finished and idle():
                    break
        except AssertionError as e:
            self.errors.append(str(e))
            return self.errors
        if not needed <= finished:
            self.errors.append(f"deadlock: roles {sorted(needed - finished)} never finished")
        return self.errors


# ------------------------------------------------------------------ packed forward
def packed(items, seed, *, slots=4, q_after_s=True, gate=True, early_needs_group1=True, readers=11, softmax=(300, 1500)):
    """items: (nkv0, nkv1) key tiles of the two groups, as the kernel makes them: equal, one more for group 1, or
    none for it."""
    run = Run(seed)
    rng, errors = run.rng, run.errors
    full, empty = [Barrier(1) for _ in range(slots)], [Barrier(1) for _ in range(slots)]
    q1_full, q_empty = Barrier(1), [Barrier(1), Barrier(1)]
    s_full, o_final = [Barrier(1), Barrier(1)], [Barrier(1), Barrier(1)]
    p_ready = [Barrier(WARPS + 1), Barrier(WARPS + 1)]
    item_full, item_empty = [Barrier(1) for _ in range(ITEMS)], [Barrier(readers) for _ in range(ITEMS)]
    ring = [None] * ITEMS
    landed, in_flight = [None] * slots, [None] * slots
    q_now = [None, None]                           # the item whose Q tile the group's buffer holds
    tmem_s = [None, None]                          # ("S" | "P", item, j)
    p_written, o_read = {}, [set(range(WARPS)), set(range(WARPS))]
    s_done, pv_done = set(), set()
    used = {}                                      # load -> MMAs that read it and are done
    pipe = []
    first_load = [2 * sum(max(i) for i in items[:n]) for n in range(len(items) + 1)]

    def need(load):
        n = max(k for k in range(len(items)) if first_load[k] <= load)
        j = (load - first_load[n]) // 2
        return sum(j < x for x in items[n])

    def take(n, who):
        yield from run.wait(item_full[n % ITEMS], (n // ITEMS) & 1, who + " item", n // ITEMS)
        if ring[n % ITEMS] != n:
            errors.append(f"{who} took item {ring[n % ITEMS]} for {n}")

    def scheduler():
        for n in range(len(items) + 1):
            if n >= ITEMS:
                yield from run.wait(item_empty[n % ITEMS], ((n // ITEMS) & 1) ^ 1, "scheduler", n // ITEMS - 1)
            ring[n % ITEMS] = n
            item_full[n % ITEMS].arrive()
            yield run.delay(50, 4000)

    def tensor_core():
        while True:
            while not pipe:
                yield ("wait", lambda: bool(pipe))
            op = pipe.pop(0)
            if op[0] == "commit":
                op[1].arrive()
                continue
            kind, i, n, j, load = op
            if landed[load % slots] != load:
                errors.append(f"{kind}{i}({n},{j}) read slot {load % slots} holding {landed[load % slots]}, wanted {load}")
            if kind == "S":
                if q_now[i] != n:
                    errors.append(f"S{i}({n},{j}) read Q of item {q_now[i]}")
                if tmem_s[i] is not None and tmem_s[i][1:] not in pv_done_of(i):
                    errors.append(f"S{i}({n},{j}) overwrote {tmem_s[i]} before P V read it")
            else:
                if tmem_s[i] != ("P", n, j):
                    errors.append(f"PV{i}({n},{j}) read TMEM holding {tmem_s[i]}")
                if j == 0:
                    if len(o_read[i]) < WARPS:
                        errors.append(f"PV{i}({n},0) overwrote an O that {WARPS - len(o_read[i])} warps have not read")
                    o_read[i] = set()
            yield run.delay(200, 300)
            used[load] = used.get(load, 0) + 1
            if kind == "S":
                tmem_s[i] = ("S", n, j)
                s_done.add((i, n, j))
            else:
                pv_done.add((i, n, j))

    def pv_done_of(i):
        return {(n, j) for g, n, j in pv_done if g == i}

    def producer():
        c, nq = 0, [0, 0]
        for n, nkv in enumerate(items):
            yield from take(n, "producer")
            item_empty[n % ITEMS].arrive()
            for x in range(2 * max(nkv)):
                slot = c % slots
                yield from run.wait(empty[slot], ((c // slots) & 1) ^ 1, "producer", c // slots - 1 if c >= slots else None)
                if in_flight[slot] is not None:
                    errors.append(f"load {c} issued into slot {slot} with a load in flight")
                if c >= slots and used.get(c - slots, 0) < need(c - slots):
                    errors.append(f"load {c} overwrote load {c - slots} before its MMAs ran")
                full[slot].expect_tx(1 if x else 2)
                full[slot].arrive()
                in_flight[slot], landed[slot] = c, None

                def land(slot=slot, c=c):
                    in_flight[slot], landed[slot] = None, c
                    full[slot].complete_tx(1)
                run.later(300, 3000, land)
                if x == 0:
                    for i in range(2):
                        if nkv[i] == 0:
                            continue
                        yield from run.wait(q_empty[i], (nq[i] & 1) ^ 1, f"producer q{i}", nq[i] - 1 if nq[i] else None)
                        nq[i] += 1
                        last = q_now[i]
                        if last is not None and (i, last, items[last][i] - 1) not in s_done:
                            errors.append(f"Q{i} of item {n} overwrote that of item {last} before its last S")
                        q_now[i] = None
                        bar = q1_full if i else full[slot]
                        if i:
                            bar.expect_tx(1)
                            bar.arrive()

                        def land_q(i=i, n=n, bar=bar):
                            q_now[i] = n
                            bar.complete_tx(1)
                        run.later(300, 3000, land_q)
                c += 1

    def issuer():
        cur, np, nq1 = 0, [0, 0], 0

        def first(n, early):
            nonlocal cur, nq1
            if not early:
                yield from run.wait(full[cur % slots], (cur // slots) & 1, "issuer K_0", cur // slots)
                pipe.extend([("S", 0, n, 0, cur), ("commit", s_full[0])])
            if items[n][1] > 0:
                yield from run.wait(q1_full, nq1 & 1, "issuer Q_1", nq1)
                nq1 += 1
                pipe.extend([("S", 1, n, 0, cur), ("commit", s_full[1])])
            cur += 1

        yield from take(0, "issuer")
        item_empty[0].arrive()
        yield from first(0, False)
        for n, nkv in enumerate(items):
            yield from take(n + 1, "issuer")
            have = n + 1 < len(items)
            if have:
                item_empty[(n + 1) % ITEMS].arrive()
            for j in range(max(nkv)):
                v = cur
                cur += 1
                early = False
                for i in range(2):
                    if i == 1 and j + 1 == max(nkv) and have and (items[n + 1][1] > 0 or not early_needs_group1) and \
                            full[cur % slots].passes((cur // slots) & 1):
                        early = True
                        pipe.extend([("S", 0, n + 1, 0, cur), ("commit", s_full[0])])
                    if j >= nkv[i]:
                        continue
                    yield from run.wait(p_ready[i], np[i] & 1, f"issuer P{i}", np[i])
                    np[i] += 1
                    pipe.append(("PV", i, n, j, v))
                    if j + 1 < nkv[i]:
                        pipe.extend([("S", i, n, j + 1, cur), ("commit", s_full[i])])
                    else:
                        pipe.append(("commit", o_final[i]))
                if j + 1 < max(nkv):
                    cur += 1
                elif have:
                    yield from first(n + 1, early)

    def watcher():
        c0, np, ns = 0, [0, 0], [0, 0]

        def hand(i):
            if np[i] > 0 and gate:
                yield from run.wait(p_ready[i], (np[i] - 1) & 1, f"watcher gate{i}", np[i] - 1)
            elif p_ready[i].done < np[i]:
                errors.append(f"watcher arrived for P-ready{i} phase {np[i]} inside phase {p_ready[i].done}")
            p_ready[i].arrive()
            np[i] += 1

        for n, nkv in enumerate(items):
            yield from take(n, "watcher")
            item_empty[n % ITEMS].arrive()
            nmax = max(nkv)
            last = 1 if nkv[1] == nmax else 0
            yield from run.wait(full[c0 % slots], (c0 // slots) & 1, "watcher K_0", c0 // slots)
            for j in range(nmax):
                cv = c0 + 2 * j + 1
                yield from run.wait(full[cv % slots], (cv // slots) & 1, "watcher V", cv // slots)
                if j + 1 < nmax:
                    yield from run.wait(full[(cv + 1) % slots], ((cv + 1) // slots) & 1, "watcher K", (cv + 1) // slots)
                if last == 1 and j < nkv[0]:
                    yield from hand(0)
                if q_after_s or j + 1 < nmax:
                    yield from run.wait(s_full[last], (ns[last] + j) & 1, "watcher S", ns[last] + j)
                empty[(cv - 1) % slots].arrive()
                if cv > 1:
                    empty[(cv - 2) % slots].arrive()
                if j + 1 == nmax:
                    for i in range(2):
                        if nkv[i]:
                            q_empty[i].arrive()
                yield from hand(last)
            c0 += 2 * nmax
            ns = [ns[0] + nkv[0], ns[1] + nkv[1]]

    def group(i, w):
        ns = no = 0
        for n, nkv in enumerate(items):
            yield from take(n, f"softmax{i}")
            for j in range(nkv[i]):
                yield from run.wait(s_full[i], ns & 1, f"softmax{i} S", ns)
                ns += 1
                if tmem_s[i] != ("S", n, j):
                    errors.append(f"softmax{i} warp {w} read S({n},{j}) from TMEM holding {tmem_s[i]}")
                yield run.delay(*softmax)
                done = p_written.setdefault((i, n, j), set())
                done.add(w)
                if j > 0 and rng.random() < 0.3 and (i, n, j - 1) not in pv_done:
                    errors.append(f"softmax{i} rescaled O while P V({n},{j - 1}) was pending")
                if len(done) == WARPS:
                    tmem_s[i] = ("P", n, j)
                p_ready[i].arrive()
            item_empty[n % ITEMS].arrive()
            if nkv[i]:
                yield from run.wait(o_final[i], no & 1, f"softmax{i} O", no)
                no += 1
                if (i, n, nkv[i] - 1) not in pv_done:
                    errors.append(f"softmax{i} read O of item {n} before its last P V")
                yield run.delay(300, 3000)
                o_read[i].add(w)

    roles = [tensor_core(), scheduler(), producer(), issuer(), watcher()] + [group(i, w) for i in range(2) for w in range(WARPS)]
    return run.go(roles, {0}, 25000.0 * (sum(map(max, items)) + len(items) + 4), lambda: not pipe)


TWO_HEADS = [[(1, 1)] * 6, [(3, 3), (2, 2), (1, 1), (1, 1), (1, 1)], [(7, 7), (1, 1), (5, 5)], [(2, 2)] * 9, [(4, 4)]]
ONE_HEAD = [[(1, 2), (1, 0), (1, 0)], [(3, 4), (2, 0), (1, 2), (1, 0), (5, 6)], [(1, 0)] * 7, [(2, 2), (2, 0), (3, 3)]]


@pytest.mark.parametrize("items", TWO_HEADS + ONE_HEAD)
@pytest.mark.parametrize("slots", [4, 10])
@pytest.mark.parametrize("softmax", [(300, 1500), (50, 6000)])
def test_packed_protocol_holds(items, slots, softmax):
    for seed in range(25):
        errs = packed(items, seed, slots=slots, softmax=softmax)
        assert not errs, (items, seed, errs[:3])


def bad_packed(cases, **kw):
    return sum(bool(packed(items, seed, softmax=(50, 6000), **kw)) for items in cases for seed in range(15))


def test_packed_q_goes_back_after_the_last_s():
    assert bad_packed(TWO_HEADS, q_after_s=False) > 0


def test_packed_watcher_gate_needed_with_a_deeper_ring():
    assert bad_packed(TWO_HEADS, slots=10, gate=False) > 0


def test_packed_early_s_only_where_the_next_item_has_group_1():
    """Else the next item's first S of group 0 is what the watcher takes for this item's last."""
    assert bad_packed(ONE_HEAD, early_needs_group1=False) > 0


# ------------------------------------------------------------------ cache attention
def cached(tiles, seed, *, ring=6, q_bufs=2, infos=8, q_empty_count=2, rescale_wait=True, softmax=(200, 900)):
    """tiles: of each segment."""
    run = Run(seed)
    rng, errors = run.rng, run.errors
    full, empty = [Barrier(1) for _ in range(ring)], [Barrier(1) for _ in range(ring)]
    info_full = [Barrier(1) for _ in range(infos)]
    s_full = [Barrier(1), Barrier(1)]
    p_ready, p_empty = [Barrier(WARPS), Barrier(WARPS)], [Barrier(1), Barrier(1)]
    q_full, q_empty = [Barrier(1) for _ in range(q_bufs)], [Barrier(q_empty_count) for _ in range(q_bufs)]
    total = sum(tiles)
    seg_of = [g for g, n in enumerate(tiles) for _ in range(n)]
    first = [sum(tiles[:g]) for g in range(len(tiles))]
    landed, in_flight = [None] * ring, [None] * ring
    info = [None] * infos
    q_now, q_scale = [None] * q_bufs, [None] * q_bufs
    s_now, s_read = [None, None], {}
    p_now = [None, None]                           # (tile, warps)
    o_read = set(range(WARPS))
    s_done, pv_done, info_read, scales_read = set(), set(), {}, {}
    used, pipe = set(), []
    meet = {}                                      # the softmax warps' named barrier

    def gather(key):
        meet[key] = meet.get(key, 0) + 1
        yield ("wait", lambda: meet[key] == WARPS)

    def tensor_core():
        while True:
            while not pipe:
                yield ("wait", lambda: bool(pipe))
            op = pipe.pop(0)
            if op[0] == "commit":
                op[1].arrive()
                continue
            kind, t, load = op
            nonlocal o_read
            if landed[load % ring] != load:
                errors.append(f"{kind}({t}) read slot {load % ring} holding {landed[load % ring]}, wanted {load}")
            b = t & 1
            if kind == "S":
                if q_now[seg_of[t] % q_bufs] != seg_of[t]:
                    errors.append(f"S({t}) read Q of segment {q_now[seg_of[t] % q_bufs]}")
                if t >= 2 and len(s_read.get(t - 2, ())) < WARPS:
                    errors.append(f"S({t}) overwrote S({t - 2}) before all had read it")
                s_now[b] = None
            else:
                if p_now[b] is None or p_now[b][0] != t or len(p_now[b][1]) < WARPS:
                    errors.append(f"PV({t}) read a P buffer holding {p_now[b]}")
                if t == first[seg_of[t]]:
                    if t and len(o_read) < WARPS:
                        errors.append(f"PV({t}) overwrote an O that was not read")
                    o_read = set()
            yield run.delay(100, 200)
            used.add(load)
            if kind == "S":
                s_now[b] = t
                s_done.add(t)
            else:
                pv_done.add(t)

    def producer():
        c = 0
        for t in range(total):
            for _ in range(2):
                slot = c % ring
                yield from run.wait(empty[slot], ((c // ring) & 1) ^ 1, "producer", c // ring - 1 if c >= ring else None)
                if in_flight[slot] is not None or (c >= ring and c - ring not in used):
                    errors.append(f"load {c} overwrote load {c - ring} before its MMAs ran")
                full[slot].expect_tx(1)
                full[slot].arrive()
                in_flight[slot], landed[slot] = c, None

                def land(slot=slot, c=c):
                    in_flight[slot], landed[slot] = None, c
                    full[slot].complete_tx(1)
                run.later(300, 3000, land)
                c += 1
            if t >= infos and len(info_read.get(t - infos, ())) < WARPS:
                errors.append(f"scales of tile {t} overwrote those of tile {t - infos} before all had read them")
            info[t % infos] = t
            info_full[t % infos].arrive()
            yield run.delay(20, 400)

    def issuer():
        def scores(t):
            yield from run.wait(full[2 * t % ring], (2 * t // ring) & 1, "issuer K", 2 * t // ring)
            pipe.extend([("S", t, 2 * t), ("commit", s_full[t & 1]), ("commit", empty[2 * t % ring])])

        t = 0
        for g, n in enumerate(tiles):
            yield from run.wait(q_full[g % q_bufs], (g // q_bufs) & 1, "issuer Q", g // q_bufs)
            yield from scores(t)
            for j in range(n):
                if j + 1 < n:
                    yield from scores(t + 1)
                else:
                    pipe.append(("commit", q_empty[g % q_bufs]))
                v = 2 * t + 1
                yield from run.wait(full[v % ring], (v // ring) & 1, "issuer V", v // ring)
                yield from run.wait(p_ready[t & 1], (t >> 1) & 1, "issuer P", t >> 1)
                pipe.extend([("PV", t, v), ("commit", p_empty[t & 1]), ("commit", empty[v % ring])])
                t += 1

    def queries():
        for g in range(len(tiles)):
            b = g % q_bufs
            yield from run.wait(q_empty[b], ((g // q_bufs) & 1) ^ 1, "queries", g // q_bufs - 1 if g >= q_bufs else None)
            if g >= q_bufs:
                old = g - q_bufs
                if first[old] + tiles[old] - 1 not in s_done:
                    errors.append(f"Q of segment {g} overwrote that of segment {old} before its last S")
                if len(scales_read.get(old, ())) < WARPS:
                    errors.append(f"scales of Q of segment {g} overwrote those of segment {old}")
            q_now[b] = None
            yield run.delay(300, 3000)
            q_now[b] = q_scale[b] = g
            q_full[b].arrive()

    def softmax_warp(w):
        t = 0
        for g, n in enumerate(tiles):
            for j in range(n):
                b = t & 1
                if j == 0:
                    yield from run.wait(q_full[g % q_bufs], (g // q_bufs) & 1, "softmax Q", g // q_bufs)
                yield from run.wait(info_full[t % infos], (t // infos) & 1, "softmax info", t // infos)
                yield from run.wait(s_full[b], (t >> 1) & 1, "softmax S", t >> 1)
                if info[t % infos] != t or s_now[b] != t or q_scale[g % q_bufs] != g:
                    errors.append(f"softmax took tile {info[t % infos]}, S({s_now[b]}), segment {q_scale[g % q_bufs]} for {t}, {g}")
                yield run.delay(50, 300)
                s_read.setdefault(t, set()).add(w)
                info_read.setdefault(t, set()).add(w)
                if j + 1 == n:
                    scales_read.setdefault(g, set()).add(w)
                grow = j == 0 or random.Random((seed, t).__hash__()).random() < 0.2      # the same for all warps
                if j > 0:
                    yield from gather(("grow?", t))
                if grow:
                    yield from gather(("top", t))
                    yield from gather(("raised", t))
                    if j > 0 and rescale_wait:
                        yield from run.wait(p_empty[b ^ 1], ((t - 1) >> 1) & 1, "softmax rescale", (t - 1) >> 1)
                    if j > 0 and t - 1 not in pv_done:
                        errors.append(f"O rescaled before P V({t - 1})")
                if t >= 2 and t - 2 not in pv_done:
                    errors.append(f"P({t}) overwrote P({t - 2}) before P V read it")
                if p_now[b] is None or p_now[b][0] != t:
                    p_now[b] = (t, set())
                yield run.delay(*softmax)
                p_now[b][1].add(w)
                p_ready[b].arrive()
                t += 1
            last = t - 1
            yield from gather(("sums", g))
            if w == 0 and q_empty_count == 2:
                q_empty[g % q_bufs].arrive()
            yield from run.wait(p_empty[last & 1], (last >> 1) & 1, "softmax O", last >> 1)
            yield from gather(("final", g))
            if last not in pv_done:
                errors.append(f"O of segment {g} read before its last P V")
            yield run.delay(200, 2000)
            o_read.add(w)

    roles = [tensor_core(), producer(), issuer(), queries()] + [softmax_warp(w) for w in range(WARPS)]
    return run.go(roles, {0}, 25000.0 * (total + 2 * len(tiles) + 4), lambda: not pipe)


SEGMENTS = [[1], [5], [1, 1, 1, 1], [3, 1, 4], [9, 2], [2, 1, 1, 7, 1], [1] * 9]


@pytest.mark.parametrize("tiles", SEGMENTS)
@pytest.mark.parametrize("ring", [3, 6])
@pytest.mark.parametrize("softmax", [(200, 900), (20, 5000)])
def test_cache_protocol_holds(tiles, ring, softmax):
    for seed in range(25):
        errs = cached(tiles, seed, ring=ring, softmax=softmax)
        assert not errs, (tiles, seed, errs[:3])


def bad_cached(**kw):
    return sum(bool(cached(tiles, seed, softmax=(20, 5000), **kw)) for tiles in SEGMENTS for seed in range(15))


def test_cache_queries_wait_for_the_scales_readers_too():
    assert bad_cached(q_empty_count=1) > 0


def test_cache_rescale_waits_for_the_last_product():
    assert bad_cached(rescale_wait=False) > 0


def test_cache_info_slots_outnumber_the_tiles_ahead():
    """The ring holds the producer: with 8 slots no tile's scales are overwritten early, with 2 some are."""
    assert bad_cached(infos=2) > 0
