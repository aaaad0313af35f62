"""Host models of the chunks' attention (csrc/fa_cache8_chunk.cu), on the CPU.

The line of units: the kernel's arithmetic, step by step, against a plain enumeration of the items and their key tiles:
every key tile of every item is some part's exactly once, parts are as long as they should be, and each item that several
parts share is joined once, from the partial results that those parts wrote.

The hand-offs: the roles as coroutines with random latencies over barriers with the hardware's parity rule, every product,
buffer reuse and parity wait checked; planted changes show what the load-bearing pieces guard.
"""
import random

import pytest

from test_serving_schedule import Run
from test_wide_schedule import Barrier

TURN, CTAS = 1, 152


# ------------------------------------------------------------------ the line
def floor_sum(n, m, a, b):
    s = 0
    while n > 0:
        s += n * (n - 1) // 2 * (a // m) + n * (b // m)
        a, b = a % m, b % m
        y = a * n + b
        assert y < 2 ** 32
        n, b = y // m, y % m
        m, a = a, m
        if m == 0:
            break
    return s


class Line:
    """seqs: (new tokens, length) per sequence."""

    def __init__(self, seqs, Hkv, G, groups, causal, ctas=CTAS):
        self.seqs, self.Hkv, self.causal, self.tt, self.groups = seqs, Hkv, causal, 128 // G, groups
        self.span = self.tt * groups
        units = sum(self.tiles_before(s, self.items(s)) for s in seqs) * Hkv
        items = sum(self.items(s) for s in seqs) * Hkv
        self.turn = min(TURN, units // (2 * ctas))
        self.total = units + self.turn * items
        self.parts = min(ctas, self.total)

    def items(self, s):
        return -(-s[0] // self.span)

    def tiles(self, s, last):
        return max(1, ((s[1] - s[0] + last if self.causal else s[1]) + 127) >> 7)

    def end_of(self, s, item):
        return min(s[0], (item + 1) * self.span)

    def tiles_before(self, s, x):
        if x == 0:
            return 0
        if not self.causal:
            return x * self.tiles(s, s[0])
        total = 0
        if x == self.items(s):
            x -= 1
            total = self.tiles(s, s[0])
        if x == 0:
            return total
        past = s[1] - s[0]
        ones = 0 if past > 128 else min(x, (128 - past) // self.span)
        total += ones
        if x > ones:
            total += floor_sum(x - ones, 128, self.span, (ones + 1) * self.span + past + 127)
        return total

    def begin(self, i):
        return self.total * i // self.parts

    def part_of(self, u):
        return ((u + 1) * self.parts - 1) // self.total

    def place(self, u):
        before = 0
        for b, s in enumerate(self.seqs):
            each = self.tiles_before(s, self.items(s)) + self.turn * self.items(s)
            if u < before + each * self.Hkv:
                break
            before += each * self.Hkv
        h = (u - before) // each
        before += h * each
        lo, n = 0, self.items(s)
        while n > 1:
            step = -(-n // 32)
            k = -1
            for lane in range(32):
                i = lo + min(lane * step, n - 1)
                k += before + self.tiles_before(s, i) + self.turn * i <= u and lane * step < n
            left = n - k * step
            lo += k * step
            n = min(step, left)
        start = before + self.tiles_before(s, lo) + self.turn * lo
        return b, h, lo, u - start, start

    def segments(self, part):
        """(b, h, item, t0, t1, tiles, split, n0) as a part's roles walk them."""
        u0, u1 = self.begin(part), self.begin(part + 1)
        b, h, item, off, _ = self.place(u0)
        left, out = u1 - u0, []
        while left > 0:
            s = self.seqs[b]
            tiles = self.tiles(s, self.end_of(s, item))
            take = min(left, self.turn + tiles - off)
            t0, t1 = max(0, off - self.turn), off + take - self.turn
            tok0 = item * self.span
            split = self.groups == 2 and tok0 + self.tt >= s[0]
            n0 = max(0, min(self.tiles(s, min(s[0], tok0 + self.tt)), t1) - t0)
            seg = (b, h, item, t0, t1, tiles, split, n0)
            left -= take
            off = 0
            item += 1
            if item == self.items(s):
                item, h = 0, h + 1
                if h == self.Hkv:
                    h, b = 0, b + 1
                    while left > 0 and b < len(self.seqs) and self.seqs[b][0] == 0:
                        b += 1
                    if b >= len(self.seqs):
                        left = 0
            if t1 <= t0:
                assert left == 0
                break
            out.append(seg)
        return out

    def joins(self, i):
        """The parts that the join of second part i reads, as (part, slot), and the item; None: nothing to join."""
        if i >= self.parts:
            return None
        b, h, item, off, start = self.place(self.begin(i))
        if off <= self.turn:
            return None
        s = self.seqs[b]
        c0 = self.part_of(start + self.turn)
        if c0 != i - 1:
            return None
        c1 = self.part_of(start + self.turn + self.tiles(s, self.end_of(s, item)) - 1)
        return [(c, 0 if c > c0 or self.begin(c0) >= start else 1) for c in range(c0, c1 + 1)], (b, h, item)


def cases():
    rng = random.Random(5)
    fixed = [([(1, 1)], 1, 1), ([(0, 50), (5, 5), (0, 0), (3, 900)], 2, 4), ([(4096, 32768)], 8, 4), ([(64, 131072), (66, 70000)], 8, 8),
             ([(1024, 9000)] + [(1, 3000 + 17 * i) for i in range(24)], 8, 8), ([(700, 300)], 3, 7), ([(5000, 5000)], 1, 128),
             ([(300, 0)], 2, 1), ([(1, 60)] * 500, 4, 4)]
    for seqs, Hkv, G in fixed:
        yield seqs, Hkv, G
    for _ in range(30):
        n = rng.choice([1, 2, 5, 40])
        seqs = []
        for _ in range(n):
            new = int(rng.choice([0, 1, 2, rng.random() ** 3 * 3000]))
            seqs.append((new, max(0, new + int(rng.choice([0, rng.random() ** 2 * 20000, -rng.random() * 50, 128, 127])))))
        if any(s[0] for s in seqs):
            yield seqs, rng.choice([1, 2, 8]), rng.choice([1, 2, 3, 4, 7, 8, 64, 100])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("groups", [1, 2])
def test_every_key_tile_is_some_parts_once_and_joined(groups, causal):
    for seqs, Hkv, G in cases():
        line = Line(seqs, Hkv, G, groups, causal)
        want = {}
        for b, s in enumerate(seqs):
            n_items = -(-s[0] // line.span)
            for i in range(n_items):
                tiles = line.tiles(s, line.end_of(s, i))
                assert line.tiles_before(s, i) == sum(line.tiles(s, line.end_of(s, x)) for x in range(i))
                for h in range(Hkv):
                    want[b, h, i] = tiles
            assert line.tiles_before(s, n_items) == sum(line.tiles(s, line.end_of(s, x)) for x in range(n_items))
        got, partial = {}, {}
        for part in range(line.parts):
            segs = line.segments(part)
            assert segs, "a part without units"
            assert len(segs) == 1 or all(x[4] == x[5] for x in segs[:-1])
            for k, (b, h, item, t0, t1, tiles, split, n0) in enumerate(segs):
                assert tiles == want[b, h, item] and 0 <= t0 < t1 <= tiles
                assert t0 == 0 or k == 0                      # partial results: the first segment, or one that goes on
                got.setdefault((b, h, item), []).append((t0, t1))
                if (t0, t1) != (0, tiles):
                    slot = (part, 0 if k == 0 else 1)
                    assert slot not in partial
                    partial[slot] = (b, h, item)
        assert set(got) == set(want)
        for key, spans in got.items():
            spans.sort()
            assert spans[0][0] == 0 and spans[-1][1] == want[key]
            assert all(a[1] == b[0] for a, b in zip(spans, spans[1:]))
        joined = {}
        for i in range(1, CTAS):
            j = line.joins(i)
            if j:
                assert j[1] not in joined
                joined[j[1]] = j[0]
        assert {k for k, v in got.items() if len(v) > 1} == set(joined)
        for item, slots in joined.items():
            assert sorted(slots) == sorted(k for k, v in partial.items() if v == item)


# ------------------------------------------------------------------ the hand-offs
def chunk(segments, seed, *, groups=2, ring_k=3, q_read=True, other_empty=True, infos=8, v_late=2, s_first=True, k_first=True, land_in=(300, 1500), scales=2000, horizon=2e6, softmax=(300, 1500), convert=(200, 900)):
    """segments: (split, n0, n). WARPS stand for a softmax group's four, and for the converters'."""
    WARPS, RING_V = 2, 2
    per = 1 if groups == 2 else 2
    run = Run(seed)
    errors = run.errors
    k_full, k_empty = [Barrier(1) for _ in range(ring_k)], [Barrier(1) for _ in range(ring_k)]
    c_full, c_empty = [Barrier(1) for _ in range(2)], [Barrier(WARPS) for _ in range(2)]
    v_full, v_empty = [Barrier(WARPS) for _ in range(2)], [Barrier(1) for _ in range(2)]
    watched = groups == 2
    s_full, p_ready, o_final = ([Barrier(1), Barrier(1)], [Barrier(WARPS + watched), Barrier(WARPS + watched)], [Barrier(1), Barrier(1)])
    q_full, q_empty = Barrier(WARPS), Barrier(1 + (WARPS * groups if q_read else 0))
    other_full, other_emptied = Barrier(WARPS), Barrier(WARPS)
    info = [None] * infos
    item_full, item_empty = [Barrier(1) for _ in range(4)], [Barrier(2 + WARPS + (1 if watched else 0) + WARPS * groups) for _ in range(4)]
    ring = [None] * 4

    def take(seg, who):
        yield from run.wait(item_full[seg % 4], (seg // 4) & 1, who + " item", seg // 4)
        if ring[seg % 4] != seg:
            errors.append(f"{who} took {ring[seg % 4]} for {seg}")

    def done(seg, who):
        if ring[seg % 4] != seg:
            errors.append(f"{who}: item {seg} was overwritten")
        item_empty[seg % 4].arrive()

    def scheduler():
        for seg in range(len(segments)):
            if seg >= 4:
                yield from run.wait(item_empty[seg % 4], ((seg // 4) & 1) ^ 1, "scheduler", seg // 4 - 1)
            ring[seg % 4] = seg
            item_full[seg % 4].arrive()
            yield run.delay(50, 3000)
    k_slot, c_slot, v_slot = [None] * ring_k, [None] * 2, [set() for _ in range(2)]
    q_now, scale_now = [set()], [set()]
    tmem_s, o_owner = [None, None], [None, None]
    v_read, s_read = {}, {}
    pipe, done_pv = [], set()
    p_count = {}
    o_reading = [set(), set()]

    def tensor_core():
        while True:
            while not pipe:
                yield ("wait", lambda: bool(pipe))
            op = pipe.pop(0)
            if op[0] == "commit":
                op[1].arrive()
                continue
            kind, seg, buf, g, t, first = op
            if kind == "S":
                if k_slot[t % ring_k] != t:
                    errors.append(f"S({t}) read K {k_slot[t % ring_k]}")
                if q_now[0] != {(seg, w) for w in range(WARPS)}:
                    errors.append(f"S({t}) of segment {seg} read Q {q_now[0]}")
                if tmem_s[buf] is not None and tmem_s[buf][0] == "P" and tmem_s[buf][1:] not in done_pv:
                    errors.append(f"S({t}) overwrote P {tmem_s[buf]}")
                yield run.delay(400, 600)
                tmem_s[buf] = ("S", g, t)
            else:
                if tmem_s[buf] != ("P", g, t):
                    errors.append(f"PV({g},{t}) read {tmem_s[buf]}")
                for x in range(per):
                    c = t * per + x
                    if v_slot[c % 2] != {(c, w) for w in range(WARPS)}:
                        errors.append(f"PV({t}) read V {v_slot[c % 2]}, wanted {c}")
                if first and o_reading[g]:
                    errors.append(f"PV({g},{t}) overwrote O while it was read")
                yield run.delay(400, 600)
                for x in range(per):
                    c = t * per + x
                    if v_slot[c % 2] != {(c, w) for w in range(WARPS)}:
                        errors.append(f"V {c} changed under PV({t})")
                done_pv.add((g, t))
                o_owner[g] = seg

    def producer():
        t = 0
        for seg, (split, n0, n) in enumerate(segments):
            yield from take(seg, "producer")
            done(seg, "producer")
            for i in range(n + 1):                       # K a tile ahead of V
                if i < n:
                    yield from run.wait(k_empty[t % ring_k], ((t // ring_k) & 1) ^ 1, "producer K", t // ring_k - 1)
                    ready = [0]

                    def land(t=t, ready=ready):          # the bytes and the producer's arrival behind the scales
                        ready[0] += 1
                        if ready[0] == 2:
                            k_full[t % ring_k].arrive()

                    def bytes_there(t=t, land=land):
                        k_slot[t % ring_k] = t
                        land()
                    run.later(*land_in, bytes_there)
                    yield run.delay(5, scales)
                    info[t % infos] = t
                    land()
                    t += 1
                for x in range(per if i > 0 else 0):
                    c = (t - 2 if i < n else t - 1) * per + x
                    yield from run.wait(c_empty[c % 2], ((c // 2) & 1) ^ 1, "producer V", c // 2 - 1)

                    def land_v(c=c):
                        c_slot[c % 2] = c
                        c_full[c % 2].arrive()
                    run.later(*land_in, land_v)

    def issuer():
        t, np = 0, [0, 0]

        def scores(seg, buf, g, t):
            pipe.append(("S", seg, buf, g, t, False))
            pipe.append(("commit", s_full[buf]))
            yield run.delay(20, 300)

        def k_there(t):
            yield from run.wait(k_full[t % ring_k], (t // ring_k) & 1, f"S {t}", t // ring_k)

        def p_there(buf):
            yield from run.wait(p_ready[buf], np[buf] & 1, f"P ready {buf}", np[buf])
            np[buf] += 1
        for seg, (split, n0, n) in enumerate(segments):
            yield from take(seg, "issuer")
            done(seg, "issuer")
            yield from run.wait(q_full, seg & 1, "issuer Q", seg)
            if groups == 1:
                for j in range(-1, n):
                    if j + 1 < n:
                        at = t + j + 1
                        yield from k_there(at)
                        yield from scores(seg, at & 1, 0, at)
                        pipe.append(("commit", k_empty[at % ring_k]))
                    else:
                        pipe.append(("commit", q_empty))
                    if j >= 0:
                        yield from p_there((t + j) & 1)
                        for x in range(per):
                            c = (t + j) * per + x
                            yield from run.wait(v_full[c % 2], (c // 2) & 1, f"V {c}", c // 2)
                        pipe.append(("PV", seg, (t + j) & 1, 0, t + j, j == 0))
                        for x in range(per):
                            pipe.append(("commit", v_empty[((t + j) * per + x) % 2]))
                pipe.append(("commit", o_final[0]))
            else:
                k_next = t
                for i in range(-2, n if split else 2 * n):
                    gr, j = i & 1, i if split else i >> 1
                    mine, next_j, last = (n if split or gr else n0), (i + 2 if split else j + 1), split or gr
                    if j >= mine:
                        continue
                    if i >= 0:
                        yield from p_there(gr)
                        pipe.append(("PV", seg, gr, gr, t + j, i <= 1 if split else j == 0))
                        yield run.delay(20, 300)
                    elif next_j < mine and (split or not gr or n0 <= 0):
                        yield from k_there(k_next)
                    if next_j < mine:
                        assert k_next == t + next_j
                        yield from scores(seg, gr, gr, t + next_j)
                        k_next += bool(last)
                    elif i >= 0:
                        pipe.append(("commit", o_final[gr]))
                    if last and next_j + 1 == n:
                        pipe.append(("commit", q_empty))
            t += n

    def watcher():
        t0, k_seen, v_back, ns, np = 0, 0, 0, [0, 0], [0, 0]

        def hand(g):
            if np[g] > 0:
                yield from run.wait(p_ready[g], (np[g] - 1) & 1, f"watcher P {g}", np[g] - 1)
            p_ready[g].arrive()
            np[g] += 1

        def k_there(last):
            nonlocal k_seen
            while k_seen <= last:
                yield from run.wait(k_full[k_seen % ring_k], (k_seen // ring_k) & 1, f"watcher K {k_seen}", k_seen // ring_k)
                k_seen += 1
        for seg, (split, n0, n) in enumerate(segments):
            yield from take(seg, "watcher")
            done(seg, "watcher")
            for x in range(n):
                t, g = t0 + x, x & 1 if split else 1
                early = (split or x == 0) and s_first

                def s_done():
                    yield from run.wait(s_full[g], ns[g] & 1, f"watcher S {t}", ns[g])
                    ns[g] += 1
                    k_empty[t % ring_k].arrive()
                    nonlocal v_back
                    while v_back <= (t - v_late if split and x > 0 else t - 1):
                        v_empty[v_back & 1].arrive()
                        v_back += 1
                if early:
                    if k_first:
                        yield from k_there(t)
                    yield from s_done()
                yield from run.wait(v_full[t & 1], (t >> 1) & 1, f"watcher V {t}", t >> 1)
                yield from k_there(t0 + min(n - 1, x + 2 if split else x + 1))
                if not split and x < n0:
                    yield from hand(0)
                if not early:
                    yield from s_done()
                yield from hand(g)
                yield run.delay(20, 500)
            if not split:
                ns[0] += n0
            t0 += n

    def converter(w):
        t = 0
        for seg, (split, n0, n) in enumerate(segments):
            yield from take(seg, "converter")
            yield from run.wait(q_empty, (seg & 1) ^ 1, "converter Q", seg - 1)
            q_now[0] = {x for x in q_now[0] if x[0] == seg}
            scale_now[0] = {x for x in scale_now[0] if x[0] == seg}
            yield run.delay(300, 2500)
            q_now[0].add((seg, w))
            scale_now[0].add((seg, w))
            q_full.arrive()
            done(seg, "converter")
            for j in range(n):
                for x in range(per):
                    c = t * per + x
                    yield from run.wait(c_full[c % 2], (c // 2) & 1, f"codes {c}", c // 2)
                    yield from run.wait(v_empty[c % 2], ((c // 2) & 1) ^ 1, f"V empty {c}", c // 2 - 1)
                    if c_slot[c % 2] != c:
                        errors.append(f"converted codes {c_slot[c % 2]} for {c}")
                    if info[t % infos] != t:
                        errors.append(f"converter read info {info[t % infos]} for {t}")
                    v_slot[c % 2] = {y for y in v_slot[c % 2] if y[0] == c}
                    yield run.delay(*convert)
                    if c_slot[c % 2] != c:
                        errors.append(f"codes {c} changed under the conversion")
                    v_slot[c % 2].add((c, w))
                    c_empty[c % 2].arrive()
                    v_full[c % 2].arrive()
                t += 1

    def softmax_warp(g, w):
        t, ns, no, nm = 0, [0, 0], 0, 0
        for seg, (split, n0, n) in enumerate(segments):
            x0, dx = (g, 2) if split else (0, 1)
            nx = n if split or g == 1 or groups == 1 else n0
            yield from take(seg, f"softmax {g}")
            yield from run.wait(q_full, seg & 1, f"softmax {g} Q", seg)
            yield run.delay(5, 300)
            if scale_now[0] != {(seg, x) for x in range(WARPS)} and nx > x0:
                errors.append(f"softmax {g} read scales {scale_now[0]} in {seg}")
            if q_read:
                q_empty.arrive()
            for x in range(x0, nx, dx):
                at = t + x
                buf = at & 1 if groups == 1 else g
                want = at >> 1 if groups == 1 else ns[0]
                yield from run.wait(s_full[buf], want & 1, f"softmax {g} S {at}", want)
                ns[0] += 1
                if info[at % infos] != at:
                    errors.append(f"softmax {g} read info {info[at % infos]} for {at}")
                if tmem_s[buf] is None or tmem_s[buf][1:] != (g, at):
                    errors.append(f"softmax {g} read {tmem_s[buf]}, wanted S of {at}")
                yield run.delay(*softmax)
                if info[at % infos] != at:
                    errors.append(f"softmax {g}: info {at} overwritten")
                p_count[g, at] = p_count.get((g, at), 0) + 1
                if p_count[g, at] == WARPS:
                    tmem_s[buf] = ("P", g, at)
                p_ready[buf].arrive()
            t += n
            if nx > x0:
                yield from run.wait(o_final[g], no & 1, f"softmax {g} O", no)
                no += 1
                if o_owner[g] != seg:
                    errors.append(f"O of {g} is of {o_owner[g]}, wanted {seg}")
            if split and g == 1:
                other_full.arrive()
                if other_empty:
                    yield from run.wait(other_emptied, nm & 1, "group 1 waits for the join", nm)
                nm += 1
                done(seg, "softmax 1")
                continue
            both = groups == 2 and split
            if both:
                yield from run.wait(other_full, nm & 1, "group 0 waits for group 1", nm)
                nm += 1
            done(seg, f"softmax {g}")
            mine = [g] if nx > x0 else []
            mine += [1] if both and n > 1 else []
            for i in mine:
                o_reading[i].add(w)
                if o_owner[i] != seg:
                    errors.append(f"group {g} reads O {i} of {o_owner[i]} in {seg}")
            yield run.delay(300, 4000)
            for i in mine:
                o_reading[i].discard(w)
                if o_owner[i] != seg:
                    errors.append(f"O {i} changed while group {g} read it in {seg}")
            if both:
                other_emptied.arrive()

    roles = [producer(), issuer(), tensor_core()] + [converter(w) for w in range(WARPS)]
    roles += [softmax_warp(g, w) for g in range(groups) for w in range(WARPS)]
    roles += [scheduler()] + ([watcher()] if watched else [])
    return run.go(roles, {2}, horizon, lambda: not pipe)


def random_segments(rng, groups):
    out = []
    for i in range(rng.randint(1, 14)):
        n = rng.choice([1, 1, 1, 2, 2, 3, 5, 9, 12])
        split = groups == 2 and rng.random() < 0.6
        n0 = n if split or groups == 1 else max(0 if i == 0 else 1, n - rng.randint(0, 2))
        out.append((split, n0, n))
    return out


@pytest.mark.parametrize("groups", [1, 2])
def test_hand_offs(groups):
    for seed in range(150):
        segs = random_segments(random.Random(seed), groups)
        kw = {}
        if seed % 3 == 1:
            kw = dict(softmax=(10, 6000), convert=(10, 6000))
        if seed % 3 == 2:
            kw = dict(convert=(10, 5000), land_in=(5, 50), scales=20)
        errors = chunk(segs, seed, groups=groups, ring_k=3 if groups == 2 else 2, **kw)
        assert not errors, (segs, errors[:3])


@pytest.mark.parametrize("planted", [dict(q_read=False), dict(other_empty=False), dict(infos=2), dict(v_late=1), dict(s_first=False), dict(k_first=False, land_in=(5, 50), scales=20)])
def test_planted_changes_are_found(planted):
    bad = 0
    for seed in range(60):
        segs = [(True, n, n) for n in random.Random(seed).choices([1, 2, 7, 12], k=10)]
        bad += bool(chunk(segs, seed, softmax=(10, 6000), convert=(10, 6000), horizon=5e5, **planted))
    assert bad, planted
