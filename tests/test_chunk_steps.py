"""Host models of two parts of the chunks' attention (csrc/fa_cache8_chunk.cu) that the model of its hand-offs
(tests/test_chunk_schedule.py) walks through one step at a time or leaves out, on the CPU.

The issuing loop of two groups runs a segment's middle steps two at a time, with descriptors and parities of its own: it
gives out the same products, waits and commits, in the same order, as one step at a time.

With one group (wide heads) S of the next tile is out before a tile's P V, so a softmax warp that rescales O waits for the V
stage that the product before read last: as coroutines, no product runs while O is read and written.

Planted changes show what each piece guards.
"""
import random

import pytest

from test_serving_schedule import Run
from test_wide_schedule import Barrier

RING_K, STEP_K, STEP_V = 3, 16384 >> 4, 32768 >> 4
KD0, VD0 = 0x10000 | 4096, 0x4000000 | 8192 + 1024           # descriptors' lower halves: an offset field over an address


def one_by_one(segments):
    """What the issuer does, step by step: ("wait", group, parity), ("PV", group, V's descriptor, accumulates),
    ("S", group, K's descriptor, Q's rows), ("O", group), ("Q",)."""
    ops, tile, count = [], 0, [0, 0]
    for split, n0, n in segments:
        for i in range(-2, n if split else 2 * n):
            g, j = i & 1, i if split else i >> 1
            mine, nxt, last = (n if split or g else n0), (i + 2 if split else j + 1), split or g
            if j >= mine:
                continue
            if i >= 0:
                ops.append(("wait", g, count[g] & 1))
                count[g] += 1
                ops.append(("PV", g, VD0 + ((tile + j) & 1) * STEP_V, i > 1 if split else j > 0))
            if nxt < mine:
                ops.append(("S", g, KD0 + (tile + nxt) % RING_K * STEP_K, 1 if g and not split else 0))
            elif i >= 0:
                ops.append(("O", g))
            if last and nxt + 1 == n:
                ops.append(("Q",))
        tile += n
    return ops


def as_written(segments, *, more=0, k_ahead=0, carry=True, resume=0, turn=True):
    """The same as the kernel's code goes about it."""
    ops, tile, np = [], 0, 0
    for split, n0, n in segments:
        i, end = -2, n if split else 2 * n
        while i < end:
            if i == 0:
                pairs = (int((n - 3) / 2) if split else n0 - 2) + more       # (rounded towards 0)
                va, vb = VD0 + (tile & 1) * STEP_V, VD0 + ((tile + split) & 1) * STEP_V
                turn_v = 0 if split or not turn else VD0 ^ (VD0 + STEP_V)
                ka = (tile + (2 if split else 1) + k_ahead) % RING_K
                kb = (ka + 1) % RING_K if split else ka
                kda, kdb = KD0 + ka * STEP_K, KD0 + kb * STEP_K

                def step(kd):
                    kd += STEP_K
                    return KD0 if kd == KD0 + RING_K * STEP_K else kd
                par, par1 = np & 1, np >> 1
                for j in range(pairs):
                    ops.append(("wait", 0, par))
                    ops.append(("PV", 0, va, j > 0))
                    ops.append(("S", 0, kda, 0))
                    ops.append(("wait", 1, par1))
                    ops.append(("PV", 1, vb, j > 0))
                    ops.append(("S", 1, kdb, 0 if split else 1))
                    par, par1 = par ^ 1, par1 ^ 1
                    va, vb = va ^ turn_v, vb ^ turn_v
                    kda = step(kdb)
                    kdb = step(kda) if split else kda
                if pairs > 0:
                    if carry:
                        np = par | par1 << 1
                    i = 2 * pairs + resume
            g, j = i & 1, i if split else i >> 1
            mine, nxt, last = (n if split or g else n0), (i + 2 if split else j + 1), split or g
            if j < mine:
                if i >= 0:
                    ops.append(("wait", g, np >> g & 1))
                    np ^= 1 << g
                    ops.append(("PV", g, VD0 + ((tile + j) & 1) * STEP_V, i > 1 if split else j > 0))
                if nxt < mine:
                    ops.append(("S", g, KD0 + (tile + nxt) % RING_K * STEP_K, 1 if g and not split else 0))
                elif i >= 0:
                    ops.append(("O", g))
                if last and nxt + 1 == n:
                    ops.append(("Q",))
            i += 1
        tile += n
    return ops


def all_segments():
    """(split, group 0's tiles, tiles): group 0 has at most one fewer, none among them."""
    for n in range(1, 20):
        yield True, n, n
        yield False, n, n
        yield False, n - 1, n


def chains():
    segs = list(all_segments())
    for first in segs:
        for then in segs:
            yield [first, then]
    rng = random.Random(3)
    for _ in range(500):
        yield rng.choices(segs, k=9)


def test_two_at_a_time_is_the_same_as_one_by_one():
    for chain in chains():
        assert as_written(chain) == one_by_one(chain), chain


@pytest.mark.parametrize("planted", [dict(more=1), dict(k_ahead=1), dict(carry=False), dict(resume=1), dict(turn=False)])
def test_planted_changes_to_the_steps_are_found(planted):
    assert any(as_written(chain, **planted) != one_by_one(chain) for chain in chains()), planted


def test_a_group_s_product_is_issued_before_its_next_scores():
    """Why two groups rescale O without a wait: S of a group's tile, which the softmax has waited for, is behind the group's
    product of the tile before."""
    for chain in chains():
        given, done = [0, 0], [0, 0]                         # S and P V of each group
        for op in as_written(chain):
            if op[0] == "S":
                assert given[op[1]] == done[op[1]]
                given[op[1]] += 1
            elif op[0] == "PV":
                done[op[1]] += 1
                assert given[op[1]] == done[op[1]]


# ------------------------------------------------------------------ wide heads: O's rescale
def wide(segments, seed, *, waits=True, phase=0, softmax=(300, 1500), convert=(200, 900), grows=0.5, horizon=2e6):
    """segments: key tiles of each. Two V stages to a tile in a ring of two, S in two buffers, four softmax warps; K and Q
    are there."""
    WARPS, PER, RING = 4, 2, 2
    run = Run(seed)
    errors, rng = run.errors, random.Random(seed)
    v_full, v_empty = [Barrier(1) for _ in range(RING)], [Barrier(1) for _ in range(RING)]
    s_full, p_ready, o_final = [Barrier(1), Barrier(1)], [Barrier(WARPS), Barrier(WARPS)], Barrier(1)
    pipe, busy, using, given = [], [None], set(), [0]

    def tensor_core():
        while True:
            while not pipe:
                yield ("wait", lambda: bool(pipe))
            op = pipe.pop(0)
            if op[0] == "commit":
                op[1].arrive()
            elif op[0] == "S":
                yield run.delay(400, 600)
            else:
                if using:
                    errors.append(f"product {op[1]} began while O was rescaled by {using}")
                busy[0] = op[1]
                yield run.delay(200, 400)
                if using:
                    errors.append(f"product {op[1]} ended while O was rescaled by {using}")
                busy[0] = None

    def converters():
        for c in range(PER * sum(segments)):
            yield from run.wait(v_empty[c % RING], ((c // RING) & 1) ^ 1, f"V empty {c}", c // RING - 1)
            yield run.delay(*convert)
            v_full[c % RING].arrive()

    def issuer():
        t = 0
        for n in segments:
            for j in range(-1, n):
                if j + 1 < n:
                    pipe.append(("S", t + j + 1))
                    pipe.append(("commit", s_full[(t + j + 1) & 1]))
                    yield run.delay(20, 300)
                if j < 0:
                    continue
                yield from run.wait(p_ready[(t + j) & 1], ((t + j) >> 1) & 1, f"P {t + j}", (t + j) >> 1)
                for x in range(PER):
                    c = (t + j) * PER + x
                    yield from run.wait(v_full[c % RING], (c // RING) & 1, f"V {c}", c // RING)
                    pipe.append(("PV", c))
                    given[0] += 1
                    pipe.append(("commit", v_empty[c % RING]))
                    yield run.delay(20, 300)
            pipe.append(("commit", o_final))
            t += n

    def softmax_warp(w):
        t = 0
        for seg, n in enumerate(segments):
            for at in range(t, t + n):
                yield from run.wait(s_full[at & 1], at >> 1 & 1, f"softmax S {at}", at >> 1)
                yield run.delay(*softmax)
                if at > t and rng.random() < grows:
                    c = at * PER - 1
                    if waits:
                        yield from run.wait(v_empty[c % RING], ((c // RING) & 1) ^ phase, f"rescale {at}", c // RING)
                    if given[0] != PER * at:
                        errors.append(f"O was rescaled for tile {at} with {given[0]} products given out")
                    if busy[0] is not None:
                        errors.append(f"O was rescaled for tile {at} during product {busy[0]}")
                    using.add((w, at))
                    yield run.delay(100, 800)
                    using.discard((w, at))
                p_ready[at & 1].arrive()
            yield from run.wait(o_final, seg & 1, "O final", seg)
            t += n

    roles = [tensor_core(), converters(), issuer()] + [softmax_warp(w) for w in range(WARPS)]
    return run.go(roles, {0}, horizon, lambda: not pipe)


def test_wide_heads_rescale_between_products():
    for seed in range(120):
        segs = random.Random(seed).choices([1, 1, 2, 3, 7, 12], k=8)
        kw = [dict(), dict(softmax=(10, 6000), convert=(10, 6000)), dict(softmax=(10, 60), convert=(10, 60), grows=0.9)][seed % 3]
        errors = wide(segs, seed, **kw)
        assert not errors, (segs, errors[:3])


@pytest.mark.parametrize("planted", [dict(waits=False), dict(phase=1)])
def test_planted_changes_to_the_rescale_are_found(planted):
    assert any(wide([1, 7, 12, 3], seed, softmax=(10, 3000), convert=(10, 3000), horizon=5e5, **planted) for seed in range(30)), planted
