"""How the cache's attention deals its work to CTAs, step by step as the kernels do it (cache8 Line, Place, Segment and
RowParts): every block of every row group is some CTA's, and the second kernel looks for a group's partial results
where the first one put them."""
import random

import pytest

TURN = 4


def line(lens, groups, ctas):
    blocks = [max(1, -(-n // 64)) for n in lens]
    units = sum(blocks) * groups
    turn = 0 if units >> 28 else min(TURN, units // (2 * ctas))
    total = units + turn * len(lens) * groups
    parts = min(ctas, total)
    return blocks, turn, total, parts, lambda i: total * i // parts, lambda u: ((u + 1) * parts - 1) // total


def segments(blocks, groups, turn, u0, u1):
    """A part's (sequence, group, blk0, blk1, first unit of the group), in order."""
    b = before = 0
    u = u0
    while u < u1:
        while u - before >= (blocks[b] + turn) * groups:
            before += (blocks[b] + turn) * groups
            b += 1
        span = blocks[b] + turn
        row = (u - before) // span
        off = u - before - row * span
        nxt = min(u1, u + span - off)
        blk0, blk1 = max(0, off - turn), off + (nxt - u) - turn
        if blk1 <= blk0:
            assert nxt == u1 and u != u0               # only a part's end may lie in a turn
            return
        yield b, row, blk0, blk1, before - turn * b * groups + row * blocks[b]
        u = nxt


CASES = [([300], 8, 304), ([1], 1, 304), ([0, 0, 5], 2, 304), ([131072, 131072], 8, 304), ([5000] * 6, 16, 304),
         ([0, 64, 65, 20000, 3], 3, 152), ([700] * 70, 2, 304), ([64] * 400, 8, 304), ([1] * 3000, 4, 304),
         ([64 * 608], 1, 304), ([64 * 607], 1, 304), ([64 * 2432 + 1], 1, 304)]
rng = random.Random(5)
CASES += [([rng.choice([0, 1, 64, rng.randrange(9000)]) for _ in range(rng.randint(1, 60))], rng.randint(1, 16),
           rng.choice([7, 152, 304])) for _ in range(40)]


@pytest.mark.parametrize("lens,groups,ctas", CASES)
def test_every_block_once_and_partial_results_where_the_join_looks(lens, groups, ctas):
    blocks, turn, total, parts, begin, part_of = line(lens, groups, ctas)
    seen, slots, units = {}, {}, set()
    for i in range(parts):
        mine = list(segments(blocks, groups, turn, begin(i), begin(i + 1)))
        assert mine                                    # no CTA without work
        for k, (b, row, blk0, blk1, unit0) in enumerate(mine):
            assert seen.get((b, row), 0) == blk0       # in order, nothing left out
            seen[b, row] = blk1
            units.update(range(unit0 + blk0, unit0 + blk1))
            if (blk0, blk1) != (0, blocks[b]):
                slot = 2 * i + (k > 0)
                assert slot not in slots
                slots[slot] = (b, row)
    assert seen == {(b, row): n for b, n in enumerate(blocks) for row in range(groups)}
    assert units == set(range(sum(blocks) * groups))
    before = 0
    for b, n in enumerate(blocks):
        for row in range(groups):
            ua = before + turn * b * groups + row * (n + turn)
            c0, c1 = part_of(ua + turn), part_of(ua + turn + n - 1)
            first = 0 if begin(c0) >= ua else 1
            want = [2 * c + (first if c == c0 else 0) for c in range(c0, c1 + 1)] if c0 < c1 else []
            assert [s for s, g in sorted(slots.items()) if g == (b, row)] == want
        before += n * groups


def test_shares_are_even():
    """32 sequences of 2048 to 8192 tokens, 8 heads: blocks and turns together differ by one between CTAs."""
    r = random.Random(1)
    lens = [r.randrange(2048, 8193) for _ in range(32)]
    blocks, turn, total, parts, begin, _ = line(lens, 8, 304)
    assert turn == TURN and {begin(i + 1) - begin(i) for i in range(parts)} <= {total // parts, total // parts + 1}
