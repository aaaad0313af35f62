"""Which items the packed forward's CTAs take, step by step as its scheduler warp does it (csrc/fa_fwd_packed.cu, Finder
and the line's rounds): every (tile, sequence, head) is some CTA's exactly once, those with the most key tiles first (CPU)."""
import random

import pytest


class Finder:
    """r only grows: the index w only falls, and C(w + 1), C(w) are kept between calls, and within an index where the last
    look-up ended."""

    def __init__(self, lens, unit):
        self.n = [-(-x // unit) for x in lens]
        self.w = max(self.n, default=0)
        self.above = self.upto = 0
        self.at = self.before = 0
        self.searches = self.steps = 0

    def count(self, x):
        return sum(max(0, n - x) for n in self.n)

    def find(self, r):
        if r >= self.upto:
            self.searches += 1
            lo, hi = 0, self.w
            if self.w == 0 or self.count(0) <= r:
                return None
            while hi - lo > 1:
                mid = (lo + hi) >> 1
                if self.count(mid) > r:
                    lo = mid
                else:
                    hi = mid
            self.w, self.above, self.upto = lo, self.count(lo + 1), self.count(lo)
            self.at = self.before = 0
        k = r - self.above - self.before
        for s0 in range(self.at, len(self.n), 32):          # a warp's 32 sequences at a time
            self.steps += 1
            hit = [s for s in range(s0, min(s0 + 32, len(self.n))) if self.n[s] > self.w]
            if k < len(hit):
                self.at = s0
                return self.w, hit[k]
            k -= len(hit)
            self.before += len(hit)
        return None


def items(lens, Hq, Hkv, sms):
    """Per CTA its (tile or pair, sequence, head or pair) in order, as the launch and the scheduler deal them."""
    two_heads = Hq // Hkv % 2 == 0
    unit, inner = (128, Hq // 2) if two_heads else (256, Hq)
    most = (sum(lens) + (unit - 1) * len(lens)) // unit * inner
    grid = min(most, sms)
    out = []
    for c in range(grid):
        finder, mine, n = Finder(lens, unit), [], 0
        while True:
            at = n * grid + (grid - 1 - c if n & 1 else c)
            r, n = at // inner, n + 1
            got = finder.find(r)
            if got is None:
                break
            mine.append((*got, at - r * inner))
        out.append(mine)
    return out, unit, inner


rng = random.Random(9)
CASES = [([1], 1, 1, 152), ([256], 4, 4, 152), ([257, 1, 0, 900], 8, 1, 152), ([0, 0, 5], 3, 3, 152), ([0, 0], 2, 1, 152),
         ([2000] * 3, 6, 2, 7), ([256 * 7, 3, 512, 511, 513], 2, 1, 5), ([2] * 300 + [130, 0, 700] + [1, 0] * 100 + [290], 2, 1, 152),
         ([5, 0, 1] * 120 + [385], 3, 3, 11), ([16384], 64, 8, 152)]
CASES += [([rng.choice([0, 1, 127, 128, 129, 256, rng.randrange(3000)]) for _ in range(rng.randint(1, 90))],
           *rng.choice([(1, 1), (2, 1), (3, 1), (8, 2), (9, 3)]), rng.choice([1, 3, 64, 152])) for _ in range(30)]


@pytest.mark.parametrize("lens,Hq,Hkv,sms", CASES)
def test_every_item_is_one_ctas(lens, Hq, Hkv, sms):
    parts, unit, inner = items(lens, Hq, Hkv, sms)
    want = sorted((w, s, h) for s, n in enumerate(lens) for w in range(-(-n // unit)) for h in range(inner))
    assert sorted(x for p in parts for x in p) == want
    for p in parts:
        assert [w for w, _, _ in p] == sorted((w for w, _, _ in p), reverse=True)
    assert {len(p) for p in parts} <= {len(want) // max(1, len(parts)), -(-len(want) // max(1, len(parts)))}


def test_the_index_is_searched_once_per_change():
    f = Finder([1000] * 40, 128)
    assert [f.find(r)[0] for r in range(320)] == [w for w in range(7, -1, -1) for _ in range(40)] and f.searches == 8
    assert f.find(320) is None


def test_the_look_up_goes_on_where_it_ended():
    """The steps of a CTA's look-ups: the sequences once per index, and one for each item."""
    lens = [70] * 5000 + [0, 300] * 500
    f = Finder(lens, 128)
    total = sum(-(-n // 128) for n in lens)
    for r in range(0, total, 7):
        f.find(r)
    assert f.steps <= f.searches * -(-len(lens) // 32) + -(-total // 7)
