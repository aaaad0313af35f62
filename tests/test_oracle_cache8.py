"""Pins of the cache oracle (oracle/cache8.py) on things other than itself."""
import math
import random

import numpy as np
import pytest

import oracle
from oracle import cache8 as oc
from oracle.fp8 import e4m3_decode


def pool(rng, P, H, d):
    codes = [rng.integers(0, 256, (P, H, 64, d)).astype(np.uint8) for _ in range(2)]
    for c in codes:
        c[(c & 0x7F) == 0x7F] = 0x30
    scales = [np.exp2(rng.integers(-6, -3, (P, H))).astype(np.float32) for _ in range(2)]
    return dict(k=codes[0], v=codes[1], k_scale=scales[0], v_scale=scales[1],
                weight=rng.random((P, H, 64)).astype(np.float32))


def test_power_scale_is_the_smallest_that_holds():
    for amax in (448.0, 448.1, 224.0, 1.0, 0.875, 0.8751, 3.4e38, 1e-30, 2.0 ** -133):
        s = oc.power_scale(amax)
        assert math.log2(s) == int(math.log2(s)) and amax <= 448 * s
        assert s == 2.0 ** -126 or amax > 448 * (s / 2)
    assert oc.power_scale(0) == 1.0


def test_append_then_read_back_is_within_half_a_step():
    rng = np.random.default_rng(0)
    c = pool(rng, 6, 2, 16)
    k, v = rng.standard_normal((2, 150, 16)), 30 * rng.standard_normal((2, 150, 16))
    table = np.array([[3, 1, 5], [0, 2, 4]])
    a = oc.append(c, k, v, [0, 100, 150], [0, 70], table)
    for h in range(2):
        K, V, _ = oc.gather(a, table[0], h, 100)
        for x, y in ((K, k), (V, v)):
            s = np.abs(y[h, :100]).max() / 448
            assert (np.abs(x - y[h, :100]) <= 2.0 ** -4 * np.abs(y[h, :100]) + 2 * s * 2.0 ** -10).all()
    # sequence 1: 70 tokens there, so slots 0..5 of block 2 keep their values unless the scale grew
    for h in range(2):
        old, new = (e4m3_decode(z["k"][2, h, :6]) * float(z["k_scale"][2, h]) for z in (c, a))
        ratio = float(a["k_scale"][2, h] / c["k_scale"][2, h])
        assert ratio >= 1 and np.abs(old - new).max() <= float(a["k_scale"][2, h]) * 2.0 ** -10
    assert (a["k"][4] == c["k"][4]).all() and (a["weight"][3] == 0).all()      # untouched block, new tokens' weights


def test_attend_is_the_dense_attention_of_the_values():
    rng = np.random.default_rng(1)
    c = pool(rng, 5, 2, 16)
    table = np.array([[4, 2, 0]])
    q = rng.standard_normal((1, 6, 3, 16))
    n = 150
    o, lse, sums = oc.attend(c, q, table, [n], True, 0.3)
    K, V = np.stack([oc.gather(c, table[0], h, n)[0] for h in range(2)]), np.stack([oc.gather(c, table[0], h, n)[1] for h in range(2)])
    ro, rl = oracle.forward(q, K[None], V[None], True, 0.3)
    assert np.abs(o - ro).max() < 1e-12 and np.abs(lse - rl).max() < 1e-12
    assert np.allclose(sums[0].sum(1), 9)          # three heads x three queries, one each
    w = oc.add_weights(c, sums, table, [n], 0.5)
    assert np.allclose(w[2, 1, 7], 0.5 * c["weight"][2, 1, 7] + sums[0][1, 71])


def test_absent_blocks_take_no_part():
    rng = np.random.default_rng(2)
    c = pool(rng, 4, 1, 16)
    q = rng.standard_normal((1, 1, 1, 16))
    o1, l1, _ = oc.attend(c, q, np.array([[3, -1, 2]]), [160], True, 1.0)
    o2, l2, _ = oc.attend(c, q, np.array([[3, 2]]), [96], True, 1.0)
    assert np.allclose(o1, o2) and np.allclose(l1, l2)
    o3, l3, _ = oc.attend(c, q, np.array([[9]]), [30], True, 1.0)
    assert (o3 == 0).all() and np.isneginf(l3).all()


def test_choose_by_hand_and_by_brute_force():
    assert oc.choose([5, 1, 5, 5, 0, 9], 4, 1) == [0, 2, 3, 5]
    assert oc.choose([5, 1, 5, 5, 0, 9], 3, 1) == [0, 2, 5]
    assert oc.choose([1, float("nan"), 3, 2], 2, 0) == [1, 2]
    assert oc.choose([1, 2], 5, 3) == [0, 1]
    rng = random.Random(3)
    for _ in range(200):
        n = rng.randint(1, 30)
        w = [rng.choice([0.0, 1.0, 2.0, 2.5]) for _ in range(n)]
        keep = rng.randint(1, n)
        recent = rng.randint(0, keep)
        got = oc.choose(w, keep, recent)
        assert len(got) == keep and got == sorted(set(got)) and set(range(n - recent, n)) <= set(got)
        out = [i for i in range(n - recent) if i not in got]
        for i in got:
            if i < n - recent:
                assert all(w[i] > w[j] or (w[i] == w[j] and i < j) for j in out)


def test_evict_moves_values_weights_and_order():
    rng = np.random.default_rng(4)
    c = pool(rng, 8, 2, 16)
    table, to = np.array([[1, 6, 3], [0, 2, 4]]), np.array([[5, 7], [-1, 7]])
    out, new, kept = oc.evict(c, table, [180, 40], 70, 10, to[:, :2])
    assert list(new) == [70, 40] and (kept[1, 0] == list(range(40)) + [-1] * 30).all()
    for h in range(2):
        pick = kept[0, h]
        K0, V0, _ = oc.gather(c, table[0], h, 180)
        K1, _, _ = oc.gather(out, to[0], h, 64)
        assert np.abs(K1 - K0[pick[:64]]).max() <= float(out["k_scale"][5, h]) * 2.0 ** -10
        assert (out["weight"][5, h] == c["weight"][table[0, pick[:64] // 64], h, pick[:64] % 64]).all()


def test_packed_is_one_dense_attention_per_sequence():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((4, 20, 8)), rng.standard_normal((2, 20, 8)), rng.standard_normal((2, 20, 8))
    o, lse = oc.packed(q, k, v, [1, 1, 9, 18], True, 0.5)
    assert np.isnan(o[:, 0]).all() and np.isnan(o[:, 18:]).all()
    for a, e in ((1, 9), (9, 18)):
        for i in range(a, e):
            for h in range(4):
                s = 0.5 * k[h // 2, a:i + 1] @ q[h, i]
                p = np.exp(s) / np.exp(s).sum()
                assert np.allclose(o[h, i], p @ v[h // 2, a:i + 1]) and np.isclose(lse[h, i], np.log(np.exp(s).sum()))


@pytest.mark.parametrize("x,want", [(1.0, 0x38), (-2.0, 0xC0), (np.inf, 0x7E), (-np.inf, 0xFE), (np.nan, 0x7F)])
def test_encode_specials(x, want):
    assert oc.encode([x], 1.0)[0] == want
