"""Attention of chunks of new tokens over the 8-bit cache, on the GPU against 64 bits (the cache's values as oracle/cache8.py
reads them).

Bound, per element, with A = scale max_j sum_c |q_c k_jc| of the row, n keys:
  logits   (2 d + 8) 2^-23 A: two terms of d exact products added in fp32 by the tensor core (2^-23 each, truncated), scales; and
           what the terms of Q leave of values below 2^-9 of the row's largest, 2^-17 of it each;
  P        2^-11 (f16), 2^-20 (ex2, its argument's sum); as a ratio to l twice the logits' error; 2^-31 of the row's
           largest P times its scale, times the code;
  sums     n 2^-23 for O and for l;
  result   2^-8 |O| (bf16).
"""
import os

import numpy as np
import pytest
import torch

from oracle import cache8 as oc
from oracle import rope as orope
from oracle.fp8 import e4m3_decode
from test_cache8_gpu import DEV, bf16, f64, ints, make, to_gpu

pytestmark = pytest.mark.gpu


def check(c, q, table, news, lens, causal, scale, o, lse, rows=None):
    """q [Hq, T, d]; every row of every chunk, or `rows` of each."""
    qd, o, lse = f64(q), f64(o), f64(lse)
    Hq, _, d = qd.shape
    Hkv, P = c["k"].shape[1], c["k"].shape[0]
    at = 0
    for b, n in enumerate(news):
        held = min(max(int(lens[b]), 0), table.shape[1] * 64)
        for h in range(Hkv):
            K, V, pos = oc.gather(c, table[b], h, held)
            page = np.asarray(table[b])[pos // 64]
            vs = c["v_scale"][page, h].astype(np.float64)
            codes = np.abs(e4m3_decode(c["v"][page, h, pos % 64]))
            pick = range(n) if rows is None or n <= rows else sorted({0, 1, n - 1, n - 2, *np.random.default_rng(b).integers(0, n, rows)})
            for r in pick:
                m = int((pos <= r + held - n).sum()) if causal else len(pos)
                for j in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                    x, got, gl = qd[j, at + r], o[j, at + r], lse[j, at + r]
                    if m == 0:
                        assert (got == 0).all() and np.isneginf(gl), (b, j, r)
                        continue
                    s = scale * (K[:m] @ x)
                    top = s.max()
                    p = np.exp(s - top)
                    l = p.sum()
                    p /= l
                    rl, ro = top + np.log(l), p @ V[:m]
                    A = scale * (np.abs(K[:m]) @ np.abs(x)).max()
                    qmax = np.abs(x).max()
                    small = (np.abs(x) < 2.0 ** -9 * qmax) & (x != 0)
                    ds = (2 * d + 8) * 2.0 ** -23 * A + scale * 2.0 ** -17 * qmax * np.abs(K[:m])[:, small].sum(1).max()
                    rel = 2.0 ** -11 + 2.0 ** -20 + 2 * ds + 2 * m * 2.0 ** -23
                    tol = 2.0 ** -8 * np.abs(ro) + rel * (p @ np.abs(V[:m])) + 2.0 ** -31 * (p * vs[:m]).max() * codes[:m].sum(0) + 1e-30
                    err = np.abs(got - ro)
                    assert (err <= tol).all(), (b, j, r, float((err / tol).max()))
                    ltol = ds + 2.0 ** -20 + m * 2.0 ** -23 + abs(rl) * 2.0 ** -22
                    assert abs(gl - rl) <= ltol, (b, j, r, gl, rl)
        at += n


def run(fa, c, q, table, news, lens, causal=True, scale=None, **kw):
    cu = ints(np.concatenate([[0], np.cumsum(news)]))
    out = fa.fwd_cache8_packed(q, to_gpu(fa, c), cu, ints(table), ints(lens), causal=causal, scale=scale, **kw)
    fa.check_device_status()
    return out


CASES = [
    # new tokens and cached ones before them per sequence, Hq, Hkv, d, causal
    ([1], [0], 1, 1, 128, True),                                    # one token, nothing before it
    ([1, 1, 1], [0, 63, 64], 8, 2, 128, True),
    ([5], [300], 4, 1, 64, True),                                   # one row tile, three key tiles
    ([16], [496], 8, 1, 128, True),                                 # exactly one row tile of 128, four key tiles
    ([17], [600], 8, 1, 128, True),                                 # one token in the second row tile
    ([33, 0, 7, 1, 64], [0, 9, 1000, 127, 128], 8, 2, 128, True),
    ([300], [0], 2, 2, 128, True),                                  # no groups: 256 tokens in an item
    ([129, 256, 257], [1, 0, 70], 3, 1, 64, True),                  # 42 tokens per row tile, two rows of it without one
    ([40, 3], [100, 300], 14, 2, 80, True),                         # groups of seven
    ([40, 3], [100, 300], 14, 2, 48, False),
    ([9, 50], [190, 260], 4, 4, 16, True),                          # the narrowest
    ([3, 30], [40, 5], 128, 1, 112, True),                          # a group of 128: a token per row tile
    ([5, 20], [200, 1], 100, 1, 96, True),
    ([70, 1], [333, 200], 4, 2, 256, True),                         # wide
    ([130, 65], [0, 500], 6, 3, 192, True),
    ([33, 2, 128], [77, 640, 128], 8, 1, 144, False),
    ([700], [900], 8, 8, 128, True),
]


@pytest.mark.parametrize("news,past,Hq,Hkv,d,causal", CASES)
def test_chunks(fa, news, past, Hq, Hkv, d, causal):
    lens = [a + b for a, b in zip(news, past)]
    c, table = make(sum(lens) + d + Hq, lens, Hkv, d, spread=2)
    T = sum(news)
    q = bf16(np.random.default_rng(d), T, Hq, d).to(DEV).transpose(0, 1)       # a projection's layout
    o, lse = run(fa, c, q, table, news, lens, causal)
    assert o.stride() == q.stride() or T == 1 or Hq == 1
    check(c, q, table, news, lens, causal, d ** -0.5, o, lse, rows=24)
    # head by head in memory: the same bits
    o2, lse2 = run(fa, c, q.contiguous(), table, news, lens, causal)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_more_new_tokens_than_are_held_and_absent_blocks(fa):
    """Rows that see no key give 0 and -inf; blocks outside the pool are absent; lengths outside the table are taken
    within."""
    news, lens = [30, 300, 20, 4], [10, 0, 500, 10 ** 6]
    c, table = make(3, [500] * 4, 2, 128)
    table[2, 0], table[2, 3], table[3, 1], table[3, 7] = -1, 10 ** 6, -7, len(c["k"])
    q = bf16(np.random.default_rng(1), 8, sum(news), 128).to(DEV)
    for x in ("k", "v"):                                              # values where the longest length reaches
        c[x][table[3, 8]] = 0x30
    for causal in (True, False):
        o, lse = run(fa, c, q, table, news, lens, causal)
        check(c, q, table, news, lens, causal, 128 ** -0.5, o, lse, rows=40)


@pytest.mark.parametrize("d", [128, 256])
def test_many_parts_and_their_join(fa, d):
    """Long pasts: one item over many CTAs, several items over neighbouring ones, both row tiles; the same bits twice."""
    for news, past, Hq, Hkv in (([3], [40000], 4, 2), ([20, 40, 1], [9000, 12345, 777], 16, 2), ([1] * 9 + [200], [900 + 211 * i for i in range(10)], 8, 4)):
        lens = [a + b for a, b in zip(news, past)]
        c, table = make(sum(lens), lens, Hkv, d)
        q = bf16(np.random.default_rng(d), Hq, sum(news), d).to(DEV)
        o, lse = run(fa, c, q, table, news, lens)
        check(c, q, table, news, lens, True, d ** -0.5, o, lse, rows=5)
        again = run(fa, c, q, table, news, lens)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("po2", [True, False])
def test_scales_far_apart(fa, d, po2):
    """V scales 2^40 apart between blocks: P times its scale stays within f16, small ones keep their digits."""
    news, past = [50, 2], [700, 1500]
    lens = [a + b for a, b in zip(news, past)]
    c, table = make(11, lens, 2, d, spread=20, po2=po2)
    q = (bf16(np.random.default_rng(2), 8, sum(news), d) * 3).to(DEV)
    o, lse = run(fa, c, q, table, news, lens)
    check(c, q, table, news, lens, True, d ** -0.5, o, lse, rows=12)


def test_zero_scales(fa):
    """A K scale of 0 makes equal logits, a V scale of 0 zeros; all of them 0 as well."""
    news, past = [20, 3], [400, 130]
    lens = [a + b for a, b in zip(news, past)]
    c, table = make(13, lens, 2, 64)
    c["k_scale"][table[0, ::2]] = 0
    c["v_scale"][table[0, 1::2]] = 0
    c["v_scale"][table[1], 1] = 0
    c["k_scale"][table[1], 0] = 0
    q = bf16(np.random.default_rng(2), 4, sum(news), 64).to(DEV)
    o, lse = run(fa, c, q, table, news, lens)
    check(c, q, table, news, lens, True, 0.125, o, lse)


def test_growing_logits_and_tiny_queries(fa):
    """Keys that grow along the sequence raise the references all the way; queries with values far below their largest,
    zero queries, subnormal ones."""
    news, past = [70], [3000]
    lens = [3070]
    c, table = make(17, lens, 1, 128, spread=0)
    for i in range(48):
        c["k_scale"][table[0, i]] = 2.0 ** (-9 + i / 8)
    q = bf16(np.random.default_rng(5), 2, 70, 128)
    q[0, 3] = 0
    q[0, 4] *= 2.0 ** -130
    q[1, 5, ::2] *= 2.0 ** -10
    q[1, 6, 1:] *= 2.0 ** -14
    q[1, 7] *= 2.0 ** 20
    q = q.to(torch.bfloat16).to(DEV)
    o, lse = run(fa, c, q, table, news, lens, scale=0.02)
    check(c, q, table, news, lens, True, 0.02, o, lse)


def test_nan_and_infinity(fa):
    """A query row with an infinity or NaN becomes NaN, the others stay; a NaN key makes NaN of the rows that see it; codes of
    slots that hold no token are never looked at (they are NaN in every test here)."""
    news, past = [40], [200]
    lens = [240]
    c, table = make(19, lens, 1, 64)
    q = bf16(np.random.default_rng(5), 2, 40, 64)
    q[0, 3, 5], q[1, 9, 60] = float("nan"), float("inf")
    q = q.to(DEV)
    o, lse = run(fa, c, q, table, news, lens)
    bad = torch.isnan(lse).cpu().numpy()
    assert bad[0, 3] and bad[1, 9] and bad.sum() == 2 and torch.isnan(o).any(-1).cpu().numpy().sum() == 2
    c["k"][table[0, 3], 0, 220 - 192, 7] = 0x7F                       # key 220: rows from 20 on
    o, lse = run(fa, c, bf16(np.random.default_rng(6), 2, 40, 64).to(DEV), table, news, lens)
    bad = torch.isnan(lse).cpu().numpy()
    assert bad[:, 20:].all() and not bad[:, :20].any()


def test_rows_of_no_sequence_and_given_outputs(fa):
    news, lens = [9, 20], [100, 333]
    c, table = make(23, lens, 2, 128)
    T = 60
    wide = bf16(np.random.default_rng(3), T, 12, 128).to(DEV)
    q = wide[:, 2:10].transpose(0, 1)                                  # heads cut out of a wider projection
    cu = ints([5, 14, 34])
    out, lse = torch.full((T, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV).transpose(0, 1), torch.full((8, T), 5.0, device=DEV)
    g = to_gpu(fa, c)
    n = fa.load().fa_fwd_cache8_packed_workspace_bytes(2, T, 8, 2, 128, table.shape[1])
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    fa.fwd_cache8_packed(q, g, cu, ints(table), ints(lens), out=out, lse=lse, workspace=ws)
    fa.check_device_status()
    check(c, q[:, 5:34], table, news, lens, True, 128 ** -0.5, out[:, 5:34], lse[:, 5:34])
    for x in (out[:, :5], out[:, 34:]):
        assert (x == 7).all()
    assert (lse[:, :5] == 5).all() and (lse[:, 34:] == 5).all()
    with pytest.raises(fa.FAError, match="WORKSPACE"):
        fa.fwd_cache8_packed(q, g, cu, ints(table), ints(lens), workspace=ws[256:])


def test_agrees_with_the_single_tokens_call(fa):
    lens = [700, 65, 3000]
    c, table = make(29, lens, 4, 128)
    q = bf16(np.random.default_rng(7), 3, 16, 2, 128).to(DEV)
    g = to_gpu(fa, c)
    a, la = fa.fwd_cache8(q, g, ints(table), ints(lens))
    packed = q.permute(1, 0, 2, 3).reshape(16, 6, 128)
    b, lb = fa.fwd_cache8_packed(packed, g, ints([0, 2, 4, 6]), ints(table), ints(lens))
    fa.check_device_status()
    b, lb = b.view(16, 3, 2, 128).transpose(0, 1), lb.view(16, 3, 2).transpose(0, 1)
    assert float((a.float() - b.float()).abs().max()) <= 2.0 ** -7 * float(a.float().abs().max())
    assert float((la - lb).abs().max()) <= 2.0 ** -16


def test_many_sequences(fa):
    """Hundreds of sequences, most of one token, some of none."""
    rng = np.random.default_rng(31)
    news = [int(x) for x in rng.choice([0, 1, 1, 1, 2, 9], 700)]
    lens = [n + int(rng.integers(0, 150)) for n in news]
    c, table = make(31, lens, 1, 64)
    q = bf16(rng, 4, sum(news), 64).to(DEV)
    o, lse = run(fa, c, q, table, news, lens)
    check(c, q, table, news, lens, True, 0.125, o, lse)


def test_graph_streams_and_workspaces(fa):
    """A captured call replays on what the buffers hold then; calls on two streams with a workspace each."""
    news, lens = [30, 1], [2000, 900]
    c, table = make(37, lens, 2, 128)
    g = to_gpu(fa, c)
    q = bf16(np.random.default_rng(3), 8, 31, 128).to(DEV)
    cu, tb, ln = ints([0, 30, 31]), ints(table), ints(lens)
    want = [t.clone() for t in fa.fwd_cache8_packed(q, g, cu, tb, ln)]
    o, lse = torch.zeros_like(q), torch.zeros(8, 31, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.fwd_cache8_packed(q, g, cu, tb, ln, out=o, lse=lse)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    ln.copy_(ints([1500, 400]))
    graph.replay()
    other = fa.fwd_cache8_packed(q, g, cu, tb, ints([1500, 400]))
    torch.cuda.synchronize()
    assert torch.equal(o, other[0]) and torch.equal(lse, other[1]) and not torch.equal(o, want[0])
    n = fa.load().fa_fwd_cache8_packed_workspace_bytes(2, 31, 8, 2, 128, table.shape[1])
    streams, results = [torch.cuda.Stream() for _ in range(2)], []
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in range(2)]
    ln.copy_(ints(lens))
    torch.cuda.synchronize()
    for s, w in zip(streams, ws):
        with torch.cuda.stream(s):
            results.append([fa.fwd_cache8_packed(q, g, cu, tb, ln, workspace=w) for _ in range(4)])
    torch.cuda.synchronize()
    for r in results:
        for a, b in r:
            assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_the_same_bits_many_times(fa):
    """Hand-offs under many timings: short items one behind the other, long ones over several CTAs, wide heads, with nothing
    between the calls."""
    rng = np.random.default_rng(43)
    for d, news, past in ((128, [40] * 30 + [300, 1, 1, 1], [0, 90, 200] * 10 + [2500, 5000, 10, 4000]), (64, [700, 33, 1], [3000, 50, 9000]),
                          (256, [130, 20, 1, 64], [100, 2000, 5000, 0])):
        lens = [a + b for a, b in zip(news, past)]
        c, table = make(43 + d, lens, 4, d)
        g, q = to_gpu(fa, c), bf16(rng, 16, sum(news), d).to(DEV)
        cu, tb, ln = ints(np.concatenate([[0], np.cumsum(news)])), ints(table), ints(lens)
        o, lse = fa.fwd_cache8_packed(q, g, cu, tb, ln)
        bad = torch.zeros((), dtype=torch.int64, device=DEV)
        for _ in range(150):
            o2, l2 = fa.fwd_cache8_packed(q, g, cu, tb, ln)
            bad += (o2 != o).any() | (l2 != lse).any()
        fa.check_device_status()
        assert int(bad) == 0
        check(c, q, table, news, lens, True, d ** -0.5, o, lse, rows=2)


def test_stall_is_reported(fa):
    news, lens = [30], [700]
    c, table = make(41, lens, 1, 128)
    q = bf16(np.random.default_rng(3), 4, 30, 128).to(DEV)
    os.environ["FA_TEST_STALL"] = "1"
    try:
        fa.fwd_cache8_packed(q, to_gpu(fa, c), ints([0, 30]), ints(table), ints(lens))
        with pytest.raises(fa.FAError, match="TIMEOUT"):
            fa.check_device_status()
    finally:
        del os.environ["FA_TEST_STALL"]
    o, lse = run(fa, c, q, table, news, lens)
    check(c, q, table, news, lens, True, 128 ** -0.5, o, lse)


@pytest.mark.parametrize("d", [64, 256])
def test_a_prompt_in_pieces(fa, d):
    """As served: each step rotates Q, appends the piece's rotated K and V and attends; against attention of the whole in 64
    bits on the values that the cache held at each step."""
    Hq, Hkv, B = 4, 2, 2
    gen = torch.Generator().manual_seed(d)
    freqs = [1e4 ** (-i / (d // 2)) for i in range(d // 2)]
    plan = fa.new_rope(freqs)
    pieces = [[70, 1], [1, 130], [200, 0], [1, 1]]
    cache = fa.new_cache8(20, Hkv, d)
    table = np.random.default_rng(0).permutation(20)[:16].reshape(2, 8).astype(np.int32)
    held = [0, 0]
    for news in pieces:
        T = sum(news)
        qkv = torch.randn(T, Hq + 2 * Hkv, d, generator=gen).to(torch.bfloat16).to(DEV)
        q, k, v = (x.transpose(0, 1) for x in qkv.split([Hq, Hkv, Hkv], 1))
        at = np.concatenate([np.arange(h, h + n) for h, n in zip(held, news)])
        cu = ints(np.concatenate([[0], np.cumsum(news)]))
        turned, _ = fa.rope(q, None, plan, ints(at))
        fa.cache8_append(cache, k, v, cu, ints(table), ints(held), rope=plan)
        held = [h + n for h, n in zip(held, news)]
        o, lse = fa.fwd_cache8_packed(turned, cache, cu, ints(table), ints(held))
        fa.check_device_status()
        want = orope.rotate(f64(q), freqs, [0] * len(freqs), at[None])
        assert np.abs(f64(turned) - want).max() <= 2.0 ** -7 * np.abs(want).max()
        c = {x: getattr(cache, x).cpu().numpy() for x in ("k", "v", "k_scale", "v_scale")}
        check(c, turned, table, news, held, True, d ** -0.5, o, lse, rows=20)
