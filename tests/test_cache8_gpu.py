"""The 8-bit cache on the GPU against the double-precision oracle (oracle/cache8.py): append and eviction bit for
bit, the attention and its weights within bounds derived from the formats.

Attention bound, per element, with A = scale max_j sum_c |q_c k_jc| of the row, n keys:
  logits   (d + 8) 2^-23 A: d exact products added in fp32 by the tensor core (2^-23 each, truncated), scales;
  P        2^-12 (three e4m3 terms), below 2^-11, 2^-20 (ex2, its argument's sum); as a ratio to l twice the logits' error;
  sums     n 2^-23 for O and for l;
  result   2^-8 |O| (bf16).
P is also off by 2^-25 of the row's largest: no more than the other half of 2^-11 where the keys that matter are few (a
long tail of small ones has a test of its own); n 2^-31 of the largest term on top.
"""
import threading

import numpy as np
import pytest
import torch

from oracle import cache8 as oc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
NAN = 0x7F


def make(seed, lens, Hkv, d, spread=3, spare=1, po2=True):
    """A pool in shuffled blocks with NaN codes in every slot that holds no token, and the sequences' table."""
    rng = np.random.default_rng(seed)
    need = [-(-n // 64) for n in lens]
    width = max(max(need), 1) + spare
    P = len(lens) * width + 2
    table = rng.permutation(P)[: len(lens) * width].reshape(len(lens), width).astype(np.int32)
    c = {x: np.full((P, Hkv, 64, d), NAN, np.uint8) for x in ("k", "v")}
    sc = {x: np.exp2(rng.integers(-6 - spread, -5 + spread, (P, Hkv))).astype(np.float32) for x in ("k_scale", "v_scale")}
    if spread > 5:                                     # logits stay moderate whatever V's scales
        sc["k_scale"] = np.exp2(rng.integers(-8, -5, (P, Hkv))).astype(np.float32)
    if not po2:
        sc = {x: (s * (1 + rng.random(s.shape))).astype(np.float32) for x, s in sc.items()}
    w = np.full((P, Hkv, 64), np.nan, np.float32)
    for b, n in enumerate(lens):
        for pos in range(0, n, 64):
            m = min(64, n - pos)
            page = table[b, pos // 64]
            for x in ("k", "v"):
                y = torch.from_numpy(rng.standard_normal((Hkv, m, d)).astype(np.float32) * 48).clamp_(-448, 448)
                c[x][page, :, :m] = y.to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            w[page, :, :m] = rng.random((Hkv, m)).astype(np.float32) ** 4
    return dict(c, **sc, weight=w), table


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


def to_gpu(fa, c):
    return fa.Cache8(**{n: torch.from_numpy(x.copy()).to(DEV) for n, x in c.items()})


def ints(x):
    return torch.as_tensor(np.asarray(x, np.int32), device=DEV)


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def check_attention(c, q, table, lens, causal, scale, o, lse, sums, got_w=None, decay=None):
    qd = f64(q)
    ro, rl, rs = oc.attend(c, qd, table, lens, causal, scale)
    B, Hq, Nq, d = qd.shape
    Hkv = c["k"].shape[1]
    o, lse = f64(o), f64(lse)
    want_w = oc.add_weights(c, rs, table, lens, decay) if got_w is not None else None
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * 64)
        wtol = np.zeros((Hkv, n))
        for h in range(Hkv):
            K, V, pos = oc.gather(c, table[b], h, n)
            for j in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                for r in range(Nq):
                    seen = pos <= r + n - Nq if causal else np.ones(len(pos), bool)
                    if not seen.any():
                        assert (o[b, j, r] == 0).all() and np.isneginf(lse[b, j, r])
                        continue
                    A = scale * (np.abs(qd[b, j, r]) @ np.abs(K[seen]).T).max()
                    ds = (d + 8) * 2.0 ** -23 * A
                    p = np.exp(scale * (K[seen] @ qd[b, j, r]) - rl[b, j, r])
                    rel = 2.0 ** -11 + 2.0 ** -20 + 2 * ds + 2 * len(p) * 2.0 ** -23
                    tol = 2.0 ** -8 * np.abs(ro[b, j, r]) + rel * (p @ np.abs(V[seen])) + len(p) * 2.0 ** -22 * 2.0 ** -9 * np.abs(V[seen] * p[:, None]).max() + 1e-30
                    err = np.abs(o[b, j, r] - ro[b, j, r])
                    assert (err <= tol).all(), (b, j, r, float((err / tol).max()))
                    ltol = ds + 2.0 ** -20 + len(p) * 2.0 ** -23 + abs(rl[b, j, r]) * 2.0 ** -22
                    assert abs(lse[b, j, r] - rl[b, j, r]) <= ltol, (b, j, r)
                    wtol[h, pos[seen]] += p * (2 * ds + 2.0 ** -19 + ltol + A * 2.0 ** -21)
        if got_w is not None:
            for i in range(n):
                page = table[b, i // 64]
                if 0 <= page < c["k"].shape[0]:
                    w = want_w[page, :, i % 64]
                    assert (np.abs(got_w[page, :, i % 64] - w) <= wtol[:, i] + 2.0 ** -22 * np.abs(w)).all(), (b, i)


CASES = [
    # lens, Hq, Hkv, Nq, d, causal
    ([0, 1, 15, 16, 17, 63, 64, 65, 130], 8, 2, 1, 128, True),     # 4 rows per KV head
    ([1000, 333], 8, 1, 1, 128, True),                              # exactly one tile of 8
    ([300, 5], 9, 1, 1, 64, True),                                  # 9 rows in a chunk of 16
    ([257], 4, 2, 8, 128, True),                                    # 16 rows, eight new tokens
    ([3, 200], 4, 4, 5, 64, True),                                  # more new tokens than keys
    ([190, 70], 17, 1, 1, 128, False),                              # 17 rows: three chunks of 8, the last nearly empty
    ([700], 32, 1, 2, 128, True),                                   # 64 rows: four chunks of 16
    ([129], 33, 1, 1, 64, True),
    ([150, 2], 64, 1, 2, 128, True),                                # the most rows: 128
    ([400, 65], 6, 3, 3, 256, True),                                # wide
    ([100], 20, 1, 1, 256, True),                                   # wide: two chunks of 16
    ([128, 40], 2, 2, 1, 16, True),                                 # the narrowest
    ([97, 260], 4, 4, 2, 48, True),
    ([97, 260], 4, 2, 1, 80, False),
    ([333, 1], 4, 2, 2, 192, True),
    ([70, 77, 88, 100, 146], 16, 16, 1, 48, True),                  # fewer units than CTAs
]


@pytest.mark.parametrize("lens,Hq,Hkv,Nq,d,causal", CASES)
def test_attention_and_weights(fa, lens, Hq, Hkv, Nq, d, causal):
    c, table = make(sum(lens) + d + Hq, lens, Hkv, d)
    c["weight"][np.isnan(c["weight"])] = 7.0                          # stays where no token is
    q = bf16(np.random.default_rng(d), len(lens), Hq, Nq, d)
    g = to_gpu(fa, c)
    scale = d ** -0.5
    o, lse = fa.fwd_cache8(q.to(DEV), g, ints(table), ints(lens), causal=causal, weight_decay=0.75)
    again = fa.fwd_cache8(q.to(DEV), g._replace(weight=None), ints(table), ints(lens), causal=causal)
    fa.check_device_status()
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])    # the same bits, with weights or without
    w = f64(g.weight)
    check_attention(c, q, table, lens, causal, scale, o, lse, None, w, 0.75)
    held = np.zeros(w.shape, bool)
    for b, n in enumerate(lens):
        for i in range(n):
            held[table[b, i // 64], :, i % 64] = True
    assert (w[~held] == 7.0).all()


@pytest.mark.parametrize("spread,po2", [(30, True), (2, False)])
def test_scales_far_apart_and_of_any_value(fa, spread, po2):
    lens = [500, 130]
    c, table = make(3, lens, 2, 128, spread=spread, po2=po2)
    q = bf16(np.random.default_rng(1), 2, 8, 1, 128)
    o, lse = fa.fwd_cache8(q.to(DEV), to_gpu(fa, c), ints(table), ints(lens))
    check_attention(c, q, table, lens, True, 128 ** -0.5, o, lse, None)


def test_sharp_logits_and_rows_of_every_magnitude(fa):
    """Logits in the hundreds (the softmax is nearly one-hot), rows of q from 1e-30 to 1e3, zeros among them."""
    lens = [900]
    c, table = make(5, lens, 1, 128)
    q = bf16(np.random.default_rng(2), 1, 8, 1, 128).float()
    q *= torch.tensor([1e-30, 1e-6, 0.0, 1.0, 10.0, 100.0, 1e3, 2.0 ** -10]).view(1, 8, 1, 1)
    q = q.to(torch.bfloat16)
    o, lse = fa.fwd_cache8(q.to(DEV), to_gpu(fa, c), ints(table), ints(lens))
    check_attention(c, q, table, lens, True, 128 ** -0.5, o, lse, None)


def test_a_row_of_nan_or_infinity_stays_alone(fa):
    lens = [100, 70]
    c, table = make(6, lens, 2, 64)
    q = bf16(np.random.default_rng(3), 2, 4, 1, 64)
    g = to_gpu(fa, c)
    want, wl = fa.fwd_cache8(q.to(DEV), g, ints(table), ints(lens))
    q[0, 1, 0, 5] = float("nan")
    q[1, 2, 0, 7] = float("inf")
    got, gl = fa.fwd_cache8(q.to(DEV), g, ints(table), ints(lens))
    same = torch.ones(2, 4, dtype=torch.bool)
    same[0, 1] = same[1, 2] = False
    assert torch.equal(got[same.to(DEV)], want[same.to(DEV)]) and torch.equal(gl[same.to(DEV)], wl[same.to(DEV)])
    assert torch.isnan(got[0, 1]).all() and torch.isnan(got[1, 2]).all()


def test_absent_blocks_and_lengths_past_the_table(fa):
    lens = [300, 200, 100]
    c, table = make(7, lens, 2, 64, spare=0)
    table[0, 1], table[1, 0], table[2, 0] = -1, c["k"].shape[0], 2 ** 30
    table[2, 1] = -5
    asked = [300, 10 ** 6, 100]                       # the second one: all that its table holds
    held = [300, table.shape[1] * 64, 100]
    for b, n in enumerate(held):                      # no NaN codes under what is now held
        for i in range(-(-n // 64)):
            if 0 <= table[b, i] < c["k"].shape[0]:
                for x in ("k", "v"):
                    y = c[x][table[b, i]]
                    y[y == NAN] = 0x30
    q = bf16(np.random.default_rng(4), 3, 4, 1, 64)
    g = to_gpu(fa, c)
    before = g.weight.clone()
    o, lse = fa.fwd_cache8(q.to(DEV), g, ints(table), ints(asked), weight_decay=0.0)
    fa.check_device_status()
    check_attention(c, q, table, held, True, 64 ** -0.5, o, lse, None, f64(g.weight), 0.0)
    assert (o[2] == 0).all() and torch.isneginf(lse[2]).all()
    untouched = np.setdiff1d(np.arange(c["k"].shape[0]), table[(table >= 0) & (table < c["k"].shape[0])])
    assert torch.equal(g.weight[untouched].nan_to_num(9), before[untouched].nan_to_num(9))


def test_long_sequences_are_split_and_give_the_same_bits_every_time(fa):
    """Lengths far apart, so that parts end inside sequences; sampled rows against the oracle."""
    lens = [20000, 3, 700, 9001]
    c, table = make(8, lens, 2, 128)
    q = bf16(np.random.default_rng(5), 4, 8, 1, 128)
    g = to_gpu(fa, c)
    o, lse = fa.fwd_cache8(q.to(DEV), g, ints(table), ints(lens))
    for _ in range(3):
        o2, l2 = fa.fwd_cache8(q.to(DEV), g, ints(table), ints(lens))
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    check_attention(c, q, table, lens, True, 128 ** -0.5, o, lse, None)


def test_a_long_tail_of_small_probabilities_counts(fa):
    """One key takes nearly all of the softmax and 131071 share the rest, each 2^-23.5 of it: O is the tail's alone.
    P is off by at most 2^-25 of the largest and 2^-12 of itself, so O by n 2^-25 max|V| + 2^-11 p|V| (P and l), and 2^-8 |O|."""
    n, d = 131072, 64
    P = n // 64
    c = {"k": np.zeros((P, 1, 64, d), np.uint8), "v": np.full((P, 1, 64, d), 0x38, np.uint8),      # 0x38: 1.0
         "k_scale": np.ones((P, 1), np.float32), "v_scale": np.ones((P, 1), np.float32)}
    table = np.random.default_rng(13).permutation(P)[None].astype(np.int32)
    first = table[0, 777], 0, 21                       # the heavy key, somewhere in the middle
    c["k"][first], c["v"][first] = 0x38, 0
    q = torch.full((1, 2, 1, d), 23.5 * np.log(2) / d, dtype=torch.bfloat16)
    s = f64(q)[0, 0, 0].sum()
    o, lse = fa.fwd_cache8(q.to(DEV), to_gpu(fa, c), ints(table), ints([n]), scale=1.0)
    tail = (n - 1) * np.exp(-s)
    want = tail / (1 + tail)
    assert np.abs(f64(o) - want).max() <= 2.0 ** -8 * want + 2.0 ** -11 * want + n * 2.0 ** -25
    assert np.abs(f64(lse) - (s + np.log1p(tail))).max() <= (d + 8) * 2.0 ** -23 * s + n * 2.0 ** -23 * want + 2.0 ** -20 * s


@pytest.mark.parametrize("lens,Hq,Hkv,Nq,d", [
    ([0, 200, 64, 1, 700, 65, 330] * 10, 4, 2, 1, 64),              # more sequences than a warp has lanes
    ([1100, 900] * 20, 2, 1, 1, 128),                               # the same, several tiles a part
    ([1500, 10, 2500, 0, 800] * 2, 4, 2, 2, 256),                   # row groups of one block among long ones
    ([3000, 2000], 40, 2, 2, 128),                                  # five chunks of 8 rows each
    ([3000, 2000], 32, 2, 2, 128),                                  # two of 16
    ([4000, 100, 2500, 3100], 8, 2, 1, 64),                         # four rows: three CTAs per SM
    ([1700, 2900], 3, 1, 5, 256),                                   # fifteen rows: one
])
def test_many_row_groups_split_between_ctas(fa, lens, Hq, Hkv, Nq, d):
    c, table = make(sum(lens) + d, lens, Hkv, d)
    q = bf16(np.random.default_rng(14), len(lens), Hq, Nq, d)
    g = to_gpu(fa, c)
    o, lse = fa.fwd_cache8(q.to(DEV), g, ints(table), ints(lens), weight_decay=0.5)
    fa.check_device_status()
    check_attention(c, q, table, lens, True, d ** -0.5, o, lse, None, f64(g.weight), 0.5)


@pytest.mark.parametrize("Hq,Nq,d", [(1, 1, 128), (128, 1, 256), (16, 8, 64)])
def test_one_block_one_head(fa, Hq, Nq, d):
    """A single unit of work: nothing to join; the most rows, in eight chunks."""
    c, table = make(20 + d, [37], 1, d, spare=0)
    q = bf16(np.random.default_rng(21), 1, Hq, Nq, d)
    g = to_gpu(fa, c)
    o, lse = fa.fwd_cache8(q.to(DEV), g, ints(table), ints([37]), weight_decay=0.25)
    fa.check_device_status()
    check_attention(c, q, table, [37], True, d ** -0.5, o, lse, None, f64(g.weight), 0.25)


def test_scales_of_zero(fa):
    """Blocks whose K or V scale is 0 hold zeros: logits of 0, values of 0."""
    lens = [200, 100]
    c, table = make(22, lens, 1, 64)
    c["k_scale"][table[0, 1]] = 0.0
    c["v_scale"][table[0, 2]] = c["v_scale"][table[1, :2]] = 0.0
    q = bf16(np.random.default_rng(23), 2, 2, 1, 64)
    o, lse = fa.fwd_cache8(q.to(DEV), to_gpu(fa, c), ints(table), ints(lens))
    check_attention(c, q, table, lens, True, 64 ** -0.5, o, lse, None)
    assert (o[1] == 0).all() and torch.isfinite(lse).all()


def test_evict_follows_lengths_in_a_graph(fa):
    lens, keep, recent = [9000, 300], 200, 16
    c, table = make(24, lens, 2, 16, spare=4)
    to, table = table[:, -4:].copy(), table[:, :-4].copy()
    g, n = to_gpu(fa, c), ints(lens)
    scratch = to_gpu(fa, c)
    fa.cache8_evict(scratch, ints(table), n, keep, recent, ints(to))
    tb, tt = ints(table), ints(to)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new, kept = fa.cache8_evict(g, tb, n, keep, recent, tt)
    for lens in ([9000, 300], [150, 257], [0, 201]):
        n.copy_(ints(lens))
        graph.replay()
        torch.cuda.synchronize()
        want, wn, wk = oc.evict(c, table, lens, keep, recent, to)
        assert np.array_equal(new.cpu().numpy(), wn) and np.array_equal(kept.cpu().numpy(), wk)
        for b in range(2):
            for i in range(int(wn[b])):
                page = to[b, i // 64], slice(None), i % 64
                assert np.array_equal(g.k.cpu().numpy()[page], want["k"][page])


def test_sequences_may_share_blocks(fa):
    """A prefix of two blocks in two tables: each sequence's result is what it gets from blocks of its own."""
    c, table = make(15, [200, 200, 200], 2, 64, spare=0)
    for x in ("k", "v", "k_scale", "v_scale"):
        for i in range(2):
            c[x][table[1, i]] = c[x][table[0, i]]
    q = bf16(np.random.default_rng(16), 3, 4, 1, 64).to(DEV)
    g = to_gpu(fa, c)
    want = fa.fwd_cache8(q, g, ints(table), ints([200, 190, 200]))
    table[1, :2] = table[0, :2]
    got = fa.fwd_cache8(q, g, ints(table), ints([200, 190, 200]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_graphs_may_share_a_workspace_one_after_the_other(fa):
    lens = [700, 90]
    c, table = make(17, lens, 2, 128)
    g, tb, n = to_gpu(fa, c), ints(table), ints(lens)
    qs = [bf16(np.random.default_rng(i), 2, 8, 1, 128).to(DEV) for i in range(2)]
    want = [fa.fwd_cache8(q, g, tb, n) for q in qs]
    size = fa.load().fa_fwd_cache8_workspace_bytes(2, 8, 2, 1, 128, table.shape[1], 0)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)      # NaN wherever it is read as floats
    graphs, outs = [], []
    for q in qs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(fa.fwd_cache8(q, g, tb, n, workspace=ws))
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_stalled_call_reports_and_the_next_one_works(fa, monkeypatch):
    lens = [700, 90]
    c, table = make(18, lens, 2, 128)
    q = bf16(np.random.default_rng(19), 2, 8, 1, 128).to(DEV)
    g = to_gpu(fa, c)
    want = fa.fwd_cache8(q, g, ints(table), ints(lens))
    for decay in (None, 0.0):
        monkeypatch.setenv("FA_TEST_STALL", "1")
        fa.fwd_cache8(q, g, ints(table), ints(lens), weight_decay=decay)
        with pytest.raises(fa.FAError) as e:
            fa.check_device_status()
        assert e.value.code == 5
        monkeypatch.setenv("FA_TEST_STALL", "0")
        got = fa.fwd_cache8(q, g, ints(table), ints(lens))
        fa.check_device_status()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_pool_offsets_past_32_bits(fa):
    """A pool of more than 2^32 codes: the last blocks hold the sequence."""
    Hkv, d, P = 8, 256, 33000
    free, _ = torch.cuda.mem_get_info()
    assert P * Hkv * 64 * d > 2 ** 32 and free > 30 << 30
    lens = [150]
    c, table = make(9, lens, Hkv, d)
    small = c["k"].shape[0]
    big = fa.new_cache8(P, Hkv, d, weight=True)
    for n, x in c.items():
        getattr(big, n)[P - small:] = torch.from_numpy(x).to(DEV)
    q = bf16(np.random.default_rng(6), 1, 16, 1, d).to(DEV)
    far = table + (P - small)
    want = fa.fwd_cache8(q, to_gpu(fa, c), ints(table), ints(lens))
    got = fa.fwd_cache8(q, big, ints(far), ints(lens), weight_decay=0.5)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    k = bf16(np.random.default_rng(7), Hkv, 3, d).to(DEV)
    fa.cache8_append(big, k, k, ints([0, 3]), ints(far), ints([150]))
    near = to_gpu(fa, c)
    fa.cache8_append(near, k, k, ints([0, 3]), ints(table), ints([150]))
    assert torch.equal(big.k[P - small:], near.k) and torch.equal(big.v_scale[P - small:], near.v_scale)
    to = ints([[1, 2]])
    fa.cache8_evict(big, ints(far), ints([150]), 100, 10, to)
    # (compared through a pool that has the destinations among its own blocks)
    free_blocks = np.setdiff1d(np.arange(small), table)[:2]
    ref, _, _ = oc.evict({n: getattr(big, n)[P - small:].cpu().numpy() for n in c}, table, [150], 100, 10, free_blocks[None])
    assert np.array_equal(big.k[1].cpu().numpy(), ref["k"][free_blocks[0]])
    assert np.array_equal(big.k[2, :, :36].cpu().numpy(), ref["k"][free_blocks[1], :, :36])


APPENDS = [
    # new tokens, tokens there, Hkv, d, token-major
    ([1, 1, 1, 1], [0, 5, 63, 64], 2, 128, True),
    ([70, 0, 1, 200], [3, 10, 127, 0], 3, 64, True),
    ([64], [64], 1, 256, False),
    ([65, 62], [63, 2], 2, 16, False),
    ([129, 3], [30, 61], 5, 80, True),
    ([40], [0], 1, 192, True),
    ([1, 0, 3, 70, 0] * 20, [0, 64, 62, 10, 5] * 20, 2, 32, True),          # more sequences than a warp has lanes
]


@pytest.mark.parametrize("new,past,Hkv,d,token_major", APPENDS)
def test_append_bit_for_bit(fa, new, past, Hkv, d, token_major):
    c, table = make(sum(new) + d, [a + b for a, b in zip(new, past)], Hkv, d, spread=1)
    rng = np.random.default_rng(d)
    T = sum(new)
    mult = np.exp2(rng.integers(-8, 8, (Hkv, T, 1)))                   # some blocks' scales grow, some don't
    k, v = (torch.from_numpy((rng.standard_normal((Hkv, T, d)) * mult).astype(np.float32)).to(torch.bfloat16) for _ in range(2))
    cu = np.concatenate([[0], np.cumsum(new)])
    g = to_gpu(fa, c)
    put = (lambda x: x.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)) if token_major else (lambda x: x.to(DEV))
    fa.cache8_append(g, put(k), put(v), ints(cu), ints(table), ints(past))
    fa.check_device_status()
    want = oc.append(c, f64(k), f64(v), cu, past, table)
    for n in c:
        got = getattr(g, n).cpu().numpy()
        assert np.array_equal(got.view(np.uint32) if got.dtype == np.float32 else got,
                              want[n].view(np.uint32) if got.dtype == np.float32 else want[n]), n


def test_append_specials(fa):
    """Zeros, infinities, NaN, the smallest values; positions past the table, absent blocks, zeros over a held scale."""
    Hkv, d = 1, 16
    c, table = make(11, [64, 64, 64], Hkv, d, spare=0)
    table[2, 0] = -1
    k = torch.zeros(Hkv, 12, d, dtype=torch.bfloat16)
    k[0, 0, :4] = torch.tensor([float("inf"), float("-inf"), float("nan"), 3.0])
    k[0, 1] = 2.0 ** -133                                              # the smallest bf16
    k[0, 4:8, 3] = 5.0
    cu, start = [0, 2, 6, 12], [0, 62, 0]                              # seq 1: two of four past its table
    g = to_gpu(fa, c)
    fa.cache8_append(g, k.to(DEV), -k.to(DEV), ints(cu), ints(table), ints(start))
    want = oc.append(c, f64(k), -f64(k), cu, start, table)
    for n in ("k_scale", "v_scale", "weight"):
        assert np.array_equal(getattr(g, n).cpu().numpy(), want[n], equal_nan=True), n
    for n in ("k", "v"):
        got = getattr(g, n).cpu().numpy()
        nan = (want[n] & 0x7F) == NAN
        assert np.array_equal(got[~nan], want[n][~nan]) and ((got[nan] & 0x7F) == NAN).all()


def test_appending_one_by_one_is_appending_at_once(fa):
    """Power-of-two scales: tokens appended one at a time leave the codes of one append, but for values that became
    subnormal on the way."""
    Hkv, d, n = 2, 64, 100
    rng = np.random.default_rng(12)
    x = torch.from_numpy((rng.standard_normal((Hkv, n, d)) * np.linspace(1, 8, n)[None, :, None]).astype(np.float32)).to(torch.bfloat16).to(DEV)
    a, b = fa.new_cache8(2, Hkv, d), fa.new_cache8(2, Hkv, d)
    table = ints([[1, 0]])
    fa.cache8_append(a, x, x, ints([0, n]), table, ints([0]))
    for i in range(n):
        fa.cache8_append(b, x[:, i:i + 1], x[:, i:i + 1], ints([0, 1]), table, ints([i]))
    assert torch.equal(a.k_scale, b.k_scale)
    va, vb = (z.k.view(torch.float8_e4m3fn).float() for z in (a, b))
    assert torch.equal(va[vb.abs() >= 2.0 ** -6], vb[vb.abs() >= 2.0 ** -6]) and (va - vb).abs().max() <= 2.0 ** -9


EVICTS = [
    # lens, keep, recent, Hkv, d
    ([517, 192], 130, 32, 4, 64),
    ([5000, 1, 0, 64, 65], 64, 0, 2, 128),
    ([3000], 100, 100, 1, 16),            # only the recent ones
    ([1025, 1024], 1023, 1, 2, 80),
    ([300], 300, 10, 3, 256),             # nothing to drop
    ([70, 9], 1, 0, 1, 192),
    ([200, 0, 64, 130] * 12, 100, 7, 2, 16),
]


@pytest.mark.parametrize("lens,keep,recent,Hkv,d", EVICTS)
@pytest.mark.parametrize("ties", [False, True])
def test_evict_bit_for_bit(fa, lens, keep, recent, Hkv, d, ties):
    room = -(-keep // 64)
    c, table = make(sum(lens) + keep, lens, Hkv, d, spare=room)
    to, table = table[:, -room:].copy(), table[:, :-room].copy()
    if ties:
        c["weight"] = np.where(np.isnan(c["weight"]), np.nan, np.floor(c["weight"] * 6)).astype(np.float32)
        c["weight"][table[0, 0], :, :3] = [-0.0, np.nan, np.inf] if lens[0] > 3 else 0
    g = to_gpu(fa, c)
    new, kept = fa.cache8_evict(g, ints(table), ints(lens), keep, recent, ints(to))
    fa.check_device_status()
    want, wn, wk = oc.evict(c, table, lens, keep, recent, to)
    assert np.array_equal(new.cpu().numpy(), wn) and np.array_equal(kept.cpu().numpy(), wk)
    for n in c:
        assert np.array_equal(getattr(g, n).cpu().numpy(), want[n], equal_nan=want[n].dtype == np.float32), n


@pytest.mark.parametrize("lens,keep,recent,Hkv", [
    ([9000, 20000, 100, 8193], 3000, 77, 2),          # several CTAs share a sequence; one has less than a stretch
    ([8300], 8299, 0, 1),                             # all but one
    ([8300], 8200, 8199, 1),                          # one besides the recent ones
    ([430001], 66000, 64, 1),                         # more keys than the CTAs' shared memory holds
    ([5000, 4097, 4300, 64] * 3, 700, 5, 3),
    ([9000, 8193] + [10] * 158, 900, 0, 1),           # more sequences than SMs
])
@pytest.mark.parametrize("ties", [False, True])
def test_evict_long_caches(fa, lens, keep, recent, Hkv, ties):
    test_evict_bit_for_bit(fa, lens, keep, recent, Hkv, 16, ties)


def test_evict_with_absent_blocks(fa):
    lens, keep = [200], 120
    c, table = make(21, lens, 2, 64, spare=2)
    to, table = table[:, -2:].copy(), table[:, :-2].copy()
    table[0, 1] = -1                                   # its tokens count with weight 0
    to[0, 1] = c["k"].shape[0]                         # nowhere to write the second block
    g = to_gpu(fa, c)
    new, kept = fa.cache8_evict(g, ints(table), ints(lens), keep, 5, ints(to))
    fa.check_device_status()
    want, wn, wk = oc.evict(c, table, lens, keep, 5, to)
    assert np.array_equal(kept.cpu().numpy(), wk)
    for n in c:
        assert np.array_equal(getattr(g, n).cpu().numpy(), want[n], equal_nan=want[n].dtype == np.float32), n


def _serve(fa, g, table, steps, q, k, start):
    """steps tokens appended and attended to, one by one, weights added up."""
    n = torch.full((1,), start, dtype=torch.int32, device=DEV)
    cu = ints([0, 1])
    out = []
    for i in range(steps):
        fa.cache8_append(g, k[:, i:i + 1], k[:, i:i + 1], cu, table, n)
        n = n + 1
        out.append(fa.fwd_cache8(q[i:i + 1], g, table, n, weight_decay=1.0)[0])
    return torch.cat(out), n


def test_serving_run_prompt_steps_evict_steps(fa):
    """Prompt tokens written, steps that append and attend, an eviction, steps on the smaller cache: against the
    oracle's run of the same calls."""
    Hq, Hkv, d, n0, steps = 4, 2, 64, 90, 6
    rng = np.random.default_rng(31)
    kp, ks, q = bf16(rng, Hkv, n0, d), bf16(rng, Hkv, 2 * steps, d), bf16(rng, 2 * steps, Hq, 1, d)
    g = fa.new_cache8(6, Hkv, d, weight=True)
    c = {n: getattr(g, n).cpu().numpy() for n in ("k", "v", "k_scale", "v_scale", "weight")}
    table, to = np.array([[4, 1]], np.int32), np.array([[0, 3]], np.int32)
    fa.cache8_append(g, kp.to(DEV), kp.to(DEV), ints([0, n0]), ints(table), ints([0]))
    o1, n = _serve(fa, g, ints(table), steps, q[:steps].to(DEV), ks[:, :steps].to(DEV), n0)
    held = {x: getattr(g, x).cpu().numpy() for x in c}
    new, kept = fa.cache8_evict(g, ints(table), n, 40, 8, ints(to))
    assert int(new) == 40
    o2, n = _serve(fa, g, ints(to), steps, q[steps:].to(DEV), ks[:, steps:].to(DEV), 40)
    fa.check_device_status()
    c = oc.append(c, f64(kp), f64(kp), [0, n0], [0], table)
    for i in range(steps):
        c = oc.append(c, f64(ks)[:, i:i + 1], f64(ks)[:, i:i + 1], [0, 1], [n0 + i], table)
        check_attention(c, q[i:i + 1], table, [n0 + i + 1], True, d ** -0.5, o1[i:i + 1],
                        torch.from_numpy(oc.attend(c, f64(q[i:i + 1]), table, [n0 + i + 1], True, d ** -0.5)[1]), None)
    for x in ("k", "v", "k_scale", "v_scale"):
        assert np.array_equal(held[x], c[x]), x
    c, _, wk = oc.evict(held, table, [n0 + steps], 40, 8, to)           # by the GPU's own weights
    assert np.array_equal(kept.cpu().numpy(), wk)
    for i in range(steps):
        c = oc.append(c, f64(ks)[:, steps + i:steps + i + 1], f64(ks)[:, steps + i:steps + i + 1], [0, 1], [40 + i], to)
        j = steps + i
        check_attention(c, q[j:j + 1], to, [41 + i], True, d ** -0.5, o2[i:i + 1],
                        torch.from_numpy(oc.attend(c, f64(q[j:j + 1]), to, [41 + i], True, d ** -0.5)[1]), None)


def test_captured_step_replays(fa):
    """Append and attention captured into a graph; replays follow the buffers, the lengths on the device among them."""
    lens = [130, 64]
    c, table = make(41, [n + 8 for n in lens], 2, 128)
    rng = np.random.default_rng(42)
    k, q = bf16(rng, 2, 8, 128).to(DEV), bf16(rng, 2, 8, 1, 128).to(DEV)
    cu, tb = ints([0, 1, 2]), ints(table)

    def step(g, x, q, n):
        fa.cache8_append(g, x, x, cu, tb, n)
        return fa.fwd_cache8(q, g, tb, n + 1, weight_decay=0.5)

    want_g, n = to_gpu(fa, c), ints(lens)
    want = []
    for i in range(4):
        want.append([t.clone() for t in step(want_g, k[:, 2 * i:2 * i + 2], q, n + i)])
    g = to_gpu(fa, c)
    x, n = k[:, :2].clone(), ints(lens)
    side = torch.cuda.Stream()
    scratch = to_gpu(fa, c)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(scratch, x, q, n)
    torch.cuda.current_stream().wait_stream(side)
    graph, graph2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(g, x, q, n)
    with torch.cuda.graph(graph2):                       # a second one alive, on another cache
        step(scratch, x, q, n)
    for i in range(4):
        x.copy_(k[:, 2 * i:2 * i + 2])
        n.copy_(ints(lens) + i)
        graph.replay()
        graph2.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[i][0]) and torch.equal(out[1], want[i][1]), i
    assert torch.equal(g.weight.nan_to_num(3), want_g.weight.nan_to_num(3)) and torch.equal(g.k, want_g.k)


def test_threads_and_streams_match_solo_runs(fa):
    data = []
    for i, (lens, Hq, Hkv, d) in enumerate([([700, 20], 8, 2, 128), ([300], 4, 4, 64), ([500, 90, 8], 8, 1, 256)]):
        c, table = make(50 + i, lens, Hkv, d)
        data.append((to_gpu(fa, c), ints(table), ints(lens), bf16(np.random.default_rng(i), len(lens), Hq, 1, d).to(DEV)))
    solo = [fa.fwd_cache8(q, g, t, n) for g, t, n, q in data]
    torch.cuda.synchronize()
    got, errors = [None] * 3, []

    def worker(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    g, t, n, q = data[i]
                    got[i] = fa.fwd_cache8(q, g, t, n)
                torch.cuda.current_stream().synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=worker, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(got, solo):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
